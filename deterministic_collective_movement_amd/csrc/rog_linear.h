// rog_linear.h -- kernel arguments and launch plans of the policy head's
// products (token log probabilities from hidden states, their gradient, the
// product of 8-bit integers), shared by the host planner (rog_linear_plan.cpp)
// and the HIP kernels.  Internal to librog.so; the public interface is
// include/rog.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rog_head.h"

namespace rog {

// How a product is cut.  A step is 64 bytes of K (32 elements of two bytes, 64 of
// one), what a matrix instruction takes of 16 rows.  A leaf is 32
// consecutive columns of one shard, a block four leaves.  Every logit is one
// chain of matrix instructions over the steps in rising order, whatever the
// tile, so its bits do not depend on how many rows a call has; the statistics
// of a row are joined leaf by leaf over one tree (rog_linear_device.h).
constexpr uint32_t kStepBytes = 64;
constexpr uint32_t kPackUnit = 128;        // bytes of a packed row are a multiple of these, a line
constexpr uint32_t kLeaf = 32;
constexpr uint32_t kLinearBlock = 128;
constexpr uint64_t kMaxLinearStride = uint64_t(1) << 22;   // bytes from a row to the next: tiles are addressed in 32 bits
constexpr uint32_t kMaxDim = 1u << 17;

// A head's weight shards, cut into tiles of `tile` columns (the launch's).
struct WeightShard {
    const void *w;                     // element (0, 0)
    int64_t stride;                    // bytes from a column's weights to the next column's
    uint32_t width;                    // columns
    uint32_t col0;                     // the shard's first column in the row
};
struct WeightShards {
    uint32_t W;
    uint32_t vocab;
    WeightShard s[kMaxPeers];
    uint32_t tile0[kMaxPeers + 1];     // the shard's first tile; [W]: all tiles
    uint32_t block0[kMaxPeers + 1];    // the shard's first block of 128 columns
};

// The states of a call: rows of `dim` elements.
struct LinearRows {
    const void *x;
    int64_t stride;                    // bytes
    const uint32_t *count;             // device: how many rows there are (NULL: `rows`)
    uint32_t rows;
    uint32_t kbytes;                   // bytes of a row
};

struct ScoreArgs {
    LinearRows a;
    const int64_t *tokens;             // of row i (NULL: none)
    const uint32_t *index;             // packed rows: the caller's row (NULL: row i itself)
    float scale;                       // log2(e) / temperature
    float *target;                     // [rows] logit of the row's token
    float *rests;                      // [rows][4] as a state: the token's block without it, and the block's number
    float *states;                     // m, s, t, 0 of a row's block at row * row_step + block * block_step, in fours
    uint32_t row_step, block_step;
    WeightShards sh;
};

// Joins the units of every row.
struct JoinArgs {
    const int64_t *tokens;
    const uint32_t *index, *count;
    const float *target, *rests, *states;
    float *logp, *entropy, *lse;
    uint32_t rows, row_step, block_step;
    uint32_t vocab, blocks;
    float scale;
};

// Packs the rows that are scored, one after the other, K padded with zeros to whole lines.
struct PackArgs {
    const void *x;
    int64_t stride;
    const int64_t *tokens;
    uint32_t rows, kbytes;             // bytes of a caller's row
    uint32_t packed_bytes;             // of a packed one
    uint32_t *index, *count;
    void *packed;
    float *logp, *entropy, *lse;       // zeroed where the row is not scored
    void *zero;                        // rows of kbytes, likewise
    int64_t zero_stride;
    const float *g_logp, *g_entropy;   // binary16: the largest of them sets the scale
    float *g_scale;
    float inv_t;
    uint32_t *parts;                   // of the weights' sums: weight_parts() of the scored rows (NULL: not wanted)
    uint32_t dim_tiles, tiles, seg_tiles;
};

struct GradArgs {
    LinearRows a;                      // packed
    const int64_t *tokens;
    const uint32_t *index;
    const float *lse, *entropy, *g_logp, *g_entropy, *g_scale;
    float inv_t, scale;                // 1 / temperature, log2(e) / temperature
    void *g, *g_all;                   // [rows][g_stride / 2] coefficients of the piece's columns; binary16: by the rows' own
                                       // scales, and by that of all (else one array)
    int64_t g_stride;                  // bytes
    uint32_t tile_begin;               // the piece's first tile
    uint32_t tiles;                    // and how many it has
    WeightShards sh;
};

// One launch of the gradient's products for a piece.
struct BackArgs {
    LinearRows a;                      // packed
    const uint32_t *index;
    const float *g_logp, *g_entropy, *g_scale;
    float inv_t;
    const void *g, *g_all;
    int64_t g_stride;
    uint32_t tile_begin, tiles;
    uint32_t seg_begin, segs;          // segments of the piece
    uint32_t row_tiles, dim_tiles;     // upper bounds of the grid
    float *part;                       // sums of d_hidden: of each of the piece's segments [rows][dim_pad], or running ones
    uint64_t part_seg;                 // floats from a segment's to the next (0: running)
    uint32_t dim_pad;
    uint32_t first, last;              // the running sum's first and last piece
    void *d_hidden;
    int64_t d_stride;
    uint32_t dim;
    WeightShards sh;
    uint32_t seg0[kMaxPeers + 1];      // a shard's first segment
    uint32_t seg_tiles;                // tiles of a segment
    void *dw[kMaxPeers];
    int64_t dw_stride[kMaxPeers];      // bytes
    uint32_t splits;                   // parts of the rows that the weights' gradients are summed over apart, at most
    const uint32_t *parts;             // device: how many there are (read if there may be several)
    float *dw_part;                    // their sums: [splits][columns of the piece][dim_pad], if there are several
    uint64_t dw_part_split;            // floats from a part's to the next
};

// Adds a piece's partial sums to the running ones in the segments' order; after the last piece to d_hidden.
struct BackJoinArgs {
    const float *part;
    float *running;
    uint64_t part_seg;
    uint32_t segs, dim_pad, dim;
    uint32_t first, last;
    const uint32_t *index, *count;
    const float *g_logp, *g_entropy;
    float inv_t;
    uint32_t rows;
    void *d_hidden;
    int64_t d_stride;
};

struct QuantizeArgs {
    const void *x;
    int64_t stride;                    // bytes
    int8_t *q;
    int64_t q_stride;
    float *scale;
    uint32_t rows, dim;
};

struct LinearI8Args {
    LinearRows a;
    const float *row_scale;
    WeightShards sh;
    const float *scale[kMaxPeers];
    void *out[kMaxPeers];
    int64_t out_stride[kMaxPeers];     // bytes
};

// Tiles of a product of weights and states: columns x rows of a workgroup, waves along each, stages of K in the
// shared memory (kWide: steps of 64 bytes multiplied from registers, else lines of 128).
template <int COLUMNS, int ROWS, int WM, int WN, int STAGES, bool WIDE>
struct Form {
    static constexpr int kColumns = COLUMNS, kRows = ROWS, kWM = WM, kWN = WN, kStages = STAGES, kThreads = 64 * WM * WN;
    static constexpr int kFM = COLUMNS / WM / 16, kFN = ROWS / WN / 16;
    static constexpr bool kWide = WIDE, kTail = COLUMNS == 256;   // the largest tile: see place_of()
    // waves that share a block of columns
    static constexpr int kShare = COLUMNS / WM < int(kLinearBlock) ? int(kLinearBlock) / (COLUMNS / WM) : 1;
    static_assert(COLUMNS % kLinearBlock == 0 && COLUMNS / WM % 32 == 0 && COLUMNS / WM <= int(kLinearBlock), "whole leaves, blocks");
};
// Up to 64 rows a call is bound by the weights' bytes: small tiles, whole lines, one or two of them in flight per
// workgroup and two workgroups per CU, which have 80 KiB of shared memory each (one 32003 x 512 bf16 head: 7.7 us, 4.2 TB/s;
// 64 rows of 131072 x 4096: 178 us, 6.1 TB/s).  Four slabs of 128 + 32 rows are those 80 KiB, and the score's and the
// coefficients' tiles have their rows' numbers beside them: three there (scores with four slabs and one workgroup per
// CU, and with three and two, us: 16 x 131072 x 4096 192.7 and 186.5, 4 x 50257 x 1600 35.6 and 31.5, 7 x 100000 x 768 40.8
// and 34.1, 3 x 65536 x 5120 122.6 and 123.5, 1 x 131072 x 2048 116 and 121.5), but where a CU has no second
// workgroup anyway (in a graph, 1 x 32003 x 512 13.6 with four and 13.95 with three, 3 x 32003 x 1024 19.1 and 19.7).  The
// 8-bit product has two with four slabs (16 x 131072 x 4096 104.7, with three 105.4).  Past that by the matrix units: 256 x 256 take 128 elements of an operand from the shared memory per
// 16 x 16 x 32 instruction and lane group, the least of the tiles tried (8192 rows of 131072 x 4096: 256 x 128 by
// eight waves 1060 TFLOP/s and by four 1134, 256 x 256 by 2 x 2 waves 1183, by 2 x 4 1380); eight waves are two per
// SIMD, with 128 accumulators of their 256 registers each.
typedef Form<128, 32, 4, 1, 3, false> FormFew;
typedef Form<128, 32, 4, 1, 4, false> FormFewDeep;
typedef Form<128, 64, 4, 1, 3, false> FormSome;
typedef Form<128, 128, 2, 2, 4, true> FormMid;
typedef Form<256, 256, 2, 4, 4, true> FormWide;
typedef Form<128, 128, 2, 4, 4, true> FormQuarter;   // of a wide tile, by as many threads
constexpr uint32_t kCus = 256;         // workgroups of the wide form that run at a time
// Tiles past the last whole round of the CUs up to which they are dealt in quarters: a round of quarters takes less than half of a
// round of tiles, and 64 tiles are one round of them (us, whole and in quarters: 1024 rows of K 1600 with 20, 40, 64, 88, 100,
// 128 and 160 tiles past the third round 188 and 179, 187 and 172, 188 and 175, 188 and 190, 189 and 190.5, 189 and 191,
// 192 and 210; of K 4096 with 40, 88, 128 and 160 past the first 188 and 155, 190 and 195, 194 and 203, 200 and 243).
constexpr uint32_t kTailSplit = 64;
enum { kFormFew = 0, kFormSome = 1, kFormMid = 2, kFormWide = 3 };

struct ScorePlan {
    int32_t form;
    uint32_t grid;
    bool direct, packs;
    PackArgs pack;
    ScoreArgs args;
    JoinArgs join;
    uint64_t workspace_bytes;
};

// Columns of a tile of the gradient's pieces.
constexpr uint32_t kGradTile = 256;
// Bytes of a piece's coefficients (one segment at least): written once and read twice, they fit the Infinity Cache, and a
// piece of a large batch is still eight rounds of the CUs and more (4096 rows of 65536 x 4096: 128, 256 and 512 MiB within 2 %).
constexpr uint64_t kPieceBytes = 256ull << 20;
constexpr uint32_t kMostPieceTiles = 4096;
// Rows of a part at least, where the weights' sums are cut: a part's sums go through memory and are joined (us, whole and in parts
// of 1024, 2048 and 4096 rows and more: 65536 x 1000 x 256 1326, 302, 254, 261; 8192 x 4000 x 320 218, 134, 124, 155;
// 4096 x 4000 x 512 128, 136, 133, 127).
constexpr uint32_t kPartRows = 2048;

// Tiles of a piece for so many rows.
__host__ __device__ inline uint32_t piece_tiles(uint64_t rows, uint32_t seg_tiles) {
    const uint64_t tiles = kPieceBytes / ((rows ? rows : 1) * kGradTile * 2);
    return uint32_t(tiles < seg_tiles ? seg_tiles : tiles > kMostPieceTiles ? kMostPieceTiles : tiles);
}

// Parts that the weights' sums over `rows` scored rows are cut into: where a piece's 256 x 256 tiles of the weights would
// leave CUs idle, as many as there are CUs for.  The sums' order goes by this, so it goes by the scored rows (which
// the device counts) and not by the rows of the call, nor by the form or the pieces that those decide.
__host__ __device__ inline uint32_t weight_parts(uint32_t rows, uint32_t dim_tiles, uint32_t tiles, uint32_t seg_tiles) {
    const uint32_t piece = piece_tiles(rows, seg_tiles), sums = dim_tiles * (tiles < piece ? tiles : piece);
    const uint32_t idle = kCus / sums, most = rows / kPartRows, parts = idle < most ? idle : most;
    return parts ? parts : 1;
}

struct GradPlan {
    rog_dtype dtype;
    int32_t form;                      // few and some: up to 64 rows; mid: few tiles; wide
    bool direct, direct_back, running;
    uint32_t pieces, piece_tiles;      // tiles of a piece: whole segments' or all
    PackArgs pack;
    GradArgs coef;
    BackArgs back;
    BackJoinArgs join;
    uint64_t workspace_bytes;
};

struct LinearI8Plan {
    int32_t form;
    uint32_t grid;
    bool direct;
    LinearI8Args args;
};

// Validate and plan (no HIP calls); without `addresses` only what the shapes decide.
rog_status plan_linear_logprob(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim, const rog_weight_shard *shards, int W,
                               rog_dtype dtype, float temperature, const int64_t *tokens, const rog_logprob_out *out, void *workspace,
                               size_t workspace_bytes, bool addresses, bool has_tokens, ScorePlan *p);
rog_status plan_linear_grad(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim, const rog_weight_shard *shards, int W,
                            rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse, const float *entropy,
                            const float *g_logp, const float *g_entropy, void *d_hidden, int64_t d_hidden_stride,
                            const rog_grad_shard *d_weights, void *workspace, size_t workspace_bytes, bool addresses, GradPlan *p);
// Workgroups of a piece's launches.
struct PieceGrid {
    uint32_t coefficients, states, weights, join, weights_join;
};
// Sets coef and back to piece i (pieces are laid one after the other).
PieceGrid lay_piece(GradPlan *p, uint32_t i);
rog_status plan_quantize(const void *x, int64_t row_stride, size_t rows, int64_t dim, rog_dtype dtype, int8_t *q, int64_t q_stride,
                         float *scale, QuantizeArgs *a);
rog_status plan_linear_i8(const int8_t *q, int64_t q_stride, const float *scale, size_t rows, int64_t dim, const rog_i8_shard *shards, int W,
                          rog_dtype out_dtype, const rog_grad_shard *out, LinearI8Plan *p);

hipError_t launch_pack(const PackArgs &a, hipStream_t s);
hipError_t launch_coefficients(const GradPlan &p, const GradArgs &a, uint32_t grid, hipStream_t s);

static_assert(sizeof(BackArgs) <= 4096 && sizeof(LinearI8Args) <= 4096, "kernel arguments stay below 4 KiB");

}  // namespace rog
