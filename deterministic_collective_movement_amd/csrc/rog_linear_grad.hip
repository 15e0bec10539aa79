// rog_linear_grad.hip -- HIP kernels of the gradient of token log probabilities
// in hidden states and head weights for gfx950 (CDNA4), and the C entry point
// that launches them.
//
// With the coefficients G_ij = (g_i (1[j = t_i] - p_ij) - e_i p_ij (log p_ij + H_i)) / T
// (rog_linear_score.hip makes them anew from the states and weights, a piece of
// the vocabulary at a time, rounded to the weights' type as the matrix units take
// them):
//     dw_j = sum_i G_ij h_i          dh_i = sum_j G_ij w_j
// One launch takes both products of a piece; they share nothing but G.
#include <hip/hip_runtime.h>

#include "rog_linear_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

typedef __attribute__((address_space(1))) f32x4 gf32x4_out;
typedef __attribute__((address_space(1))) uint16_t gu16_out;

// Eight outputs, rounded once, to `to` (the first `n` of them).
template <int DT>
__device__ __forceinline__ void put8(uint8_t *to, const float (&x)[8], uint32_t n) {
    vec16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = narrow_word<DT>(x + 2 * i);
    if (n >= 8) {
        *(gvec16any_out *)to = v;      // at any alignment
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < n) ((gu16_out *)to)[i] = uint16_t(v[i / 2] >> (16 * (i % 2)));
}

template <int FM, int FN>
__device__ __forceinline__ void pair_all(f32x4 (&acc)[FM][FN]) {
#pragma unroll
    for (int f = 0; f < FM; f += 2)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a = acc[f][j][i], b = acc[f + 1][j][i];
                pair_up(a, b);
                acc[f][j][i] = a;
                acc[f + 1][j][i] = b;
            }
}

// What takes the scale of a row's coefficients off again.
template <int DT, class Args>
__device__ __forceinline__ float unscale(const Args &p, uint32_t row) {
    if constexpr (DT != ROG_DTYPE_F16) return 1.0f;
    else return 1.0f / power_for(most_of(p.g_logp[row], p.g_entropy ? p.g_entropy[row] : 0.0f, p.inv_t));
}

// A tile's sums of a segment to its partial sums, or added to the running ones, or to the end.
template <int DT, int FM, int FN, int WN>
__device__ __forceinline__ void put_states(uint32_t s, uint32_t d0, uint32_t n0, uint32_t rows, f32x4 (&acc)[FM][FN]) {
    const BackArgs &p = fresh_args<BackArgs>();
    const bool running = p.part_seg == 0, first = running && p.first && s == 0, last = running && p.last && s + 1 == p.segs;
    pair_all(acc);
    const uint32_t t = fresh_thread(), l = t % 64, m0 = t / 64 / WN * (FM * 16), w0 = t / 64 % WN * (FN * 16);
    float *part = p.part + uint64_t(s) * p.part_seg;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t n = n0 + w0 + 16 * j + l % 16;
        if (n >= rows) continue;
        const uint32_t row = p.index[n];
        const float inv = last ? unscale<DT>(p, row) : 1.0f;
        uint8_t *out = static_cast<uint8_t *>(p.d_hidden) + uint64_t(row) * uint64_t(p.d_stride);
#pragma unroll
        for (int f = 0; f < FM / 2; ++f) {
            const uint32_t d = d0 + m0 + 32 * f + 8 * eight_of(l / 16);
            if (d >= p.dim) continue;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = acc[2 * f + i / 4][j][i % 4];
            gf32x4_out *at = (gf32x4_out *)(part + uint64_t(n) * p.dim_pad + d);
            if (running && !first) {
                const f32x4 lo = at[0], hi = at[1];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (i < 4 ? lo[i % 4] : hi[i % 4]) + x[i];
            }
            if (last) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= inv;
                put8<DT>(out + d * 2, x, p.dim - d);
            } else {
                at[0] = f32x4{x[0], x[1], x[2], x[3]};
                at[1] = f32x4{x[4], x[5], x[6], x[7]};
            }
        }
    }
}

// The rows of part `split`: whole lines of 64, the same number but for the last.
struct RowPart {
    uint32_t first, rows;
};
__device__ __forceinline__ RowPart part_of(uint32_t split, uint32_t parts, uint32_t rows) {
    if (parts == 1) return RowPart{0, rows};
    const uint32_t each = ((rows + parts - 1) / parts + 63) / 64 * 64, first = split * each;
    return RowPart{first < rows ? first : 0, first >= rows ? 0 : rows - first < each ? rows - first : each};
}
__device__ __forceinline__ uint32_t parts_of(const BackArgs &p) { return p.splits > 1 ? uniform(*p.parts) : 1; }

// A tile's sums for columns v0 on and elements d0 on of shard r, of part `split` of the rows.
template <int DT, int FM, int FN, int WN>
__device__ __forceinline__ void put_weights(uint32_t split, uint32_t parts, uint32_t r, uint32_t v0, uint32_t d0, uint32_t width, f32x4 (&acc)[FM][FN]) {
    const BackArgs &p = fresh_args<BackArgs>();
    pair_all(acc);
    const uint32_t t = fresh_thread(), l = t % 64, m0 = t / 64 / WN * (FM * 16), w0 = t / 64 % WN * (FN * 16);
    const float inv = DT == ROG_DTYPE_F16 ? 1.0f / *p.g_scale : 1.0f;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t v = v0 + w0 + 16 * j + l % 16;
        if (v >= width) continue;
        uint8_t *out = static_cast<uint8_t *>(p.dw[r]) + uint64_t(v) * uint64_t(p.dw_stride[r]);
#pragma unroll
        for (int f = 0; f < FM / 2; ++f) {
            const uint32_t d = d0 + m0 + 32 * f + 8 * eight_of(l / 16);
            if (d >= p.dim) continue;
            if (parts > 1) {
                const uint32_t column = (p.sh.tile0[r] - p.tile_begin) * kGradTile + v;      // of the piece
                gf32x4_out *at = (gf32x4_out *)(p.dw_part + split * p.dw_part_split + uint64_t(column) * p.dim_pad + d);
                at[0] = acc[2 * f][j];
                at[1] = acc[2 * f + 1][j];
                continue;
            }
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = acc[2 * f + i / 4][j][i % 4] * inv;
            put8<DT>(out + d * 2, x, p.dim - d);
        }
    }
}

constexpr int kBM = 256;   // elements of the states and weights of a tile

template <int DT, int BN, int WM, int WN, bool DIRECT>
__device__ __forceinline__ void back_states(const BackArgs &p, uint32_t id, uint32_t rows, const TileMemory &memory) {
    constexpr int THREADS = 64 * WM * WN, FM = kBM / WM / 16, FN = BN / WN / 16;
    typedef ColSteps<kBM, THREADS, DIRECT> A;
    typedef RowSteps<false, BN, THREADS, true, 2> B;
    const uint32_t tn = (rows + BN - 1) / BN, each = p.dim_tiles * tn;
    const bool running = p.part_seg == 0;              // one workgroup takes all segments of the piece, in their order
    const uint32_t in = id % each, d0 = in % p.dim_tiles * kBM, n0 = in / p.dim_tiles * BN;
    const uint32_t begin = running ? 0 : id / each, end = running ? p.segs : begin + 1;
    for (uint32_t s = begin; s < end; ++s) {
        const uint32_t seg = p.seg_begin + s;
        uint32_t r = 0;
        while (seg >= p.seg0[r + 1]) ++r;
        const WeightShard sh = p.sh.s[r];
        const uint32_t tile = (seg - p.seg0[r]) * p.seg_tiles, v0 = tile * kGradTile;
        const uint32_t cols = sh.width - v0 < p.seg_tiles * kGradTile ? sh.width - v0 : p.seg_tiles * kGradTile;
        const uint64_t g_col = uint64_t(p.sh.tile0[r] + tile - p.tile_begin) * kGradTile * 2;
        A a(static_cast<const uint8_t *>(sh.w) + uint64_t(v0) * uint64_t(sh.stride) + d0 * 2, sh.stride, cols, p.dim - d0);
        B b(static_cast<const uint8_t *>(p.g) + uint64_t(n0) * uint64_t(p.g_stride) + g_col, p.g_stride, rows - n0,
                  p.seg_tiles * kGradTile * 2);
        f32x4 acc[FM][FN] = {};
        const uint32_t wave = fresh_thread() / 64;
        if (s != begin) __syncthreads();               // the last slab's readers
        Tile<DT, FM, FN, A, B>().template run<true>(a, b, (cols + 31) / 32, false, wave / WN * (FM * 16), wave % WN * (FN * 16), memory, acc);

        put_states<DT, FM, FN, WN>(s, d0, n0, rows, acc);
    }
}

template <int DT, int BN, int WM, int WN>
__device__ __forceinline__ void back_weights(const BackArgs &p, uint32_t id, uint32_t parts, uint32_t rows, const TileMemory &memory) {
    constexpr int THREADS = 64 * WM * WN, FM = kBM / WM / 16, FN = BN / WN / 16;
    typedef ColSteps<kBM, THREADS, true> A;
    typedef ColSteps<BN, THREADS, true> B;
    static_assert(BN == int(kGradTile), "a tile of the piece");
    const uint32_t all = p.dim_tiles * p.tiles, split = id / all;
    const RowPart part = part_of(split, parts, rows);
    const TileAt at = tile_at(id % all, p.dim_tiles, p.tiles);
    const uint32_t tile = p.tile_begin + at.n, d0 = at.m * kBM;
    const uint32_t r = shard_of_tile(p.sh, tile), v0 = (tile - p.sh.tile0[r]) * kGradTile, width = p.sh.s[r].width;
    A a(static_cast<const uint8_t *>(p.a.x) + uint64_t(part.first) * uint64_t(p.a.stride) + d0 * 2, p.a.stride, part.rows,
        uint32_t(p.a.stride) / 2 - d0);
    B b(static_cast<const uint8_t *>(p.g_all) + uint64_t(part.first) * uint64_t(p.g_stride) + uint64_t(at.n) * BN * 2, p.g_stride, part.rows, BN);
    const uint32_t wave = fresh_thread() / 64;
    f32x4 acc[FM][FN] = {};
    Tile<DT, FM, FN, A, B>().run(a, b, (part.rows + 31) / 32, false, wave / WN * (FM * 16), wave % WN * (FN * 16), memory, acc);

    put_weights<DT, FM, FN, WN>(split, parts, r, v0, d0, width, acc);
}

// Both products of a piece, in tiles of 256 x 256.  The longer chains first: the states' run over a segment's (or, running, the piece's)
// columns, the weights' over the rows (8192 x 32000 x 320: 911 us so, 1033 with the states' always first).  Bound by the
// matrix units (4096 x 32768 of 4096 bf16, 3584 rows scored: 1.55 ms, 1240 TFLOP/s): ds_read_b64_tr_b16 brings half the
// bytes of ds_read_b128 per instruction, so an operand with K along its rows costs twice the reads of one with rows
// along K, and the weights' product has two.
template <int DT, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN) void rog_linear_back_kernel(BackArgs p) {
    ROG_TILE_MEMORY(kStages, kBM * kStepBytes, BN * kStepBytes);
    const uint32_t rows = uniform(*p.a.count), states = (p.part_seg ? p.segs : 1) * p.dim_tiles * ((rows + BN - 1) / BN);
    const uint32_t parts = parts_of(p), weights = p.dim_tiles * p.tiles * parts, before = rows / parts > (p.part_seg ? p.seg_tiles : p.tiles) * kGradTile ? weights : 0;
    const uint32_t id = blockIdx.x;
    if (id >= before && id - before < states) back_states<DT, BN, WM, WN, DIRECT>(p, id - before, rows, memory);
    else if (id < states + weights) back_weights<DT, BN, WM, WN>(p, before ? id : id - states, parts, rows, memory);
}

// FM x FN fragments of a wave over two steps of K, brought together.
template <int DT, int FM, int FN, class C>
struct BothSteps {
    static __device__ __forceinline__ void run(C &a, C &b, uint32_t m0, uint32_t n0, const TileMemory &mem, f32x4 (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)   // as in Tile
        const typename C::template Reader<0> ra(m0), rb(n0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a.stage(mem.a[i]);
            b.stage(mem.b[i]);
        }
        arrive<0>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            vec16 fa[FM], fb[FN];
#pragma unroll
            for (int f = 0; f < FM; ++f) fa[f] = ra.get(mem.a[i], f);
#pragma unroll
            for (int f = 0; f < FN; ++f) fb[f] = rb.get(mem.b[i], f);
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[f][j] = Mat<DT>::mma(fa[f], fb[j], acc[f][j]);
        }
#else
        (void)a, (void)b, (void)m0, (void)n0, (void)mem, (void)acc;
#endif
    }
};

// The same for few rows or little work.  d_hidden: 64 elements of a segment for 64 rows, up to seven lines of each
// operand's rows in flight and two multiplied at a time: a chain over a segment cannot be cut further, so a workgroup
// has to bring its share of the weights fast (33 x 32003 x 1024: the call 69.3, 58.3 and 64.1 us with 1, 2 and 4 lines
// at a time; the kernel 23 us for the 66 MB of weights, 128 workgroups with a CU each).
constexpr int kFewElements = 64, kFewSide = 128, kFewThreads = 256, kFewStages = 8, kFewGroup = 2;
template <int DT, bool DIRECT>
__global__ __launch_bounds__(kFewThreads) void rog_linear_few_states_kernel(BackArgs p) {
    typedef ColLines<kFewThreads, DIRECT> A;
    typedef RowLines<false, 64, kFewThreads, true, 2> B;
    ROG_TILE_MEMORY(kFewStages, A::kBytes, B::kBytes);
    const uint32_t rows = uniform(*p.a.count), dim_tiles = (p.dim + kFewElements - 1) / kFewElements, each = dim_tiles * p.row_tiles;
    const uint32_t s = blockIdx.x / each, d0 = blockIdx.x % dim_tiles * kFewElements, n0 = blockIdx.x % each / dim_tiles * 64;
    const uint32_t seg = p.seg_begin + s;
    if (n0 >= rows) return;
    uint32_t r = 0;
    while (seg >= p.seg0[r + 1]) ++r;
    const WeightShard sh = p.sh.s[r];
    const uint32_t tile = (seg - p.seg0[r]) * p.seg_tiles, v0 = tile * kGradTile;
    const uint32_t cols = sh.width - v0 < p.seg_tiles * kGradTile ? sh.width - v0 : p.seg_tiles * kGradTile;
    A a(static_cast<const uint8_t *>(sh.w) + uint64_t(v0) * uint64_t(sh.stride) + d0 * 2, sh.stride, cols, p.dim - d0);
    B b(static_cast<const uint8_t *>(p.g) + uint64_t(n0) * uint64_t(p.g_stride) + uint64_t(p.sh.tile0[r] + tile - p.tile_begin) * kGradTile * 2,
        p.g_stride, rows - n0, (cols + 63) / 64 * 128);
    const uint32_t wave = threadIdx.x / 64;
    f32x4 acc[2][2] = {};
    Stream<DT, 2, 2, kFewStages, kFewGroup, A, B>::run(a, b, (cols + 63) / 64, wave / 2 * 32, wave % 2 * 32, memory, acc);
    put_states<DT, 2, 2, 2>(s, d0, n0, rows, acc);
}

// d_weight: 128 columns x 128 elements; of up to 64 rows both steps of K at once.  Bound by the gradient's bytes (33 x 32003 x 1024:
// 17.7 us for 66 MB, 3.7 TB/s; a workgroup is one load, one product and one write).
template <int DT, bool FEW>
__global__ __launch_bounds__(kFewThreads) void rog_linear_few_weights_kernel(BackArgs p) {
    typedef ColSteps<kFewSide, kFewThreads, true> C;
    ROG_TILE_MEMORY(FEW ? 2 : kStages, C::kBytes, C::kBytes);
    const uint32_t rows = uniform(*p.a.count), sides = (p.dim + kFewSide - 1) / kFewSide;
    const uint32_t all = sides * p.tiles * 2, split = FEW ? 0 : blockIdx.x / all, id = blockIdx.x - split * all;
    const uint32_t parts = FEW ? 1 : parts_of(p);
    if (split >= parts) return;
    const RowPart of = part_of(split, parts, rows);
    const uint32_t part = id / sides, d0 = id % sides * kFewSide;       // of the piece's parts of 128 columns
    const uint32_t tile = p.tile_begin + part / 2, r = shard_of_tile(p.sh, tile);
    const uint32_t v0 = (tile - p.sh.tile0[r]) * kGradTile + part % 2 * kFewSide, width = p.sh.s[r].width;
    if (v0 >= width) return;
    C a(static_cast<const uint8_t *>(p.a.x) + uint64_t(of.first) * uint64_t(p.a.stride) + d0 * 2, p.a.stride, of.rows,
        uint32_t(p.a.stride) / 2 - d0);
    C b(static_cast<const uint8_t *>(p.g_all) + uint64_t(of.first) * uint64_t(p.g_stride) + uint64_t(part) * kFewSide * 2, p.g_stride, of.rows,
        kFewSide);
    const uint32_t wave = threadIdx.x / 64, m0 = wave / 2 * 64, w0 = wave % 2 * 64;
    f32x4 acc[4][4] = {};
    if constexpr (FEW) BothSteps<DT, 4, 4, C>::run(a, b, m0, w0, memory, acc);
    else Tile<DT, 4, 4, C, C>().run(a, b, (of.rows + 31) / 32, false, m0, w0, memory, acc);
    put_weights<DT, 4, 4, 2>(split, parts, r, v0, d0, width, acc);
}

// Adds the segments' partial sums of a row in their order, eight of them in flight (893 x 1600, 13 segments: 19.7 us
// for 75 MB; 33 x 1024, 8 segments: 4.7).
template <int DT>
__global__ __launch_bounds__(256) void rog_linear_back_join_kernel(BackJoinArgs p) {
    const uint32_t rows = *p.count, vecs = p.dim_pad / 8;   // a thread has eight elements of a row
    const uint64_t id = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    const uint32_t n = uint32_t(id / vecs), d = uint32_t(id % vecs) * 8;
    if (n >= rows || d >= p.dim) return;
    typedef const __attribute__((address_space(1))) f32x4 gf32x4;
    const uint64_t at = uint64_t(n) * p.dim_pad + d;
    float x[8];
    if (!p.first) {
        const f32x4 lo = ((gf32x4 *)(p.running + at))[0], hi = ((gf32x4 *)(p.running + at))[1];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < 4 ? lo[i % 4] : hi[i % 4];
    }
    constexpr uint32_t DEEP = 8;       // segments' loads at a time
    for (uint32_t s = 0; s < p.segs; s += DEEP) {
        f32x4 v[DEEP][2];
#pragma unroll
        for (uint32_t u = 0; u < DEEP; ++u) {
            const float *from = p.part + (s + u < p.segs ? s + u : s) * p.part_seg + at;
            v[u][0] = ((gf32x4 *)from)[0];
            v[u][1] = ((gf32x4 *)from)[1];
        }
#pragma unroll
        for (uint32_t u = 0; u < DEEP; ++u)
            if (s + u < p.segs)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = p.first && s + u == 0 ? v[u][i / 4][i % 4] : x[i] + v[u][i / 4][i % 4];
    }
    if (!p.last) {
        ((gf32x4_out *)(p.running + at))[0] = f32x4{x[0], x[1], x[2], x[3]};
        ((gf32x4_out *)(p.running + at))[1] = f32x4{x[4], x[5], x[6], x[7]};
        return;
    }
    const uint32_t row = p.index[n];
    const float inv = unscale<DT>(p, row);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    put8<DT>(static_cast<uint8_t *>(p.d_hidden) + uint64_t(row) * uint64_t(p.d_stride) + d * 2, x, p.dim - d);
}

// Adds the parts' sums of a column of the piece in their order; a thread has eight elements.
template <int DT>
__global__ __launch_bounds__(256) void rog_linear_weights_join_kernel(BackArgs p) {
    const uint32_t vecs = p.dim_pad / 8, parts = parts_of(p);
    if (parts == 1) return;            // the sums are where they belong
    const uint64_t id = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    const uint32_t column = uint32_t(id / vecs), d = uint32_t(id % vecs) * 8;
    if (column >= p.tiles * kGradTile || d >= p.dim) return;
    const uint32_t tile = p.tile_begin + column / kGradTile, r = shard_of_tile(p.sh, tile);
    const uint32_t v = (tile - p.sh.tile0[r]) * kGradTile + column % kGradTile;
    if (v >= p.sh.s[r].width) return;
    typedef const __attribute__((address_space(1))) f32x4 gf32x4;
    const float *from = p.dw_part + uint64_t(column) * p.dim_pad + d;
    f32x4 lo = ((gf32x4 *)from)[0], hi = ((gf32x4 *)from)[1];
    for (uint32_t s = 1; s < parts; ++s) {
        from += p.dw_part_split;
        lo = lo + ((gf32x4 *)from)[0];
        hi = hi + ((gf32x4 *)from)[1];
    }
    const float inv = DT == ROG_DTYPE_F16 ? 1.0f / *p.g_scale : 1.0f;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (i < 4 ? lo[i % 4] : hi[i % 4]) * inv;
    put8<DT>(static_cast<uint8_t *>(p.dw[r]) + uint64_t(v) * uint64_t(p.dw_stride[r]) + d * 2, x, p.dim - d);
}

template <int DT>
hipError_t launch_back(const GradPlan &p, const BackArgs &a, const PieceGrid &grid, hipStream_t s) {
    if (p.form == kFormWide)
        return p.direct_back ? launch(rog_linear_back_kernel<DT, 256, 2, 4, true>, grid.states + grid.weights, 512, a, s)
                             : launch(rog_linear_back_kernel<DT, 256, 2, 4, false>, grid.states + grid.weights, 512, a, s);
    const hipError_t e = p.direct_back ? launch(rog_linear_few_states_kernel<DT, true>, grid.states, kFewThreads, a, s)
                                       : launch(rog_linear_few_states_kernel<DT, false>, grid.states, kFewThreads, a, s);
    if (e != hipSuccess) return e;
    return p.form == kFormMid ? launch(rog_linear_few_weights_kernel<DT, false>, grid.weights, kFewThreads, a, s)
                              : launch(rog_linear_few_weights_kernel<DT, true>, grid.weights, kFewThreads, a, s);
}

}  // namespace
}  // namespace rog

extern "C" {

ROG_API rog_status rog_linear_logprob_grad(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim,
                                           const rog_weight_shard *shards, int W, rog_dtype dtype, float temperature,
                                           const int64_t *tokens, const float *lse, const float *entropy, const float *g_logp,
                                           const float *g_entropy, void *d_hidden, int64_t d_hidden_stride,
                                           const rog_grad_shard *d_weights, void *workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    using namespace rog;
    GradPlan p;
    const rog_status st = plan_linear_grad(hidden, hidden_stride, rows, dim, shards, W, dtype, temperature, tokens, lse, entropy, g_logp,
                                           g_entropy, d_hidden, d_hidden_stride, d_weights, workspace, workspace_bytes, true, &p);
    if (st != ROG_OK || rows == 0) return st;
    hipError_t e = launch_pack(p.pack, stream);
    for (uint32_t i = 0; i < p.pieces && e == hipSuccess; ++i) {
        const PieceGrid grid = lay_piece(&p, i);
        e = launch_coefficients(p, p.coef, grid.coefficients, stream);
        if (e == hipSuccess) e = dtype == ROG_DTYPE_BF16 ? launch_back<ROG_DTYPE_BF16>(p, p.back, grid, stream)
                                                         : launch_back<ROG_DTYPE_F16>(p, p.back, grid, stream);
        if (e == hipSuccess && grid.join)
            e = dtype == ROG_DTYPE_BF16 ? launch(rog_linear_back_join_kernel<ROG_DTYPE_BF16>, grid.join, 256, p.join, stream)
                                        : launch(rog_linear_back_join_kernel<ROG_DTYPE_F16>, grid.join, 256, p.join, stream);
        if (e == hipSuccess && grid.weights_join)
            e = dtype == ROG_DTYPE_BF16 ? launch(rog_linear_weights_join_kernel<ROG_DTYPE_BF16>, grid.weights_join, 256, p.back, stream)
                                        : launch(rog_linear_weights_join_kernel<ROG_DTYPE_F16>, grid.weights_join, 256, p.back, stream);
    }
    return launched(e);
}

}  // extern "C"
