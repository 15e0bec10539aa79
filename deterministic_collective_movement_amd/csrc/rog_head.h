// rog_head.h -- kernel arguments and launch plans of the vocabulary-side
// operators (token log probabilities, their gradient, the policy loss), shared
// by the host planner (rog_head_plan.cpp) and the HIP kernels.  Internal to
// librog.so; the public interface is include/rog.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rog_internal.h"

namespace rog {

// How a row of logits is cut.  A block is 2048 consecutive columns of one shard
// (a shard's last one may be shorter), 32 columns per lane of one wave; blocks
// are numbered through the shards in rank order.  A unit is four blocks that
// one wave takes one after the other: a row of at most four blocks is one
// unit; a longer row is cut into chunks of sixteen blocks, and unit w of a
// chunk is every fourth of its blocks from the w-th on (so that the waves of a
// workgroup share the row evenly).  The partial states are joined in one
// order, whatever the launch form: the blocks of a unit one after the other in
// each lane, then the unit's lanes; then units 64 apart one after the other,
// and the 64 sums last.  So a row's bits depend on its values, its shards'
// widths and the temperature alone, not on how many rows a call has or which
// workgroups computed them.
constexpr uint32_t kHeadBlock = 2048;      // columns of a block
constexpr uint32_t kUnitBlocks = 4;
constexpr uint32_t kChunkUnits = 4;
constexpr uint32_t kChunkBlocks = kUnitBlocks * kChunkUnits;
constexpr int kHeadThreads = 256;          // a workgroup: four waves, one per unit of a chunk
constexpr uint32_t kGradPieceBytes = 2048; // the gradient's piece of a row: two 16-byte vectors per lane of one wave
// The grid of a launch of `groups` workgroups (below 2^31): a dispatch counts the
// work-items of each dimension in 32 bits, so more than 2^22 go over two.  The
// kernels number a workgroup by head_group() (a constant row length: the grid's
// own would be one more line of kernel arguments), and those past the end leave
// at once.
constexpr uint32_t kGridRowLog = 22;
inline dim3 head_grid(uint32_t groups) {
    const uint32_t most = 1u << kGridRowLog;
    return groups <= most ? dim3(groups) : dim3(most, (groups + most - 1) / most);
}
constexpr int kMaxTopK = 32;
constexpr uint32_t kTopSlots = 8;          // entries per lane and wave in the top-k table

// Tunables, measured on MI355X; a variant build may override one with -D.
// When a row of `units` units is split over workgroups: a workgroup per row
// takes about 4 us + 0.8 us per unit up to 256 rows (a wave takes its blocks one
// after the other), a split launch about 5.5 us + 2.9 ns per workgroup, with
// alternatives 8.5 us + 3.9 ns; so for rows + kSplitCost / units <= kSplitRows.
// Measured in us, split against not: 131072 bf16 columns (16 units), 64 rows
// 8.5 / 17.0, 192 14.4 / 17.5, 224 16.1 / 17.5, 256 17.2 / 17.8; 50257 (7), 64
// 5.8 / 9.1, 176 9.8 / 10.0, 208 10.6 / 10.1; 32000 binary32 (4), 80 6.1 / 6.9,
// 112 7.0 / 7.1, 144 8.2 / 7.2.  With 8 alternatives: 131072, 192 20.2 / 20.8,
// 224 22.8 / 21.3; 50257, 64 9.6 / 12, 144 13.8 / 13.1; 32000 binary32, 64
// 8.6 / 9.2, 96 9.8 / 8.9.
#ifndef ROG_SPLIT_ROWS
#define ROG_SPLIT_ROWS 270
#endif
#ifndef ROG_SPLIT_ROWS_TOP
#define ROG_SPLIT_ROWS_TOP 205
#endif
constexpr uint32_t kSplitRows = ROG_SPLIT_ROWS, kSplitRowsTop = ROG_SPLIT_ROWS_TOP, kSplitCost = 600;
// Logits' bytes from which their loads are streamed past the caches: 4096 x
// 131072 bf16 163-170 us streamed against 186 cached, its gradient 330 against
// 349, 8627 x 8192 26.2 against 29.6; below, the Infinity Cache may hold them
// (1021 x 50257 binary16 20.4 cached against 21.0, its gradient after it 30.0
// against 34.8).
#ifndef ROG_HEAD_NT_MIN_BYTES
#define ROG_HEAD_NT_MIN_BYTES (128ull << 20)
#endif
#ifndef ROG_WAVE_ROWS
#define ROG_WAVE_ROWS 4
#endif
constexpr uint32_t kWaveRows = ROG_WAVE_ROWS;   // rows (waves) of a workgroup of the one-wave-per-row form
constexpr uint32_t kMaxVocab = 1u << 31;   // columns of a row: below this

// The front of a workspace: arrival counters, zero between calls, each in a
// 128-byte line of its own (counters that share a line are counted one after
// the other: 64 rows of 131072 columns took 12.2 us with their counters packed,
// 8.9 apart).  A split launch counts row r's workgroups in counter r, the policy
// loss its own in counter 0.  Partial states follow.
constexpr uint32_t kHeadCounters = 1024;
constexpr uint32_t kCounterStride = 128 / sizeof(uint32_t);
constexpr size_t kHeadCounterBytes = size_t(kHeadCounters) * kCounterStride * sizeof(uint32_t);

// Floats of a split row's partial states: m, s, t of each unit (padded to 4),
// then 64 lanes' maxima for each of four entries per unit.
constexpr uint32_t kUnitFloats = 4 + 4 * 64;

struct Shard {
    const void *x;                     // element (0, 0)
    int64_t stride;                    // bytes from a row to the next
    uint32_t width;                    // columns
    uint32_t col0;                     // the shard's first column in the row
};
// The shards of a row, cut into blocks.
struct HeadShards {
    uint32_t W;
    uint32_t blocks;                   // of a row
    uint32_t even;                     // blocks of every shard where they have as many each, else 0
    Divider even_div;                  // divides by it
    Shard s[kMaxPeers];
    uint32_t block0[kMaxPeers + 1];    // the shard's first block; [W]: all blocks
};

// What every workgroup reads first stands together at the front (the first
// read of each 64-byte line of the arguments takes more than half a
// microsecond), up to the first shard.
struct LogprobArgs {
    const int64_t *tokens;             // NULL: no token, every row scored
    uint32_t rows;
    uint32_t chunks, units;            // units that have blocks
    uint32_t slot_shift;               // log2 of a wave's blocks that one entry of the top-k table covers
    uint32_t top_k;
    uint32_t vocab;
    float scale;                       // log2(e) / temperature
    float inv_t;                       // 1 / temperature
    float bound;                       // |x| that leaves the scaled range (no binary16 does)
    float inv_t_rest;                  // 1 / temperature - inv_t
    float *logp, *entropy, *lse, *top_logp;
    int64_t *top_ids;
    uint32_t *counters;                // split: one per row
    float *part;                       // split: per row, the units' states and their lanes' maxima
    HeadShards sh;
};

struct LogprobGradArgs {
    const int64_t *tokens;
    const float *lse, *entropy, *g_logp, *g_entropy;
    float inv_t;                       // 1 / temperature
    float inv_t_rest;                  // and what its rounding left off
    uint32_t vocab;
    uint32_t groups;                   // pieces of all rows
    Divider pieces_div;                // divides by sh.blocks, the pieces of a row
    HeadShards sh;                     // its blocks are pieces here
    void *g[kMaxPeers];
    int64_t g_stride[kMaxPeers];       // bytes
};

struct PolicyArgs {
    const float *logp, *old_logp, *adv, *weight, *ref, *entropy;
    float *stats, *g_logp, *g_entropy;
    uint32_t *counter;
    double *part;                      // [groups][4]
    uint64_t n;
    float lo, hi;                      // log(1 - clip_low), log(1 + clip_high)
    float ratio_lo, ratio_hi;          // e^lo, e^hi
    float kl_coef, entropy_coef, grad_scale, w_all;
    uint32_t groups;
    uint32_t tiles;                    // tiles per workgroup
};

static_assert(sizeof(LogprobArgs) <= 4096 && sizeof(LogprobGradArgs) <= 4096, "kernel arguments stay below 4 KiB");

struct LogprobPlan {
    rog_head_plan_info info;
    LogprobArgs args;
    rog_dtype dtype;
    bool nt_loads;                     // logits are streamed past the caches
};
struct LogprobGradPlan {
    uint32_t grid;
    LogprobGradArgs args;
    rog_dtype dtype;
    bool nt_loads;
};
struct PolicyPlan {
    PolicyArgs args;
};

// The policy loss: tiles of 1024 tokens, four per thread of a workgroup; up to
// kPolicyGroups workgroups, each with a run of consecutive tiles.
constexpr uint32_t kPolicyTile = 1024;
constexpr uint32_t kPolicyGroups = 512;

// Validate and plan (no HIP calls).
rog_status plan_logprob(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype, float temperature,
                        const int64_t *tokens, int top_k, const rog_logprob_out *out, void *workspace,
                        size_t workspace_bytes, rog_logprob_form form, bool check_workspace, LogprobPlan *p);
rog_status plan_logprob_grad(const rog_logit_shard *shards, const rog_grad_shard *grads, int W, size_t rows,
                             rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse,
                             const float *entropy, const float *g_logp, const float *g_entropy,
                             LogprobGradPlan *p);
rog_status plan_policy(const rog_policy_in *in, size_t n, const rog_policy_params *params,
                       const rog_policy_out *out, void *workspace, size_t workspace_bytes, PolicyPlan *p);

}  // namespace rog
