/*
 * rog.h -- rank-ordered gather (rog) and rank-ordered sum for MI355X (gfx950,
 * CDNA4).
 *
 * C ABI of librog.so.  Plain C types, device pointers and sizes; no PyTorch
 * types.  Every entry point below is implemented by hand-written HIP kernels in
 * deterministic_collective_movement_amd/csrc/.
 *
 * The operation is the copy at the heart of a deterministic all-gather
 * (RL-Align/RL-Kernel PR #491, "perf(cuda): vectorize the deterministic
 * all-gather copy and right-size its single-block path", section "What", the
 * copy_rank_ordered bullet): W payloads of S bytes are concatenated in rank
 * order, so that
 *
 *     out[r*S + i] = srcs[r][i]     for 0 <= r < W, 0 <= i < S,
 *
 * byte-identical to a plain concatenation for every alignment and size.  On one
 * GPU the W peers' payloads are W caller-owned device buffers.  Beside it,
 * rog_reduce computes the rank-ordered sum at the heart of the same pages'
 * deterministic all-reduce and reduce-scatter (declared and defined below).
 *
 * Common rules for every entry point:
 *  - Pointers to data (srcs[r], out, the descriptors' buffers) are device
 *    pointers readable/writable by kernels on the current HIP device.  They are
 *    not checked for residency; the Python binding checks tensor devices.
 *  - Host arrays (the srcs array, the descriptor array) are read only during
 *    the call; their contents are copied into the kernel arguments.
 *  - The caller owns every buffer; buffers must stay valid until the work
 *    enqueued on `stream` has completed.
 *  - All argument errors are returned before anything is enqueued: on error no
 *    byte of any output is written and no HIP call has been made.
 *  - Success means the work has been enqueued on `stream` (asynchronous), as
 *    exactly one kernel launch; nothing else is enqueued, so calls can be
 *    captured into a HIP graph.
 *  - The library allocates no device or host memory, keeps no state except a
 *    thread-local copy of the last HIP error, and may be called from any thread.
 *  - Bytes outside the output range (out, W*S bytes for a gather; count
 *    elements for a sum) are never written.  Source bytes are never written,
 *    except by an in-place call where out is itself a source.  Every read lies
 *    inside a source range (S bytes for a gather, count elements for a sum) or,
 *    in the forms flagged ROG_PLAN_SHIFTED_LOADS, inside an aligned 16-byte
 *    granule that holds bytes of one (so within that range's own pages); the
 *    bytes read beyond a range are never used.
 */
#ifndef ROG_H
#define ROG_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ROG_API __attribute__((visibility("default")))

typedef enum {
    ROG_OK = 0,
    ROG_ERR_INVALID_ARGUMENT = 1, /* null pointer, W out of range, n < 0, bad path  */
    ROG_ERR_OVERLAP = 2,          /* a source range partially overlaps the output   */
    ROG_ERR_TOO_LARGE = 3,        /* size overflow or a limit below exceeded        */
    ROG_ERR_LAUNCH = 4            /* the kernel launch failed; see rog_last_hip_error */
} rog_status;

typedef enum {
    ROG_PATH_AUTO = 0,       /* single-WG iff W*S <= rog_single_wg_max_bytes()  */
    ROG_PATH_SINGLE_WG = 1,  /* one workgroup of up to 1024 threads does it all */
    ROG_PATH_MULTI_WG = 2    /* a grid of small workgroups sized from the work      */
} rog_path;

typedef enum {
    ROG_KERNEL_NONE = 0,     /* nothing to copy (S == 0): nothing is launched       */
    ROG_KERNEL_FLAT = 1,     /* a single loop over every payload's 16-byte vectors  */
    ROG_KERNEL_PEER = 2,     /* per payload: byte head, 16-byte body (aligned
                                stores, loads at any alignment), byte tail          */
    ROG_KERNEL_REDUCE = 3    /* rank-ordered sum: element head, 16-byte body of
                                aligned stores (loads at any element alignment),
                                element tail                                         */
} rog_kernel;

/* Element types of the rank-ordered sum. */
typedef enum {
    ROG_DTYPE_F32 = 0,       /* IEEE binary32, 4 bytes                               */
    ROG_DTYPE_BF16 = 1,      /* bfloat16 (top 16 bits of a binary32), 2 bytes       */
    ROG_DTYPE_F16 = 2        /* IEEE binary16, 2 bytes                               */
} rog_dtype;

/* One tensor of a batch: W source pointers, its output, its per-rank bytes. */
typedef struct {
    const void *const *srcs;   /* W device pointers (host array)                 */
    void *out;                 /* device pointer to W * bytes_per_rank bytes     */
    size_t bytes_per_rank;     /* S of this tensor; 0 is allowed (nothing copied) */
} rog_gather_desc;

/* The launch a call would make (rog_plan), for tests and inspection. */
typedef struct {
    int32_t path;              /* resolved rog_path: SINGLE_WG or MULTI_WG (AUTO never) */
    int32_t kernel;            /* rog_kernel                                            */
    uint32_t grid;             /* workgroups launched (0 when kernel == NONE)           */
    uint32_t block;            /* threads per workgroup                                 */
    uint64_t vec_ok_mask;      /* PEER kernel: bit r set iff srcs[r] and out + r*S are
                                  both 16-byte aligned (where the pages' fallback
                                  copies vectors); informational, every payload
                                  gets a 16-byte body whatever its alignment       */
    uint64_t units;            /* FLAT: 16-byte vectors W*S/16; PEER: bytes W*S;
                                  REDUCE: elements per payload                        */
    uint32_t peer_magic;       /* FLAT: floor(v / (S/16)) = (t + ((v - t) >> peer_sh1))  */
    uint32_t peer_sh1;         /*       >> peer_sh2 with t = mulhi32(v, peer_magic),     */
    uint32_t peer_sh2;         /*       exact for every 32-bit v                         */
    uint32_t flags;            /* ROG_PLAN_* bits                                       */
} rog_plan_info;

/* rog_plan_info.flags: the kernel's 16-byte loads are non-temporal (streamed
 * past the caches); set when the W*S source bytes are too many for the 256 MB
 * Infinity Cache to serve repeated calls well: from 128 MiB, for gathers and
 * sums, single or batched.  16-byte stores are always non-temporal; a
 * gather's are also written through the L2 caches at device scope.  Affects
 * speed only. */
#define ROG_PLAN_NT_LOADS 1u
/* rog_plan_info.flags: the multi-workgroup PEER or REDUCE kernel reads at least
 * one source body as aligned 16-byte granules, each lane taking the granule
 * after its own from the next lane.  Only with ROG_PLAN_NT_LOADS.  PEER: set
 * when a payload's body (from the first 256-byte boundary of its output) is
 * not empty and its source sits an odd or 2-mod-4 number of bytes past a
 * 16-byte granule there.  REDUCE: set with ROG_PLAN_NT_LOADS, for every
 * source.  Affects speed only; the bytes are the same. */
#define ROG_PLAN_SHIFTED_LOADS 2u

/*
 * rog_gather -- out[r*S + i] = srcs[r][i] for r < W, i < S, enqueued on `stream`.
 *
 * srcs            host array of W device pointers (payload r = rank r).
 * W               number of payloads, 1 <= W <= rog_max_peers().
 * bytes_per_rank  S, the byte size of every payload (one S for all, as in an
 *                 all-gather; PR #491 "What": one byte count per rank).
 * out             device pointer to W*S writable bytes.
 * stream          HIP stream (0 = null stream) of the current device.
 *
 * Path: single-workgroup when W*S <= rog_single_wg_max_bytes(), multi-workgroup
 * otherwise (PR #491 "What", kAllGatherSingleBlockMaxBytes bullet: with one
 * block doing all the work the gather is faster only for small outputs; the
 * crossover here is measured on gfx950).  Kernel: FLAT when out, S and every
 * srcs[r] are 16-byte aligned, else PEER (PR #491 "What", copy_rank_ordered).
 * Multi-workgroup FLAT moves 1 KiB chunks, the first one shorter by
 * k = (out mod 128) / 16 vectors so that the rest start on out's 128-byte
 * lines (k = 0 from 2^31 vectors on): grid = ceil((W*S/16 + k) / 64) one-wave
 * workgroups (capped).
 * PEER copies each payload as a byte head up to a 256-byte boundary of its
 * destination, a body of aligned 16-byte stores, each fed by one 16-byte load
 * of the source bytes at the same payload offset (at any source alignment; or,
 * where the loads stream past the caches, by aligned granules shared between
 * neighbouring lanes, see ROG_PLAN_SHIFTED_LOADS), and a byte tail: the pages'
 * fallback (vector copies only where both sides are aligned, bytes otherwise)
 * extended to misaligned payloads, same bytes as a byte-by-byte copy.
 *
 * Errors (nothing enqueued):
 *   ROG_ERR_INVALID_ARGUMENT  srcs NULL; W < 1 or W > rog_max_peers(); S > 0 and
 *                             out or some srcs[r] NULL.
 *   ROG_ERR_OVERLAP           some [srcs[r], srcs[r]+S) overlaps [out, out+W*S)
 *                             other than exactly (srcs[r] == out + r*S, in place).
 *   ROG_ERR_TOO_LARGE         W*S overflows, or W*S >= 2^36 (64 GiB).
 *   ROG_ERR_LAUNCH            hipLaunchKernel failed (rog_last_hip_error()).
 * S == 0: ROG_OK, nothing enqueued.  Sources may alias one another.
 */
ROG_API rog_status rog_gather(const void *const *srcs, int W, size_t bytes_per_rank,
                              void *out, hipStream_t stream);

/*
 * rog_gather_ex -- rog_gather with the path forced.  ROG_PATH_AUTO behaves
 * exactly like rog_gather.  Forcing SINGLE_WG or MULTI_WG changes only the launch
 * shape, never the bytes written; it lets tests reach each path on every case
 * (the pages' review of the size test asks that the otherwise unreachable
 * single-block branch be covered).  path outside rog_path: INVALID_ARGUMENT.
 */
ROG_API rog_status rog_gather_ex(const void *const *srcs, int W, size_t bytes_per_rank,
                                 void *out, hipStream_t stream, rog_path path);

/*
 * rog_gather_many -- n independent gathers sharing W, in one kernel launch.
 * Tensor t: out_t[r*S_t + i] = srcs_t[r][i].  The pages' all_gather_many
 * (PR #491 review threads on the benchmark) gathers a list of tensors with a
 * single synchronisation of the ranks and without copying them into one
 * buffer first; here every tensor keeps its own caller-provided
 * output and its own alignment class (flat or per-peer).
 *
 * descs  host array of n descriptors (each with a host array of W pointers).
 * n      0 <= n <= rog_max_batch(); n == 0 or all S_t == 0: ROG_OK, nothing
 *        enqueued.  n*W must not exceed rog_max_batch_pointers().
 * Errors: as rog_gather for each tensor; outputs of different tensors must not
 * overlap each other (ROG_ERR_OVERLAP), and a tensor's sources must not overlap
 * another tensor's output; limits exceeded: ROG_ERR_TOO_LARGE.
 */
ROG_API rog_status rog_gather_many(const rog_gather_desc *descs, int n, int W,
                                   hipStream_t stream);

/*
 * rog_plan -- validate exactly as rog_gather_ex and describe the launch it would
 * make, without any HIP call.  info must be non-NULL (else INVALID_ARGUMENT).
 * Pointers are only inspected as addresses.
 */
ROG_API rog_status rog_plan(const void *const *srcs, int W, size_t bytes_per_rank,
                            const void *out, rog_path path, rog_plan_info *info);

/* Output bytes W*S up to which ROG_PATH_AUTO takes the single-workgroup path
 * (inclusive), measured on MI355X: 32 KiB.  The pages' counterpart is
 * kAllGatherSingleBlockMaxBytes (RL-Align/RL-Kernel PR #491, section "What",
 * the kAllGatherSingleBlockMaxBytes bullet): one block copying the whole
 * output wins only for small outputs, the bound compares output bytes, and its
 * B200 value (64 KiB) was found by measuring both paths, as this one was on
 * gfx950.  Never fails; a constant of the build. */
ROG_API size_t rog_single_wg_max_bytes(void);

/*
 * rog_reduce -- the rank-ordered sum of W payloads of `count` elements:
 *
 *     out[i] = round( ((x_0[i] + x_1[i]) + x_2[i]) + ... + x_{W-1}[i] ),
 *
 * x_r = srcs[r], the sum taken in rank order with every addition an IEEE
 * binary32 addition rounded to nearest-even, bf16 and binary16 elements
 * widened to binary32 exactly, the first term taken as it is (a lone -0 stays
 * -0), and the result rounded once to `dtype` (nearest-even; binary16 with
 * gradual underflow and overflow to infinity; a NaN stays a NaN, its payload
 * unspecified).  Every element is summed by one thread in that fixed order, so
 * the result is the same bits on every call, whatever the launch shape.
 *
 * This is the reduction at the heart of the pages' deterministic all_reduce
 * and reduce_scatter (RL-Align/RL-Kernel PR #491, "Not in this PR": their
 * single-block paths grow with size as the gather's did; 523 us at 256 KiB
 * per rank on 8 GPUs).  The pages print no arithmetic: they call their backend
 * a fixed tree (the author's replies on the benchmark's recorded backend)
 * without saying which; the left-deep rank-order chain in binary32 above is
 * this library's reading of it.  On one GPU the W ranks are W caller-owned
 * device buffers: an all-reduce is rog_reduce over the W inputs, rank r's share
 * of a reduce-scatter is rog_reduce over the W inputs' r-th shards.
 *
 * srcs    host array of W device pointers, each to `count` elements of dtype,
 *         aligned to the element size (any alignment beyond that).
 * W       1 <= W <= rog_max_peers().
 * count   elements per payload (and in out).
 * dtype   ROG_DTYPE_F32, ROG_DTYPE_BF16 or ROG_DTYPE_F16.
 * out     device pointer to `count` writable elements, element-aligned.  out
 *         may be exactly one (or several) of the srcs (in place); any other
 *         overlap with a source is an error.  Sources may alias each other.
 * stream  HIP stream of the current device.
 *
 * Path: single-workgroup when the source bytes W * count * element size are
 * <= rog_reduce_single_wg_max_bytes() (inclusive, measured on gfx950; the
 * pages test their all-reduce bound on input bytes too), multi-workgroup
 * otherwise.
 * Errors (nothing enqueued):
 *   ROG_ERR_INVALID_ARGUMENT  srcs NULL; W out of range; dtype or path unknown;
 *                             count > 0 and out or some srcs[r] NULL or not
 *                             aligned to the element size.
 *   ROG_ERR_OVERLAP           a source overlaps out other than exactly.
 *   ROG_ERR_TOO_LARGE         count * element size overflows or is >= 2^36.
 *   ROG_ERR_LAUNCH            hipLaunchKernel failed (rog_last_hip_error()).
 * count == 0: ROG_OK, nothing enqueued.
 */
ROG_API rog_status rog_reduce(const void *const *srcs, int W, size_t count, rog_dtype dtype,
                              void *out, hipStream_t stream);

/* rog_reduce with the path forced (changes the launch shape, never the bits). */
ROG_API rog_status rog_reduce_ex(const void *const *srcs, int W, size_t count, rog_dtype dtype,
                                 void *out, hipStream_t stream, rog_path path);

/* Validate exactly as rog_reduce_ex and describe the launch, without any HIP
 * call (kernel ROG_KERNEL_REDUCE, units = count). */
ROG_API rog_status rog_reduce_plan(const void *const *srcs, int W, size_t count, rog_dtype dtype,
                                   const void *out, rog_path path, rog_plan_info *info);

/* Source bytes (W * count * element size) up to which ROG_PATH_AUTO runs
 * rog_reduce on one workgroup (inclusive), measured on MI355X: 64 KiB.  The
 * bound is compared with input bytes because the pages' all-reduce /
 * reduce-scatter fast-path bound is (RL-Align/RL-Kernel PR #491, the author's
 * reply on the benchmark's --size-bytes: the 256 KiB threshold is tested on
 * the per-rank input, world size x the output for reduce_scatter).  Never
 * fails; a constant of the build. */
ROG_API size_t rog_reduce_single_wg_max_bytes(void);

/* One tensor of a batched sum: W source pointers, its output, its count. */
typedef struct {
    const void *const *srcs;   /* W device pointers (host array)                  */
    void *out;                 /* device pointer to `count` elements              */
    size_t count;              /* elements of this tensor; 0 is allowed           */
} rog_reduce_desc;

/*
 * rog_reduce_many -- n independent rank-ordered sums sharing W and dtype, in one
 * kernel launch: tensor t gets out_t[i] = the rank-ordered sum of srcs_t[r][i]
 * (exactly as rog_reduce).  The pages' reduce_scatter_many / all_gather_many
 * (PR #491, "Tests" and the review threads on the benchmark) batch a list of
 * tensors under a single synchronisation of the ranks; here every tensor keeps its own
 * caller-provided output and the whole batch is one launch.
 *
 * descs  host array of n descriptors (each with a host array of W pointers).
 * n      0 <= n <= rog_max_batch(); n == 0 or all counts 0: ROG_OK, nothing
 *        enqueued.  n*W must not exceed rog_max_batch_pointers().
 * Errors: as rog_reduce for each tensor; besides, a tensor's output must not
 * overlap another tensor's output or sources (ROG_ERR_OVERLAP); limits
 * exceeded: ROG_ERR_TOO_LARGE.  Always the multi-workgroup shape.
 */
ROG_API rog_status rog_reduce_many(const rog_reduce_desc *descs, int n, int W, rog_dtype dtype,
                                   hipStream_t stream);

/* ===========================================================================
 * The vocabulary side of a policy: log probabilities of given tokens over W
 * vocabulary shards in rank order, their gradient, and the policy loss.
 *
 * A policy head that is split over W ranks leaves W shards of logits, rank r
 * holding `width` columns of every row.  On one GPU the W ranks are W
 * caller-owned device buffers, as above.  A row is its shards' columns one
 * after the other in rank order; V is the sum of the widths.
 *
 * Beside the common rules:
 *  - A row's result depends, bit for bit, on its logits, the shards' widths and
 *    the temperature alone: not on how many rows a call has, the row's place
 *    among them, the launch form, alignment or strides.  A token scored alone
 *    and in a batch gets the same bits.
 *  - A workspace is device memory of the caller, aligned to 16 bytes.  It is
 *    zero-filled by the caller once, before its first use; every call leaves
 *    it ready for the next.  Calls that may run at the same time (on different
 *    streams) each need their own.
 *  - All sums and row statistics are held in binary32 or binary64.
 *  - Logits are read inside their rows, or inside the aligned 32-bit word that
 *    holds some of a row's bytes; what is read beyond a row is never used.
 * ======================================================================== */

/* One vocabulary shard: row i's columns are logits[i * row_stride + 0 .. width). */
typedef struct {
    const void *logits;        /* device pointer, aligned to the element size     */
    int64_t row_stride;        /* elements from a row to the next; >= 0           */
    int64_t width;             /* columns; 0 is allowed                           */
} rog_logit_shard;

/* One shard's gradient: the width of the logits' shard, a row stride of its own. */
typedef struct {
    void *grad;                /* device pointer, aligned to the element size     */
    int64_t row_stride;        /* elements; >= width where there are rows         */
} rog_grad_shard;

/* What rog_logprob writes; any of them may be NULL (not wanted). */
typedef struct {
    float *logp;               /* [rows]        log probability of the row's token */
    float *entropy;            /* [rows]        in nats                            */
    float *lse;                /* [rows]        log-sum-exp of the scaled logits   */
    float *top_logp;           /* [rows][top_k] log probabilities, best first      */
    int64_t *top_ids;          /* [rows][top_k] their columns in the whole row     */
} rog_logprob_out;

typedef enum {
    ROG_LOGPROB_AUTO = 0,
    ROG_LOGPROB_ROW = 1,       /* one workgroup per row                           */
    ROG_LOGPROB_SPLIT = 2,     /* one workgroup per 4 blocks of a row, the last of a
                                  row to finish joins them (longer rows only)      */
    ROG_LOGPROB_WAVE = 3       /* one wave per row: all rows of at most 4 blocks, and
                                  no others                                       */
} rog_logprob_form;

/* The launch a call would make. */
typedef struct {
    int32_t form;              /* resolved rog_logprob_form (AUTO: nothing to do)  */
    uint32_t grid, block;      /* workgroups, threads per workgroup               */
    uint32_t blocks;           /* blocks of at most 2048 columns per row          */
    uint64_t workspace_bytes;  /* workspace that the call needs (0: none)         */
} rog_head_plan_info;

/*
 * rog_logprob -- per row, with z_j = x_j / temperature over its V columns:
 *
 *     lse = log sum_j e^{z_j},  logp = z_token - lse,
 *     entropy = -sum_j p_j log p_j  (p_j = e^{z_j - lse}),
 *     the top_k largest x_j, ties to the lowest column, as (column, z_j - lse).
 *
 * tokens   device array of `rows` columns, or NULL (then out->logp must be NULL
 *          and every row is scored).  A row whose token is negative is not
 *          scored, whatever its logits: 0 in logp, entropy, lse and top_logp, -1 in
 *          top_ids.  A token of V or more: the row's logp is NaN.
 * top_k    0 .. rog_max_top_k().
 *
 * Logits of -inf have probability 0 and are never alternatives: where a row has
 * fewer than top_k others, the rest is column -1, log probability -inf.  A row
 * that its mask leaves nothing (only -inf, or V = 0): lse = logp = -inf,
 * entropy 0.  A NaN or +inf anywhere in a row makes every number of it NaN and
 * its alternatives' columns -1.  Rows masked with the type's lowest finite
 * value keep their meaning (lse is held within the finite range).
 *
 * lse is one binary32 number, so at |lse| = 2^e its rounding leaves up to
 * 2^(e - 24) of it open: 0.002 at 65504, 4 at 10^8.  logp, entropy and top_logp
 * are formed from the row's sums, not from lse, and have none of that.
 *
 * Errors (nothing enqueued):
 *   ROG_ERR_INVALID_ARGUMENT  shards or out NULL; W out of range; dtype, form or
 *                             top_k out of range; temperature outside
 *                             [2^-10, 2^10]; a negative stride or width; a
 *                             needed pointer NULL or misaligned; logp without
 *                             tokens; a WAVE form for longer rows; a workspace
 *                             that is NULL, misaligned or too small.
 *   ROG_ERR_OVERLAP           an output overlaps a shard, the tokens, the
 *                             workspace or another output.
 *   ROG_ERR_TOO_LARGE         rows or V of 2^31 or more, address overflow, or 2^31
 *                             workgroups or more.
 *   ROG_ERR_LAUNCH            hipLaunchKernel failed (rog_last_hip_error()).
 * rows == 0: ROG_OK, nothing enqueued.
 */
ROG_API rog_status rog_logprob(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype,
                               float temperature, const int64_t *tokens, int top_k,
                               const rog_logprob_out *out, void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* rog_logprob with the launch form forced (never changes the bits).  SPLIT takes
 * at most rog_logprob_max_split_rows() rows. */
ROG_API rog_status rog_logprob_ex(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype,
                                  float temperature, const int64_t *tokens, int top_k,
                                  const rog_logprob_out *out, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream, rog_logprob_form form);

/* The launch form and the workspace that rog_logprob_ex would take for rows of
 * these widths (only the shards' widths are read; no HIP call). */
ROG_API rog_status rog_logprob_plan(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype,
                                    int top_k, rog_logprob_form form, rog_head_plan_info *info);

/*
 * rog_logprob_grad -- the gradient of sum_i (g_logp_i logp_i + g_entropy_i
 * entropy_i) in every logit, from what rog_logprob wrote:
 *
 *     dx_j = (g_logp (1[j = token] - p_j) - g_entropy p_j (log p_j + entropy)) / temperature
 *
 * rounded once to the logits' type.  lse and entropy are rog_logprob's of the
 * same logits, widths and temperature.  g_entropy may be NULL (0).  A row that
 * is not scored or that its mask leaves nothing gets zeros; a token of V or
 * more, or a NaN in lse, NaN.
 *
 * p_j = e^{x_j / temperature - lse} has lse's rounding in it: at |lse| = 2^e it is
 * held to a factor of e^{2^(e - 23)} (2^-17 for |lse| up to 64, 0.4 % at 65504;
 * binary32 logits beyond 10^6 that differ by little are not resolved).  Rows that
 * are uniform over their largest logits -- all of a row masked with one value, or
 * a row that is sure of one token -- have p_j = e^{-entropy} there and are right
 * at any size.  Where a temperature below 1 takes a row's largest logit past the
 * binary32 range, lse is held at the range's end and every logit that passes it
 * counts as a largest one.
 *
 * grads    W gradients.  A gradient may be exactly its logits' shard (same
 *          address and stride: in place); any other overlap is an error.
 *          Column slices of one matrix are told apart; slices with different
 *          row strides overlap here if their whole extents do.
 *          Bytes between the rows of a gradient are not written.
 * Errors as rog_logprob; a row stride below the width is INVALID_ARGUMENT.
 */
ROG_API rog_status rog_logprob_grad(const rog_logit_shard *shards, const rog_grad_shard *grads, int W, size_t rows,
                                    rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse,
                                    const float *entropy, const float *g_logp, const float *g_entropy,
                                    hipStream_t stream);

/* Inputs of the policy loss: device arrays of n binary32 values. */
typedef struct {
    const float *logp;         /* log probability now                              */
    const float *old_logp;     /* when the token was sampled                       */
    const float *advantage;
    const float *weight;       /* weight in the sums; 0: the token counts for nothing,
                                  whatever its other values.  NULL: 1 / n each     */
    const float *ref_logp;     /* under the reference policy; NULL: no KL term     */
    const float *entropy;      /* NULL: no entropy term                            */
} rog_policy_in;

typedef struct {
    float clip_low;            /* 0 <= clip_low <= 1                               */
    float clip_high;           /* >= 0; infinity: not clipped above                */
    float kl_coef;             /* finite                                           */
    float entropy_coef;        /* finite                                           */
    float grad_scale;          /* finite; factor of both gradients (not of stats)  */
} rog_policy_params;

typedef struct {
    float *stats;              /* [4]: loss, sum w kl, sum w entropy, sum w [clipped] */
    float *g_logp;             /* [n] or NULL                                      */
    float *g_entropy;          /* [n] or NULL (NULL where entropy is NULL)         */
} rog_policy_out;

/*
 * rog_policy_loss -- the clipped policy loss over n tokens and its gradient:
 *
 *     d = logp - old_logp, q = ref_logp - logp        (binary32 differences)
 *     clipped = advantage > 0 ? d > hi : advantage < 0 && d < lo
 *     l = -advantage e^{clipped ? the bound passed : d}
 *         + kl_coef (e^q - 1 - q) - entropy_coef entropy
 *     loss = sum_i weight_i l_i
 *     g_logp_i = grad_scale weight_i (-advantage e^d [not clipped] - kl_coef (e^q - 1))
 *     g_entropy_i = -grad_scale weight_i entropy_coef
 *
 * with lo = log(1 - clip_low) and hi = log(1 + clip_high) in binary32.  Weights
 * carry the ragged batch: 1 / tokens for a mean over tokens, 1 / (sequences *
 * length) for a mean over sequences, 0 for prompt and padding.  A token's own
 * l, KL and entropy are binary32; weighted they are exact in binary64, where the
 * sums are taken in an order that depends on n alone, and rounded once.
 *
 * e^d and e^q are binary32: infinite past log of its largest value, 88.72.  A token
 * of advantage 0 adds nothing of its ratio, however large, and with kl_coef 0 the
 * KL is in the stats alone.
 *
 * An output array may be exactly one of the input arrays; any other overlap, of the
 * workspace with any array too, is ROG_ERR_OVERLAP.  n == 0: stats are zero.  n of 2^34 or more: TOO_LARGE.
 */
ROG_API rog_status rog_policy_loss(const rog_policy_in *in, size_t n, const rog_policy_params *params,
                                   const rog_policy_out *out, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* Workspace bytes of rog_policy_loss over n tokens (0: none is needed). */
ROG_API size_t rog_policy_loss_workspace_bytes(size_t n);

/* Limits; constants of the build. */
ROG_API int rog_max_top_k(void);
ROG_API int rog_logprob_max_split_rows(void);

/* Largest W accepted: 64, the capacity of the kernel arguments, which carry
 * every source pointer.  The pages' collectives run over a same-host group of
 * at most eight ranks (RL-Align/RL-Kernel PR #491, "Security Architecture
 * Review", "Security Blast Radius"), so every group size they use fits.
 * Never fails; a constant of the build. */
ROG_API int rog_max_peers(void);

/* Largest n accepted by rog_gather_many, and the largest n*W. */
ROG_API int rog_max_batch(void);
ROG_API int rog_max_batch_pointers(void);

/* hipError_t of the last failed launch on this thread (0 if none). */
ROG_API int rog_last_hip_error(void);

/* Static, human-readable name of a status code ("ROG_OK", ...). */
ROG_API const char *rog_status_string(rog_status s);

#ifdef __cplusplus
}
#endif

#endif /* ROG_H */
