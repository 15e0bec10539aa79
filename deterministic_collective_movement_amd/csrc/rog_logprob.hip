// rog_logprob.hip -- HIP kernels of the token log probabilities for gfx950
// (CDNA4) and the C entry points that launch them.
//
// Per row of V logits x_j, z_j = x_j log2(e) / T, in one pass over the row:
// every lane keeps the partial states (m, s, t) of its columns (rog_head_device.h),
// states are joined in a fixed order, and with M, S, T' of the whole row
//     L = log2 S,  lse = (ref(M) + L) ln 2,  logp = ((z_token - ref(M)) - L) ln 2,
//     entropy = (L - T' / S) ln 2.
// The K best alternatives come without a second pass over the row: each lane
// leaves the maxima of its blocks in a table in shared memory.  The K-th largest
// of the 64 lanes' row maxima is a value that at least K columns reach, so only
// table entries that reach it can hold one of the K best, and only their
// columns (about K of 2048 entries) are read again.
#include <hip/hip_runtime.h>

#include "rog_head_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

constexpr uint32_t kWaves = kHeadThreads / 64;
constexpr uint32_t kSlots = 8;                 // table entries per lane and column
constexpr uint32_t kEntries = kWaves * kSlots * 64;
constexpr uint32_t kListCap = 512;             // candidates held at once

// Orders logits as unsigned numbers; -0 counts as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = f32_bits(x + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) {
    return bits_f32(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
constexpr uint32_t kOrderMinusInf = 0x007FFFFFu;   // order_of(-inf)

// Shared memory of one workgroup.
struct Shared {
    float m[kWaves][64], s[kWaves][64], t[kWaves][64];   // the columns' states
    float row[4];            // ref(M), L, M; written by the first wave
    uint32_t count[4];       // hits, candidates, extreme rows' count
    uint64_t floor_key;      // candidates are at or above it
};
struct SharedTop {
    float tab[kEntries];           // [column][slot][lane]: largest logit
    uint16_t hits[kEntries];
    uint64_t list[kListCap];
};

template <bool TOP> struct SharedFor { typedef uint32_t type; };
template <> struct SharedFor<true> { typedef SharedTop type; };

constexpr float kMaxFinite = 3.40282347e38f;

// What a row comes to: the reference of its largest logit m, l = log2 S, and
// lse in nats, held in the finite range, so that a row masked with the lowest
// finite values does not read as one masked with -inf.
struct Row {
    float r, l, m, lse;
    bool extreme;
    // log probability of a logit of the row
    __device__ __forceinline__ float logp(float x, const LogprobArgs &a) const {
        if (extreme) return (x - m) * a.inv_t - l * kLn2;
        if (x < -a.bound) return __builtin_fmaf(x, a.inv_t, -lse);      // x * scale may overflow
        return (__builtin_fmaf(x, a.scale, -r) - l) * kLn2;
    }
};

// Joins the 64 lanes' states (every lane ends with the same one up to the
// order of its sums; lane 0's is taken).
__device__ __forceinline__ State join_lanes(State st, const Scaling &c) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        st = join(st, State{__shfl_xor(st.m, d), __shfl_xor(st.s, d), __shfl_xor(st.t, d)}, c);
    return State{bits_f32(uniform(f32_bits(st.m))), bits_f32(uniform(f32_bits(st.s))), bits_f32(uniform(f32_bits(st.t)))};
}

// The columns of one table entry: block j of column `w` is block
// ((j / 4) * 4 + w) * 4 + j % 4 of the row.
__device__ __forceinline__ uint32_t column_block(uint32_t w, uint32_t j) { return ((j / 4) * 4 + w) * 4 + (j & 3); }

// The K best alternatives of a row from its table.  Called by the whole
// workgroup; lane_m: in the first wave, the lane's largest logit in the row.
template <int DT>
__device__ void alternatives(const LogprobArgs &a, uint32_t row, float lane_m, const Row &v, Shared &sh, SharedTop &top) {
    constexpr uint32_t per = Logit<DT>::kPerVec;
    const uint32_t tid = threadIdx.x, K = a.top_k;
    if (tid < 64) {
        // the K-th largest of the lanes' maxima, bit by bit
        const uint32_t o = order_of(lane_m);
        uint32_t k = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t tryk = k | 1u << bit;
            if (uint32_t(__popcll(__ballot(o >= tryk))) >= K) k = tryk;
        }
        if (k <= kOrderMinusInf) k = kOrderMinusInf + 1;      // -inf is no alternative
        if (tid == 0) sh.floor_key = uint64_t(k) << 32;
    }
    uint64_t floor_key;
    for (;;) {
        if (tid == 0) sh.count[0] = sh.count[1] = 0;
        __syncthreads();
        floor_key = sh.floor_key;
        const float floor_x = from_order(uint32_t(floor_key >> 32));
        for (uint32_t e = tid; e < kEntries; e += kHeadThreads)
            if (top.tab[e] >= floor_x) top.hits[atomicAdd(&sh.count[0], 1u)] = uint16_t(e);
        __syncthreads();
        const uint32_t vecs_shift = a.slot_shift + (Logit<DT>::kVecs == 8 ? 3 : 2);
        const uint64_t tasks = uint64_t(sh.count[0]) << vecs_shift;
        for (uint64_t q = tid; q < tasks; q += kHeadThreads) {
            const uint32_t e = top.hits[q >> vecs_shift], i = uint32_t(q) & ((1u << vecs_shift) - 1);
            const uint32_t w = e / (kSlots * 64), slot = (e / 64) % kSlots, el = e % 64;
            const uint32_t b = column_block(w, (slot << a.slot_shift) + i / Logit<DT>::kVecs);
            if (b >= a.blocks) continue;
            const BlockAt at = block_at<DT>(a.sh, 0, row, b);
            const uint32_t vi = i % Logit<DT>::kVecs;
            const vec16 vec = load_vec<DT>(at.p, at.n, vi, el);
            float x[per];
            widen_vec<DT>(vec, x);
#pragma unroll
            for (uint32_t k = 0; k < per; ++k) {
                const uint64_t key = uint64_t(order_of(x[k])) << 32 | uint32_t(~(at.col + (64 * vi + el) * per + k));
                if (x[k] >= floor_x && key >= floor_key) {
                    const uint32_t n = atomicAdd(&sh.count[1], 1u);
                    if (n < kListCap) top.list[n] = key;
                }
            }
        }
        __syncthreads();
        const uint32_t n = sh.count[1];
        if (n <= kListCap) break;
        // More columns reach the floor than the list holds (many equal logits):
        // the K-th best of those listed is a higher floor that K columns reach.
        // It rises with every turn, since the list holds more than K.
        for (uint32_t q = tid; q < kListCap; q += kHeadThreads) {
            const uint64_t key = top.list[q];
            uint32_t above = 0;
            for (uint32_t k = 0; k < kListCap; ++k) above += top.list[k] > key;
            if (above == K - 1) sh.floor_key = key;
        }
        __syncthreads();
    }
    const uint32_t n = sh.count[1];
    for (uint32_t q = tid; q < n; q += kHeadThreads) {
        const uint64_t key = top.list[q];
        uint32_t above = 0;
        for (uint32_t k = 0; k < n; ++k) above += top.list[k] > key;
        if (above < K) {
            const float x = from_order(uint32_t(key >> 32));
            const uint64_t o = uint64_t(row) * K + above;
            if (a.top_ids) a.top_ids[o] = ~uint32_t(key);
            if (a.top_logp) a.top_logp[o] = v.logp(x, a);
        }
    }
    for (uint32_t q = n + tid; q < K; q += kHeadThreads) {
        const uint64_t o = uint64_t(row) * K + q;
        if (a.top_ids) a.top_ids[o] = -1;
        if (a.top_logp) a.top_logp[o] = -kInf;
    }
}

// The same numbers for a whole row: one that is not scored, holds NaN or +inf,
// or is left nothing.
__device__ __forceinline__ void write_plain_row(const LogprobArgs &a, uint32_t row, uint32_t i, uint32_t step, float logp,
                                                float entropy, float lse, float top_logp) {
    if (i == 0) {
        if (a.logp) a.logp[row] = logp;
        if (a.entropy) a.entropy[row] = entropy;
        if (a.lse) a.lse[row] = lse;
    }
    for (uint32_t k = i; k < a.top_k; k += step) {
        if (a.top_logp) a.top_logp[uint64_t(row) * a.top_k + k] = top_logp;
        if (a.top_ids) a.top_ids[uint64_t(row) * a.top_k + k] = -1;
    }
}

// The logit of column `tok` of a row (tok below V).
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobArgs &a, uint32_t row, uint32_t tok) {
    uint32_t r = 0;
    while (r + 1 < a.W && a.sh.col0[r + 1] <= tok) ++r;
    return load_logit<DT>((gbyte *)a.sh.x[r] + int64_t(row) * a.sh.stride[r] + uint64_t(tok - a.sh.col0[r]) * Logit<DT>::kSize);
}

// Everything after the partial states: called by the whole workgroup with the
// columns' states in shared memory.
template <int DT, bool TOP>
__device__ void finish_row(const LogprobArgs &a, uint32_t row, int64_t tok, Shared &sh, SharedTop *top) {
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const Scaling c{a.scale, a.bound};
    float lane_m = -kInf;
    if (tid < 64) {
        State st[kWaves];
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) st[w] = State{sh.m[w][lane], sh.s[w][lane], sh.t[w][lane]};
        State all = join(join(st[0], st[1], c), join(st[2], st[3], c), c);
        lane_m = all.m;
        all = join_lanes(all, c);
        if (tid == 0) {
            sh.row[0] = c.ref(all.m);
            sh.row[1] = log2f(all.s);
            sh.row[2] = all.m;
            sh.row[3] = sh.row[1] - all.t / all.s;
            sh.count[2] = 0;
        }
    }
    __syncthreads();
    Row v{sh.row[0], sh.row[1], sh.row[2], (sh.row[0] + sh.row[1]) * kLn2, false};
    float entropy = sh.row[3] * kLn2;
    const float nan = __builtin_nanf("");
    if (!(v.m < kInf)) {
        write_plain_row(a, row, tid, kHeadThreads, nan, nan, nan, nan);
        return;
    }
    const bool token = tok < int64_t(a.vocab);      // tok < 0 never comes here, except for tokens == NULL
    if (v.m == -kInf) {
        write_plain_row(a, row, tid, kHeadThreads, token ? -kInf : nan, 0.0f, -kInf, -kInf);
        return;
    }
    if (v.m >= a.bound || v.m <= -a.bound) {
        // Logits this large lie so far apart that any but the largest has
        // probability 0: the row is uniform over the columns that equal it.
        uint32_t n = 0, r = 0;
        for (uint32_t b = tid / 64; b < a.blocks; b += kWaves) {
            const BlockAt at = block_at<DT>(a.sh, r, row, b);
            r = at.shard;
            for (uint32_t i = 0; i < Logit<DT>::kVecs; ++i) {
                float x[Logit<DT>::kPerVec];
                widen_vec<DT>(load_vec<DT>(at.p, at.n, i, lane), x);
                for (uint32_t k = 0; k < Logit<DT>::kPerVec; ++k) n += x[k] == v.m;
            }
        }
        atomicAdd(&sh.count[2], n);
        __syncthreads();
        v.extreme = true;
        v.l = log2f(float(sh.count[2]));
        v.lse = __builtin_amdgcn_fmed3f(__builtin_fmaf(v.m, a.inv_t, v.l * kLn2), -kMaxFinite, kMaxFinite);
        entropy = v.l * kLn2;
    }
    if (tid == 0) {
        if (a.lse) a.lse[row] = v.lse;
        if (a.entropy) a.entropy[row] = entropy;
        if (a.logp) a.logp[row] = token ? v.logp(token_logit<DT>(a, row, uint32_t(tok)), a) : nan;
    }
    if constexpr (TOP) alternatives<DT>(a, row, lane_m, v, sh, *top);
}

// One workgroup per row: wave w takes column w's quads in turn.
template <int DT, bool TOP>
__global__ __launch_bounds__(kHeadThreads) void rog_logprob_row_kernel(LogprobArgs) {
    const LogprobArgs &a = launch_args<LogprobArgs>();
    __shared__ Shared sh;
    __shared__ typename SharedFor<TOP>::type top;
    const uint32_t tid = threadIdx.x, lane = tid & 63, w = uniform(tid / 64);
    const Scaling c{a.scale, a.bound};
    for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t tok = a.tokens ? a.tokens[row] : 0;
        if (tok < 0) {
            write_plain_row(a, row, tid, kHeadThreads, 0.0f, 0.0f, 0.0f, 0.0f);
            continue;
        }
        __syncthreads();                                   // the row before is done with the shared memory
        if constexpr (TOP) {
            for (uint32_t e = tid; e < kEntries; e += kHeadThreads) top.tab[e] = -kInf;
            __syncthreads();
        }
        State column = no_state();
        uint32_t r = 0;
        for (uint32_t q = w; q < a.quads; q += kWaves) {
            State quad[4];
#pragma unroll 1
            for (uint32_t i = 0; i < 4; ++i) {
                quad[i] = no_state();
                const uint32_t b = 4 * q + i;
                if (b >= a.blocks) continue;
                const BlockAt at = block_at<DT>(a.sh, r, row, b);
                r = at.shard;
                vec16 v[Logit<DT>::kVecs];
                load_block<DT>(at, lane, v);
                float x[32];
#pragma unroll
                for (uint32_t k = 0; k < Logit<DT>::kVecs; ++k) widen_vec<DT>(v[k], x + k * Logit<DT>::kPerVec);
                quad[i] = state_of(x, c);
                if constexpr (TOP) {
                    float &e = top.tab[(w * kSlots + (((q / kWaves) * 4 + i) >> a.slot_shift)) * 64 + lane];
                    e = max_nan(e, quad[i].m);
                }
            }
            column = join(column, join(join(quad[0], quad[1], c), join(quad[2], quad[3], c), c), c);
        }
        sh.m[w][lane] = column.m;
        sh.s[w][lane] = column.s;
        sh.t[w][lane] = column.t;
        __syncthreads();
        finish_row<DT, TOP>(a, row, tok, sh, TOP ? (SharedTop *)&top : nullptr);
    }
}

template <typename K>
const void *kfn(K *k) { return reinterpret_cast<const void *>(k); }

template <int DT>
const void *logprob_kernel(const LogprobPlan &p) {
    const bool top = p.args.top_ids || p.args.top_logp;
    return top ? kfn(&rog_logprob_row_kernel<DT, true>) : kfn(&rog_logprob_row_kernel<DT, false>);
}

rog_status launch_logprob(LogprobPlan &p, hipStream_t stream) {
    const void *k = p.dtype == ROG_DTYPE_BF16  ? logprob_kernel<ROG_DTYPE_BF16>(p)
                    : p.dtype == ROG_DTYPE_F16 ? logprob_kernel<ROG_DTYPE_F16>(p)
                                               : logprob_kernel<ROG_DTYPE_F32>(p);
    void *params[] = {&p.args};
    const hipError_t e = hipLaunchKernel(k, dim3(p.info.grid), dim3(p.info.block), params, 0, stream);
    if (e != hipSuccess) {
        g_last_hip_error = int(e);
        return ROG_ERR_LAUNCH;
    }
    return ROG_OK;
}

}  // namespace
}  // namespace rog

extern "C" {

ROG_API rog_status rog_logprob_ex(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype,
                                  float temperature, const int64_t *tokens, int top_k, const rog_logprob_out *out,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream,
                                  rog_logprob_form form) {
    rog::LogprobPlan p;
    const rog_status st = rog::plan_logprob(shards, W, rows, dtype, temperature, tokens, top_k, out, workspace,
                                            workspace_bytes, form, true, &p);
    if (st != ROG_OK || p.info.form == ROG_LOGPROB_AUTO) return st;
    return rog::launch_logprob(p, stream);
}

ROG_API rog_status rog_logprob(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype,
                               float temperature, const int64_t *tokens, int top_k, const rog_logprob_out *out,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return rog_logprob_ex(shards, W, rows, dtype, temperature, tokens, top_k, out, workspace, workspace_bytes,
                          stream, ROG_LOGPROB_AUTO);
}

}  // extern "C"
