// rog_logprob_grad.hip -- HIP kernel of the token log probabilities' gradient
// for gfx950 (CDNA4) and the C entry point that launches it.
//
//     dx_j = (g (1[j = token] - p_j) - h p_j (log p_j + H)) / T,  p_j = e^{x_j / T - lse}
//          = p_j (A + B y_j) + [j = token] g / T,   y_j = log2 p_j,
//     A = -(g + h H) / T,  B = -h ln 2 / T:
// one read and one write of every logit, nothing joined between columns.
#include <hip/hip_runtime.h>

#include "rog_head_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

constexpr float kLog2EHi = 1.44269502f;                 // log2(e) in two parts
constexpr float kLog2ELo = 1.92596303e-8f;
constexpr float kExtreme = 7.442609e8f;                 // 2^30 ln 2, where rog_logprob's extreme rows begin

// A row's coefficients.
struct Coeffs {
    float a, b, g;        // A, B, g / T
    float hi, lo;         // lse log2(e) = hi + lo
};

// One block's gradient in place of its logits x[].
__device__ __forceinline__ void block_grad(float (&x)[32], const Coeffs &k, float scale) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        // z - lse in base 2; -200 stands for anything less (p is zero there)
        const float y = fmaxf(__builtin_fmaf(x[i], scale, -k.hi) - k.lo, -200.0f);
        x[i] = exp2_fast(y) * __builtin_fmaf(k.b, y, k.a);
    }
}

template <int DT>
__global__ __launch_bounds__(kHeadThreads) void rog_logprob_grad_kernel(LogprobGradArgs) {
    const LogprobGradArgs &a = launch_args<LogprobGradArgs>();
    constexpr uint32_t per = Logit<DT>::kPerVec, vecs = Logit<DT>::kVecs;
    const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64);
    const uint32_t group = blockIdx.y * gridDim.x + blockIdx.x;
    if (group >= a.groups) return;
    const uint32_t row = group / a.splits, b = group % a.splits * kGradBlocks + w;
    if (b >= a.blocks) return;
    const BlockAt at = Cursor<DT>(a.sh, row).at(b);
    typedef __attribute__((address_space(1))) uint8_t gout;
    gout *o = (gout *)a.g[at.shard] + int64_t(row) * a.g_stride[at.shard] + uint64_t(at.off) * Logit<DT>::kSize;
    const int64_t tok = a.tokens[row];
    const float lse = a.lse[row];
    float x[32];
    if (tok < 0 || lse == -kInf) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    } else {
        vec16 v[vecs];
        load_block<DT, false>(at, lane, v);
        const bool tiny = at.n < per;
        if (tiny) v[0] = load_tiny<DT>(at.p, at.n);
        widen_block<DT>(v, x);
        const float g = a.g_logp[row], h = a.g_entropy ? a.g_entropy[row] : 0.0f, H = a.entropy[row];
        Coeffs k;
        k.g = g * a.inv_t;
        k.a = -(g + h * H) * a.inv_t;
        k.b = -h * a.inv_t * kLn2;
        k.hi = lse * kLog2EHi;
        k.lo = __builtin_fmaf(lse, kLog2ELo, __builtin_fmaf(lse, kLog2EHi, -k.hi));
        const bool bad = tok >= int64_t(a.vocab) || !(lse < kInf);
        if (bad) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __builtin_nanf("");
        } else if (fabsf(lse) >= kExtreme) {
            // Logits this large lie so far apart that only those equal to the
            // largest have any probability, the same for each: e^{-H}.
            const float p = expf(-H);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                // rog_logprob's own lse of such a row, if x[i] is its largest logit
                const float z = __builtin_amdgcn_fmed3f(__builtin_fmaf(x[i], a.inv_t, H), -3.40282347e38f, 3.40282347e38f);
                x[i] = x[i] > -kInf && z == lse ? -k.g * p : 0.0f;
            }
        } else {
            block_grad(x, k, a.scale);
        }
        const int64_t t = tok - int64_t(at.col);
        if (!bad && t >= 0 && t < int64_t(at.n)) {
            // the token is in this block
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) {
                const uint32_t col = (tiny ? 0 : vec_place<DT>(at.n, i / per, lane)) + i % per;
                x[i] = uint32_t(t) == col ? x[i] + k.g : x[i];
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < vecs; ++i) {
        vec16 v;
#pragma unroll
        for (uint32_t d = 0; d < 4; ++d) v[d] = narrow_word<DT>(x + i * per + d * (per / 4));
        if (at.n >= per) {
            // where the vector was read: what it shares with other lanes' vectors, they write alike
            *(gvec16any_out *)(o + vec_place<DT>(at.n, i, lane) * Logit<DT>::kSize) = v;
        } else if (i == 0 && lane == 0) {
#pragma unroll
            for (uint32_t e = 0; e + 1 < per; ++e) {
                if (e >= at.n) continue;
                if constexpr (DT == ROG_DTYPE_F32)
                    *(__attribute__((address_space(1))) uint32_t *)(o + e * 4) = v[e];
                else
                    *(__attribute__((address_space(1))) uint16_t *)(o + e * 2) = uint16_t(e & 1 ? v[e / 2] >> 16 : v[e / 2]);
            }
        }
    }
}

template <typename K>
const void *kfn(K *k) { return reinterpret_cast<const void *>(k); }

}  // namespace
}  // namespace rog

extern "C" {

ROG_API rog_status rog_logprob_grad(const rog_logit_shard *shards, const rog_grad_shard *grads, int W, size_t rows,
                                    rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse,
                                    const float *entropy, const float *g_logp, const float *g_entropy,
                                    hipStream_t stream) {
    rog::LogprobGradPlan p;
    const rog_status st = rog::plan_logprob_grad(shards, grads, W, rows, dtype, temperature, tokens, lse, entropy,
                                                 g_logp, g_entropy, &p);
    if (st != ROG_OK || p.grid == 0) return st;
    const void *k = dtype == ROG_DTYPE_BF16  ? rog::kfn(&rog::rog_logprob_grad_kernel<ROG_DTYPE_BF16>)
                    : dtype == ROG_DTYPE_F16 ? rog::kfn(&rog::rog_logprob_grad_kernel<ROG_DTYPE_F16>)
                                             : rog::kfn(&rog::rog_logprob_grad_kernel<ROG_DTYPE_F32>);
    void *params[] = {&p.args};
    const hipError_t e = hipLaunchKernel(k, rog::head_grid(p.grid), dim3(rog::kHeadThreads), params, 0, stream);
    if (e != hipSuccess) {
        rog::g_last_hip_error = int(e);
        return ROG_ERR_LAUNCH;
    }
    return ROG_OK;
}

}  // extern "C"
