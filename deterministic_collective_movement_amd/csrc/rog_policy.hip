// rog_policy.hip -- HIP kernel of the policy loss for gfx950 (CDNA4) and the C
// entry point that launches it.
//
// Per token: d = logp - old, l = -A e^{clipped ? bound : d} + beta (e^q - 1 - q)
// - c_H H and its derivative.  A workgroup takes 2048 tokens, eight per thread,
// and sums its four totals in binary64 over a fixed tree; the last workgroup to
// finish joins the workgroups' totals in their order.  Bandwidth bound: 24
// bytes read and 8 written per token with every term.
#include <hip/hip_runtime.h>

#include "rog_head_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef const __attribute__((address_space(1))) float gfloat;
typedef const __attribute__((address_space(1))) f32x4u gvec;
typedef __attribute__((address_space(1))) float gfloat_out;
typedef __attribute__((address_space(1))) f32x4u gvec_out;

// e^q - 1 - q without cancellation: its Taylor series to q^9 / 9! for |q| <= 1/2
// (what is left out is below 2^-27 of the sum), e^q - 1 - q in binary64 beyond.
__device__ __forceinline__ float kl_term(float q) {
    if (fabsf(q) <= 0.5f) {
        float p = 1.0f / 362880.0f;
        p = __builtin_fmaf(p, q, 1.0f / 40320.0f);
        p = __builtin_fmaf(p, q, 1.0f / 5040.0f);
        p = __builtin_fmaf(p, q, 1.0f / 720.0f);
        p = __builtin_fmaf(p, q, 1.0f / 120.0f);
        p = __builtin_fmaf(p, q, 1.0f / 24.0f);
        p = __builtin_fmaf(p, q, 1.0f / 6.0f);
        p = __builtin_fmaf(p, q, 0.5f);
        return p * q * q;
    }
    return float(double(expf(q)) - 1.0 - double(q));
}

struct Totals {
    double v[4];
    __device__ __forceinline__ void add(const Totals &o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += o.v[i];
    }
};

// Sums the 256 threads' totals over a fixed tree; thread 0 has the result.
__device__ __forceinline__ Totals group_sum(Totals t, double (&sh)[4][4]) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        Totals o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = __shfl_xor(t.v[i], d);
        t.add(o);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        for (int i = 0; i < 4; ++i) sh[threadIdx.x / 64][i] = t.v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) t.v[i] = (sh[0][i] + sh[1][i]) + (sh[2][i] + sh[3][i]);
    return t;
}

__device__ __forceinline__ f32x4 load4(const float *p, uint64_t at, uint32_t n, float none) {
    f32x4 v = {none, none, none, none};
    if (!p) return v;
    gfloat *q = (gfloat *)p + at;
    if (n >= 4) return *(gvec *)q;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i < n) v[i] = q[i];
    return v;
}

__device__ __forceinline__ void store4(float *p, uint64_t at, uint32_t n, f32x4 v) {
    if (!p) return;
    gfloat_out *q = (gfloat_out *)p + at;
    if (n >= 4) {
        *(gvec_out *)q = v;
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i < n) q[i] = v[i];
}

__global__ __launch_bounds__(kHeadThreads) void rog_policy_kernel(PolicyArgs a) {
    __shared__ double sh[4][4];
    __shared__ uint32_t last;
    Totals t = {{0, 0, 0, 0}};
    for (uint32_t k = 0; k < 2; ++k) {
        const uint64_t at = uint64_t(blockIdx.x) * kPolicyGroup + 4 * (k * kHeadThreads + threadIdx.x);
        if (at >= a.n) continue;
        const uint32_t n = a.n - at < 4 ? uint32_t(a.n - at) : 4;
        const f32x4 logp = load4(a.logp, at, n, 0), old = load4(a.old_logp, at, n, 0), adv = load4(a.adv, at, n, 0);
        f32x4 w = load4(a.weight, at, n, a.w_all);
        const f32x4 ref = load4(a.ref, at, n, 0), ent = load4(a.entropy, at, n, 0);
        f32x4 g, gh;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const bool kept = i < n && w[i] != 0.0f;
            const float d = logp[i] - old[i];
            const bool over = adv[i] > 0.0f && d > a.hi, under = adv[i] < 0.0f && d < a.lo;
            const float ratio = over ? a.ratio_hi : under ? a.ratio_lo : expf(d);
            const float pg = -adv[i] * ratio;
            float loss = pg, slope = over || under ? 0.0f : pg, kl = 0.0f;
            if (a.ref) {
                const float q = ref[i] - logp[i];
                kl = kl_term(q);
                loss = __builtin_fmaf(a.kl_coef, kl, loss);
                slope = __builtin_fmaf(-a.kl_coef, expm1f(q), slope);
            }
            const float e = a.entropy ? ent[i] : 0.0f;
            loss = __builtin_fmaf(-a.entropy_coef, e, loss);
            g[i] = kept ? a.grad_scale * w[i] * slope : 0.0f;
            gh[i] = kept ? -(a.grad_scale * w[i] * a.entropy_coef) : 0.0f;
            if (kept) {
                const double wd = double(w[i]);
                t.v[0] += wd * double(loss);
                t.v[1] += wd * double(kl);
                t.v[2] += wd * double(e);
                t.v[3] += over || under ? wd : 0.0;
            }
        }
        store4(a.g_logp, at, n, g);
        store4(a.g_entropy, at, n, gh);
    }
    t = group_sum(t, sh);
    if (a.groups > 1) {
        if (threadIdx.x == 0)
            for (int i = 0; i < 4; ++i) publish(a.part + uint64_t(blockIdx.x) * 4 + i, t.v[i]);
        if (!last_to_arrive(a.counter, a.groups, last)) return;
        t = Totals{{0, 0, 0, 0}};
        for (uint32_t b = threadIdx.x; b < a.groups; b += kHeadThreads) {
            Totals o;
            for (int i = 0; i < 4; ++i) o.v[i] = collect(a.part + uint64_t(b) * 4 + i);
            t.add(o);
        }
        t = group_sum(t, sh);
    }
    if (threadIdx.x == 0)
        for (int i = 0; i < 4; ++i) a.stats[i] = float(t.v[i]);
}

}  // namespace
}  // namespace rog

extern "C" {

ROG_API rog_status rog_policy_loss(const rog_policy_in *in, size_t n, const rog_policy_params *params,
                                   const rog_policy_out *out, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    rog::PolicyPlan p;
    const rog_status st = rog::plan_policy(in, n, params, out, workspace, workspace_bytes, &p);
    if (st != ROG_OK) return st;
    void *args[] = {&p.args};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&rog::rog_policy_kernel), dim3(p.args.groups),
                                         dim3(rog::kHeadThreads), args, 0, stream);
    if (e != hipSuccess) {
        rog::g_last_hip_error = int(e);
        return ROG_ERR_LAUNCH;
    }
    return ROG_OK;
}

}  // extern "C"
