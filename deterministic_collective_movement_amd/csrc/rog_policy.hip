// rog_policy.hip -- HIP kernel of the policy loss for gfx950 (CDNA4) and the C
// entry point that launches it.
//
// Per token: d = logp - old, l = -A e^{clipped ? bound : d} + beta (e^q - 1 - q)
// - c_H H and its derivative.  A workgroup takes a run of tiles of 1024 tokens,
// four tokens per thread with the next tile's loads in flight, and sums its
// four totals in binary64 over a fixed tree (in binary32 even four tokens whose
// advantages cancel would lose the small ones; 0.2 of 31.5 us); the last workgroup
// to finish joins the workgroups' totals in their order.
//
// Bandwidth bound: 24 bytes read and 8 written per token with every term, about
// 93 vector instructions.  4194307 tokens (134 MB) take 31.5 us = 4.3 TB/s:
// some 3 us to start, 3.5 us for the join (131072 tokens take 6.8 us, 1021, one
// workgroup, 3.1), the rest over eight arrays.  The 4097 tiles are 456 runs of
// nine, so some CUs get 18 tiles and the mean is 16.  Two tiles in flight,
// streamed loads, arrival counted over 16 to 128 counters and 768 to 4096
// workgroups, whose runs come out as uneven, were all within 5 % of it.
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

// e^x: 2^(x log2 e), the product's rounding put back as a factor (e^x to about
// two units in the last place; results below 2^-126 are zero).
__device__ __forceinline__ float exp_of(float x) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;      // log2 e
    const float y = x * kHi;
    const float e = exp2_fast(y);
    const float rest = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -y));
    return fabsf(x) < 87.0f ? __builtin_fmaf(e, rest * kLn2, e) : e;     // beyond, e may be infinite or zero
}

// kl = e^q - 1 - q and grow = e^q - 1 without cancellation: the Taylor series of
// kl to q^9 / 9! for |q| <= 1/2 (what is left out is below 2^-27 of it), the
// exponential beyond.
__device__ __forceinline__ void kl_of(float q, float &kl, float &grow) {
    float p = 1.0f / 362880.0f;
    p = __builtin_fmaf(p, q, 1.0f / 40320.0f);
    p = __builtin_fmaf(p, q, 1.0f / 5040.0f);
    p = __builtin_fmaf(p, q, 1.0f / 720.0f);
    p = __builtin_fmaf(p, q, 1.0f / 120.0f);
    p = __builtin_fmaf(p, q, 1.0f / 24.0f);
    p = __builtin_fmaf(p, q, 1.0f / 6.0f);
    p = __builtin_fmaf(p, q, 0.5f);
    const float series = p * q * q, far = exp_of(q) - 1.0f;
    const bool near = fabsf(q) <= 0.5f;
    kl = near ? series : far - q;
    grow = near ? series + q : far;
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

// Four tokens of a thread, as loaded.
struct Four {
    f32x4 logp, old, adv, w, ref, ent;
};

// A thread's four tokens start at `at`; where that runs past n they are read
// from n - 4, and the first at - (n - 4) of them are other threads' (they may
// be overwritten meanwhile where gradients go in place, and are not used).
// Fewer than four tokens in all are read one by one.
__device__ __forceinline__ uint64_t place_of(uint64_t at, uint64_t n) { return n < 4 ? 0 : at < n - 4 ? at : n - 4; }

__device__ __forceinline__ f32x4 load4(const float *p, uint64_t place, uint64_t n, float none) {
    if (!p) return f32x4{none, none, none, none};
    gfloat *q = (gfloat *)p + place;
    if (n >= 4) return *(gvec *)q;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i)
        if (i < n) v[i] = q[i];
    return v;
}

__device__ __forceinline__ Four load_four(const PolicyArgs &a, uint64_t at) {
    const uint64_t place = place_of(at, a.n);
    return Four{load4(a.logp, place, a.n, 0), load4(a.old_logp, place, a.n, 0), load4(a.adv, place, a.n, 0),
                load4(a.weight, place, a.n, a.w_all), load4(a.ref, place, a.n, 0), load4(a.entropy, place, a.n, 0)};
}

// The thread's own of four values, at the tokens they were read from.
__device__ __forceinline__ void store4(float *p, uint64_t place, uint32_t first, uint32_t end, f32x4 v) {
    if (!p) return;
    gfloat_out *q = (gfloat_out *)p + place;
    if (first == 0 && end == 4) {
        __builtin_nontemporal_store(v, (gvec_out *)q);   // 34 -> 31 us at 4194307 tokens; even at small sizes
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i >= first && i < end) q[i] = v[i];
}

__global__ __launch_bounds__(kHeadThreads) void rog_policy_kernel(PolicyArgs a) {
    __shared__ double sh[4][4];
    __shared__ uint32_t last;
    Totals t = {{0, 0, 0, 0}};
    const uint64_t begin = uint64_t(blockIdx.x) * a.tiles * kPolicyTile + 4 * threadIdx.x;
    Four next = load_four(a, begin);
    for (uint32_t k = 0; k < a.tiles; ++k) {
        const uint64_t at = begin + uint64_t(k) * kPolicyTile;
        const Four x = next;
        // the next tile's loads in flight (after the last, the same again)
        next = load_four(a, k + 1 < a.tiles ? at + kPolicyTile : at);
        if (at >= a.n) break;
        const uint64_t place = place_of(at, a.n);
        const uint32_t first = uint32_t(at - place), end = a.n < 4 ? uint32_t(a.n) : 4;
        f32x4 g, gh;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const float w = i >= first && i < end ? x.w[i] : 0.0f;
            const bool kept = w != 0.0f;
            const float d = x.logp[i] - x.old[i], adv = x.adv[i];
            const bool over = adv > 0.0f && d > a.hi, under = adv < 0.0f && d < a.lo, clipped = over || under;
            // no advantage, no term: a finite ratio that binary32 holds as infinite included
            const float pg = -adv * (over ? a.ratio_hi : under ? a.ratio_lo : exp_of(adv == 0.0f && d < kInf ? 0.0f : d));
            float loss = pg, slope = clipped ? 0.0f : pg, kl = 0.0f;
            if (a.ref) {
                float grow;
                kl_of(x.ref[i] - x.logp[i], kl, grow);
                if (a.kl_coef != 0.0f) {        // else it is only watched, and may be infinite
                    loss = __builtin_fmaf(a.kl_coef, kl, loss);
                    slope = __builtin_fmaf(-a.kl_coef, grow, slope);
                }
            }
            if (a.entropy) loss = __builtin_fmaf(-a.entropy_coef, x.ent[i], loss);
            const float gw = a.grad_scale * w;
            g[i] = kept ? gw * slope : 0.0f;
            gh[i] = -(gw * a.entropy_coef);
            // a token's own numbers in binary32, its weighted terms exactly and their sums in binary64
            const double wd = double(w);
            t.v[0] = __builtin_fma(wd, double(kept ? loss : 0.0f), t.v[0]);
            if (a.ref) t.v[1] = __builtin_fma(wd, double(kept ? kl : 0.0f), t.v[1]);
            if (a.entropy) t.v[2] = __builtin_fma(wd, double(kept ? x.ent[i] : 0.0f), t.v[2]);
            t.v[3] += clipped ? wd : 0.0;
        }
        store4(a.g_logp, place, first, end, g);
        store4(a.g_entropy, place, first, end, gh);
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
