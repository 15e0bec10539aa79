// rog_logprob_grad.hip -- HIP kernel of the token log probabilities' gradient
// for gfx950 (CDNA4) and the C entry point that launches it.
//
//     dx_j = (g (1[j = token] - p_j) - h p_j (log p_j + H)) / T,  p_j = e^{x_j / T - lse}
//          = p_j (A + B z_j) + [j = token] g / T,   z_j = log p_j = x_j / T - lse,
//     A = -(g + h H) / T,  B = -h / T:
// one read and one write of every logit, nothing joined between columns.  z is
// rounded once, so where p is large, and z near 0, p keeps its last bits (in
// units of log2, with log2(e) / T rounded before it meets x, a binary32 gradient
// was 2e-7 off; so it is 5e-8).  lse is one rounded number for the row, which
// leaves a factor of e^{2^(e - 24)} open in every p at |lse| = 2^e, up to 2^e = 64
// about as much as the rounding of 1 / T does; from there on 1 / T comes in two
// parts, and rows that are uniform over their largest logits are held to that.
#include <hip/hip_runtime.h>

#include "rog_head_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

constexpr float kLog2E32 = 1.44269502f;
// |lse| above that of any row whose largest logit is below rog_logprob's bound
// (2^30 ln 2, log 2^31, and the roundings of bound, T and lse).
constexpr float kExtreme = 744261248.0f;
// |lse| from which its rounding (2^-18 and more) is looked after: a row that is
// uniform over its largest logits (masked as a whole, or sure of one token) has
// log p = -H at each of them, so a z that lies within the rounding of -H is taken
// to be -H.  Any other z that happens to lie there moves by less than one more
// rounding of lse.
constexpr float kLarge = 64.0f;

// One wave, a workgroup of its own, per piece of a row, its stores streamed.
// Bound by HBM: 4096 x 131072 bf16 over eight shards (2.15 GB) take 327-332 us =
// 6.5-6.6 TB/s with pieces of 2 KB, against 358 with four waves of 4 KB each, 372
// with 1 KB, and 365 and more where waves took several pieces in turn; read once
// and written once (counted: 1.0 times the bytes).  Pieces begin with lines of the
// gradient, whatever the row's alignment: 4000 x 100003 bf16 278 us, against 321
// with pieces counted from the row's beginning, whose ends share lines.
// 1021 x 50257 binary16, whose logits a forward pass left in the Infinity Cache,
// 31-31.5 us (192 MB); 33 x 32003 binary32 3.6 us, a launch and one round trip.
template <int DT, bool NT>
__global__ __launch_bounds__(64) void rog_logprob_grad_kernel(LogprobGradArgs) {
    const LogprobGradArgs &a = launch_args<LogprobGradArgs>();
    hold_front(a);
    constexpr uint32_t per = Logit<DT>::kPerVec, vecs = kGradPieceBytes / (64 * 16), each = vecs * per;
    const uint32_t lane = threadIdx.x;
    const uint32_t group = head_group();
    if (group >= a.groups) return;
    const uint32_t row = divide(group, a.pieces_div), piece = group - row * a.sh.blocks;
    // everything that a wave needs of its row, asked for at once
    const int64_t tok = a.tokens[row];
    const float lse = a.lse[row], H = a.entropy[row], g = a.g_logp[row], h = a.g_entropy ? a.g_entropy[row] : 0.0f;
    Cursor<DT, 64 * each> cur(a.sh, row);
    cur.seek(piece);
    typedef __attribute__((address_space(1))) uint8_t gout;
    gout *const line = (gout *)a.g[cur.shard] + int64_t(row) * a.g_stride[cur.shard];
    // pieces begin where the gradient's 128-byte lines do, but for the first
    const uint32_t head = uint32_t(reinterpret_cast<uintptr_t>((uint8_t *)line) % 128) / Logit<DT>::kSize;
    const uint32_t begin = (piece - cur.first) * (64 * each), end = begin + 64 * each - head;
    const uint32_t off = begin > head ? begin - head : 0;
    if (off >= cur.width) return;
    const BlockAt at = cur.columns(off, (end < cur.width ? end : cur.width) - off);
    gout *const o = line + uint64_t(off) * Logit<DT>::kSize;
    const bool none = tok < 0 || lse == -kInf, bad = tok >= int64_t(a.vocab) || !(lse < kInf);
    const bool tiny = at.n < per;
    float x[each];
    if (none || bad) {
#pragma unroll
        for (uint32_t i = 0; i < each; ++i) x[i] = none ? 0.0f : __builtin_nanf("");
    } else {
        Loaded<vecs> l;
        load_block<DT, NT>(at, lane, l);
        aligned_block<DT>(at.shift, l);
        if (tiny) l.v[0] = load_tiny<DT>(at.p, at.n);
#pragma unroll
        for (uint32_t i = 0; i < vecs; ++i) widen_vec<DT>(l.v[i], x + i * per);
        const float scaled = g * a.inv_t, A = -(g + h * H) * a.inv_t, B = -h * a.inv_t;
        if (fabsf(lse) >= kExtreme) {
            // Logits this large lie so far apart that only those equal to the
            // largest have any probability, the same for each: e^{-H}.
            const float p = expf(-H);
#pragma unroll
            for (uint32_t i = 0; i < each; ++i) {
                // rog_logprob's own lse of such a row, if x[i] is its largest logit
                const float z = __builtin_fmaf(x[i], a.inv_t, __builtin_fmaf(x[i], a.inv_t_rest, H));
                x[i] = x[i] > -kInf && __builtin_amdgcn_fmed3f(z, -3.40282347e38f, 3.40282347e38f) == lse ? -scaled * p : 0.0f;
            }
        } else {
            // -140 stands for anything less (p is zero there), so that 0 * z stays 0; p is at most 1
            if (fabsf(lse) >= kLarge) {
                // half a unit in the last place of lse, and what its sums and H's leave
                const float half = bits_f32((f32_bits(lse) & 0x7F800000u) - (24u << 23));
                const float open = __builtin_fmaf(half, 1.0f / 64, half) + 0x1p-18f;
#pragma unroll
                for (uint32_t i = 0; i < each; ++i) {
                    // the rest of 1 / T times -inf may be NaN: that ends at -140 too
                    const float z = __builtin_fmaf(x[i], a.inv_t_rest, __builtin_fmaf(x[i], a.inv_t, -lse));
                    x[i] = fminf(fmaxf(z, -140.0f), 0.0f);
                    x[i] = fabsf(x[i] + H) <= open ? -H : x[i];
                }
            } else {
#pragma unroll
                for (uint32_t i = 0; i < each; ++i) x[i] = fminf(fmaxf(__builtin_fmaf(x[i], a.inv_t, -lse), -140.0f), 0.0f);
            }
#pragma unroll
            for (uint32_t i = 0; i < each; ++i) x[i] = exp2_fast(x[i] * kLog2E32) * __builtin_fmaf(B, x[i], A);
        }
        const int64_t t = tok - int64_t(at.col);
        if (t >= 0 && t < int64_t(at.n)) {
            // the token is in this piece
#pragma unroll
            for (uint32_t i = 0; i < each; ++i) {
                const uint32_t col = (tiny ? 0 : vec_place<DT>(at.n, i / per, lane)) + i % per;
                x[i] = uint32_t(t) == col ? x[i] + scaled : x[i];
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < vecs; ++i) {
        vec16any v;
#pragma unroll
        for (uint32_t d = 0; d < 4; ++d) v[d] = narrow_word<DT>(x + i * per + d * (per / 4));
        if (!tiny) {
            // where the vector was read: what it shares with other lanes' vectors, they write alike
            __builtin_nontemporal_store(v, (gvec16any_out *)(o + vec_place<DT>(at.n, i, lane) * Logit<DT>::kSize));
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

template <int DT>
const void *grad_kernel(bool nt) {
    return nt ? reinterpret_cast<const void *>(&rog_logprob_grad_kernel<DT, true>)
              : reinterpret_cast<const void *>(&rog_logprob_grad_kernel<DT, false>);
}

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
    const void *k = dtype == ROG_DTYPE_BF16  ? rog::grad_kernel<ROG_DTYPE_BF16>(p.nt_loads)
                    : dtype == ROG_DTYPE_F16 ? rog::grad_kernel<ROG_DTYPE_F16>(p.nt_loads)
                                             : rog::grad_kernel<ROG_DTYPE_F32>(p.nt_loads);
    void *params[] = {&p.args};
    const hipError_t e = hipLaunchKernel(k, rog::head_grid(p.grid), dim3(64), params, 0, stream);
    if (e != hipSuccess) {
        rog::g_last_hip_error = int(e);
        return ROG_ERR_LAUNCH;
    }
    return ROG_OK;
}

}  // extern "C"
