// rog_linear_i8.hip -- HIP kernels of the product of 8-bit integers with a scale
// for each token and channel for gfx950 (CDNA4), of the quantization of rows, and
// the C entry points that launch them.
//
//     s_i = max(max_k |x_ik| / 127, 2^-126), q_ik = x_ik / s_i to the nearest integer
//     y_ij = (sum_k q_ik u_jk) s_i r_j
// The sum is exact in 32-bit integers, so y has three roundings of binary32 and
// one to the output's type whatever the order.
#include <hip/hip_runtime.h>

#include "rog_linear_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

// A row per workgroup: the largest magnitude, then the quotients.  Rows of up to
// kHeld vectors of 16 bytes per thread stay in registers between the two, longer ones are
// read again from the caches.  The division is the correctly rounded one, so any plain form gives the same integers.  One row of
// 2048 bf16 3.0 us, 48 of 4096 4.8 (a launch), 4093 of 5120 binary16 21 us (63 MB, 3.0 TB/s), a fiftieth of
// the product behind it.
constexpr uint32_t kQuantThreads = 256;
constexpr int kHeld = 4;

// 8-bit integers of the elements of a vector, in order.
template <int DT>
__device__ __forceinline__ void put_quotients(__attribute__((address_space(1))) uint8_t *to, const vec16 &v, float s, uint32_t n) {
    constexpr int E = Logit<DT>::kPerVec;
    float x[E];
    widen_vec<DT>(v, x);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float q = __builtin_rintf(x[i] / s);
        w[i / 4] |= (uint32_t(q == q ? int(q) : 0) & 0xFF) << (8 * (i % 4));
    }
    typedef uint32_t word2any __attribute__((ext_vector_type(2), aligned(1)));
    typedef uint32_t wordany __attribute__((aligned(1)));
    if (n >= uint32_t(E)) {
        if constexpr (E == 8) *(__attribute__((address_space(1))) word2any *)to = word2any{w[0], w[1]};
        else *(__attribute__((address_space(1))) wordany *)to = w[0];
    } else {
#pragma unroll
        for (uint32_t i = 0; i < uint32_t(E); ++i)
            if (i < n) to[i] = uint8_t(w[i / 4] >> (8 * (i % 4)));
    }
}

template <int DT, bool HELD>
__global__ __launch_bounds__(kQuantThreads) void rog_quantize_kernel(QuantizeArgs p) {
    constexpr uint32_t ES = Logit<DT>::kSize, E = Logit<DT>::kPerVec;
    __shared__ float most[kQuantThreads / 64];
    gbyte *row = (gbyte *)p.x + uint64_t(blockIdx.x) * uint64_t(p.stride);
    const uint32_t t = threadIdx.x, bytes = p.dim * ES;
    vec16 held[kHeld];
    float m = 0;
    const auto largest = [&](const vec16 &v) {
        float x[E];
        widen_vec<DT>(v, x);
#pragma unroll
        for (uint32_t i = 0; i < E; ++i) m = max_nan(m, fabsf(x[i]));
    };
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = row_bytes<ES>(row, (t + i * kQuantThreads) * 16, bytes);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) largest(held[i]);
    } else {
        for (uint32_t at = t * 16; at < bytes; at += kQuantThreads * 16) largest(row_bytes<ES>(row, at, bytes));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = max_nan(m, __shfl_xor(m, d));
    if (t % 64 == 0) most[t / 64] = m;
    __syncthreads();
    m = max_nan(max_nan(most[0], most[1]), max_nan(most[2], most[3]));
    const float s = m < kInf ? fmaxf(m / 127.0f, 0x1p-126f) : __builtin_nanf("");
    if (t == 0) p.scale[blockIdx.x] = s;
    __attribute__((address_space(1))) uint8_t *q = (__attribute__((address_space(1))) uint8_t *)p.q + uint64_t(blockIdx.x) * uint64_t(p.q_stride);
    const auto put = [&](uint32_t first, const vec16 &v) {
        if (first < p.dim) put_quotients<DT>(q + first, v, s, p.dim - first);
    };
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) put((t + i * kQuantThreads) * E, held[i]);
    } else {
        for (uint32_t at = t * 16; at < bytes; at += kQuantThreads * 16) put(at / ES, row_bytes<ES>(row, at, bytes));
    }
}

template <int OT>
__device__ __forceinline__ void put_out(uint8_t *to, const float (&x)[8], uint32_t n) {
    typedef __attribute__((address_space(1))) uint16_t gu16_out;
    typedef __attribute__((address_space(1))) float gf_out;
    if constexpr (OT == ROG_DTYPE_F32) {
        if (n >= 8) {
            vec16 v[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = f32_bits(x[i]);
            ((gvec16any_out *)to)[0] = v[0];     // at any alignment
            ((gvec16any_out *)to)[1] = v[1];
            return;
        }
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (i < n) ((gf_out *)to)[i] = x[i];
    } else {
        vec16 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = narrow_word<OT>(x + 2 * i);
        if (n >= 8) {
            *(gvec16any_out *)to = v;
            return;
        }
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (i < n) ((gu16_out *)to)[i] = uint16_t(v[i / 2] >> (16 * (i % 2)));
    }
}

// The tile of F's size at columns v0 of shard r and rows n0.
template <int OT, class F, bool DIRECT>
__device__ __forceinline__ void i8_tile(const LinearI8Args &p, uint32_t r, uint32_t v0, uint32_t n0, const TileMemory &memory) {
    constexpr int FM = F::kFM, FN = F::kFN;
    typedef RowProduct<kTypeI8, F, DIRECT, 1, F::kWide> Product;
    const WeightShard sh = p.sh.s[r];
    const uint32_t rows = p.a.rows;
    typename Product::A a(static_cast<const uint8_t *>(sh.w) + uint64_t(v0) * uint64_t(sh.stride), sh.stride, sh.width - v0, p.a.kbytes);
    typename Product::B b(static_cast<const uint8_t *>(p.a.x) + uint64_t(n0) * uint64_t(p.a.stride), p.a.stride, rows - n0, p.a.kbytes);
    const uint32_t wave = threadIdx.x / 64, l = threadIdx.x % 64;
    const uint32_t m0 = wave / F::kWN * (FM * 16), w0 = wave % F::kWN * (FN * 16);
    i32x4 acc[FM][FN] = {};
    Product::run(a, b, p.a.kbytes, m0, w0, memory, acc);

    constexpr uint32_t OS = Logit<OT>::kSize, LEAVES = FM / 2;
    const uint32_t v = v0 + m0 + l / 16 * 8;
    float scale[LEAVES][8];
#pragma unroll
    for (uint32_t f = 0; f < LEAVES; ++f)
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) scale[f][i] = v + 32 * f + i < sh.width ? p.scale[r][v + 32 * f + i] : 0.0f;
    // a row's leaves one after the other, so that its lines are whole before they leave the cache
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t n = n0 + w0 + 16 * j + l % 16;
        if (n >= rows) continue;
        const float s = p.row_scale[n];
        uint8_t *out = static_cast<uint8_t *>(p.out[r]) + uint64_t(n) * uint64_t(p.out_stride[r]) + uint64_t(v) * OS;
#pragma unroll
        for (uint32_t f = 0; f < LEAVES; ++f) {
            if (v + 32 * f >= sh.width) continue;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = float(acc[2 * f + i / 4][j][i % 4]) * s * scale[f][i];
            put_out<OT>(out + 32 * f * OS, x, sh.width - v - 32 * f);
        }
    }
}

// The product, its scales and one rounding to the output.  Many rows: 4093 x 50257 x 5120 to binary16 1.00-1.03 ms, 2060 TOP/s
// (a large library product of 8-bit integers reaches 2339), of which the main loop alone runs at 2870 and the rest are 411 MB
// of outputs, written between a tile's product and the next one's: by leaves of all rows instead of by rows, a line
// was evicted before it was whole, 775 MB and 1.10 ms.  Few rows are bound by the weights' bytes (48 x 131072 x 4096:
// 107-118 us, 4.6-5.2 TB/s; one row of 32000 x 2048 13.6 us, 4.8 TB/s).
template <int OT, class F, bool DIRECT>
__global__ __launch_bounds__(F::kThreads, F::kWide ? 2 : 1) void rog_linear_i8_kernel(LinearI8Args p) {
    typedef RowProduct<kTypeI8, F, DIRECT, 1, F::kWide> Product;
    constexpr uint32_t BM = F::kColumns, BN = F::kRows;
    ROG_TILE_MEMORY(F::kStages, Product::A::kBytes, Product::B::kBytes);
    const uint32_t tm = p.sh.tile0[p.sh.W], tn = (p.a.rows + BN - 1) / BN;
    if constexpr (F::kTail) {
        const Place o = place_of(blockIdx.x, tm, tn);
        if (o.none) return;
        const uint32_t r = shard_of_tile(p.sh, o.at.m), v0 = (o.at.m - p.sh.tile0[r]) * BM, n0 = o.at.n * BN;
        if (o.quarter == 4) {
            i8_tile<OT, F, DIRECT>(p, r, v0, n0, memory);
        } else {
            const uint32_t v = v0 + o.quarter % 2 * FormQuarter::kColumns, n = n0 + o.quarter / 2 * FormQuarter::kRows;
            if (v < p.sh.s[r].width && n < p.a.rows) i8_tile<OT, FormQuarter, DIRECT>(p, r, v, n, memory);
        }
    } else {
        const TileAt at = tile_at(blockIdx.x, tm, tn);
        const uint32_t r = shard_of_tile(p.sh, at.m);
        i8_tile<OT, F, DIRECT>(p, r, (at.m - p.sh.tile0[r]) * BM, at.n * BN, memory);
    }
}

template <int DT>
hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s) {
    const bool held = uint64_t(a.dim) * Logit<DT>::kSize <= kHeld * kQuantThreads * 16;
    return held ? launch(rog_quantize_kernel<DT, true>, a.rows, kQuantThreads, a, s) : launch(rog_quantize_kernel<DT, false>, a.rows, kQuantThreads, a, s);
}

template <int OT, bool DIRECT>
hipError_t launch_i8(const LinearI8Plan &p, hipStream_t s) {
    switch (p.form) {
    case kFormWide: return launch(rog_linear_i8_kernel<OT, FormWide, DIRECT>, p.grid, FormWide::kThreads, p.args, s);
    case kFormMid: return launch(rog_linear_i8_kernel<OT, FormMid, DIRECT>, p.grid, FormMid::kThreads, p.args, s);
    case kFormSome: return launch(rog_linear_i8_kernel<OT, FormSome, DIRECT>, p.grid, FormSome::kThreads, p.args, s);
    default: return launch(rog_linear_i8_kernel<OT, FormFewDeep, DIRECT>, p.grid, FormFewDeep::kThreads, p.args, s);
    }
}
template <int OT>
hipError_t launch_i8(const LinearI8Plan &p, hipStream_t s) {
    return p.direct ? launch_i8<OT, true>(p, s) : launch_i8<OT, false>(p, s);
}

}  // namespace
}  // namespace rog

extern "C" {

ROG_API rog_status rog_quantize_i8(const void *x, int64_t row_stride, size_t rows, int64_t dim, rog_dtype dtype, int8_t *q,
                                   int64_t q_stride, float *scale, hipStream_t stream) {
    using namespace rog;
    QuantizeArgs a;
    const rog_status st = plan_quantize(x, row_stride, rows, dim, dtype, q, q_stride, scale, &a);
    if (st != ROG_OK || rows == 0) return st;
    switch (dtype) {
    case ROG_DTYPE_BF16: return launched(launch_quantize<ROG_DTYPE_BF16>(a, stream));
    case ROG_DTYPE_F16: return launched(launch_quantize<ROG_DTYPE_F16>(a, stream));
    default: return launched(launch_quantize<ROG_DTYPE_F32>(a, stream));
    }
}

ROG_API rog_status rog_linear_i8(const int8_t *q, int64_t q_stride, const float *scale, size_t rows, int64_t dim,
                                 const rog_i8_shard *shards, int W, rog_dtype out_dtype, const rog_grad_shard *out, hipStream_t stream) {
    using namespace rog;
    LinearI8Plan p;
    const rog_status st = plan_linear_i8(q, q_stride, scale, rows, dim, shards, W, out_dtype, out, &p);
    if (st != ROG_OK || p.grid == 0) return st;
    switch (out_dtype) {
    case ROG_DTYPE_BF16: return launched(launch_i8<ROG_DTYPE_BF16>(p, stream));
    case ROG_DTYPE_F16: return launched(launch_i8<ROG_DTYPE_F16>(p, stream));
    default: return launched(launch_i8<ROG_DTYPE_F32>(p, stream));
    }
}

}  // extern "C"
