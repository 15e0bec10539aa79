// rog_linear_score.hip -- HIP kernels of token log probabilities from hidden
// states for gfx950 (CDNA4), and the C entry point that launches them.
//
// x_ij = h_i . w_j over K, z = x / T; per row lse, entropy and the log
// probability of one token, with no logit ever written: a tile's logits stay in
// the accumulators, where each leaf of 32 columns gives the state
//     m = max x log2(e) / T,  s = sum 2^{x log2(e) / T - m},  t = sum 2^{..} (..)
// of its columns, and the leaves' states are joined over one tree.
#include <hip/hip_runtime.h>

#include "rog_linear_device.h"

namespace rog {
namespace {

#pragma clang fp contract(off)

// Joined states of some columns, in the log2 domain.  No columns (or all at -inf): m = -inf, s = t = 0.
struct Part {
    float m, s, t;
};
constexpr float kFar = -1000.0f;   // 2^kFar is 0, and 0 times it is 0
// A state's m is rounded, and its terms' exponents x log2(e) / T - m take the rest of that along, up to 2^(e - 25) of
// |m| = 2^e either way: s is then off by as much and m + log2 s is right.  From here on the rest would leave exponents' range,
// so x log2(e) / T is rounded as m is before the difference.  (Columns masked by -10^10 to -10^38 were NaN without.)
constexpr float kHuge = 1073741824.0f;

__device__ __forceinline__ float base_of(float m) { return m == -kInf ? 0.0f : m; }

__device__ __forceinline__ Part join(const Part &a, const Part &b) {
    const float m = max_nan(a.m, b.m), at = base_of(m);
    const float da = fmaxf(a.m - at, kFar), db = fmaxf(b.m - at, kFar);
    const float fa = exp2_fast(a.m - at), fb = exp2_fast(b.m - at);
    Part o;
    o.m = m;
    o.s = __builtin_fmaf(a.s, fa, b.s * fb);
    o.t = __builtin_fmaf(__builtin_fmaf(a.s, da, a.t), fa, __builtin_fmaf(b.s, db, b.t) * fb);
    return o;
}

// The largest of a leaf's logits, of which each lane holds eight: lanes 16, 32 and 48 on hold the rest.
__device__ __forceinline__ float largest_of(const float (&x)[8]) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = max_nan(top, x[i]);
    Halves h = halves32(top, top);
    top = max_nan(h.first, h.second);
    h = halves16(top, top);
    return max_nan(h.first, h.second);
}

// x log2(e) / T - m; HUGE: m may be huge.
template <bool HUGE>
__device__ __forceinline__ float beyond(float x, float scale, float m) {
    const float d = __builtin_fmaf(x, scale, -m);
    return HUGE && fabsf(m) >= kHuge ? x * scale - m : d;
}

// s and t of the lane's eight logits about the leaf's m.
template <bool HUGE>
__device__ __forceinline__ void sums_of(const float (&x)[8], float scale, float m, float &s, float &t) {
    const float at = base_of(m);
    float e[8], u[4];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float d0 = beyond<HUGE>(x[i], scale, at), d1 = beyond<HUGE>(x[i + 1], scale, at);
        e[i] = exp2_fast(d0);
        e[i + 1] = exp2_fast(d1);
        u[i / 2] = __builtin_fmaf(e[i + 1], fmaxf(d1, kFar), e[i] * fmaxf(d0, kFar));
    }
    s = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    t = (u[0] + u[1]) + (u[2] + u[3]);
}

// The sum over the four lanes that hold a leaf.
__device__ __forceinline__ float leaf_sum(float v) {
    Halves h = halves32(v, v);
    v = h.first + h.second;
    h = halves16(v, v);
    return h.first + h.second;
}
// The same of four leaves: quarters 0, 2, 1, 3 of the wave get leaf 0, 1, 2, 3.
__device__ __forceinline__ float leaf_sums(const float (&v)[4]) {
    Halves h = halves32(v[0], v[1]);
    const float a = h.first + h.second;
    h = halves32(v[2], v[3]);
    const float b = h.first + h.second;
    h = halves16(a, b);
    return h.first + h.second;
}

// The joined state of LEAVES consecutive leaves (1, 2 or 4), the same in all lanes that hold a row.
template <int LEAVES>
__device__ __forceinline__ Part leaves_of(const float (&x)[LEAVES][8], float scale) {
    float m[LEAVES], s[LEAVES], t[LEAVES], most = 0;
#pragma unroll
    for (int f = 0; f < LEAVES; ++f) {
        m[f] = largest_of(x[f]) * scale;
        most = fmaxf(most, fabsf(m[f]));
    }
    if (__ballot(most >= kHuge)) {     // also where a leaf has no columns
#pragma unroll
        for (int f = 0; f < LEAVES; ++f) sums_of<true>(x[f], scale, m[f], s[f], t[f]);
    } else {
#pragma unroll
        for (int f = 0; f < LEAVES; ++f) sums_of<false>(x[f], scale, m[f], s[f], t[f]);
    }
    if constexpr (LEAVES == 4) {
        // a leaf in each quarter, joined across them
        const uint32_t quarter = threadIdx.x / 16 % 4;
        Part p = {quarter & 2 ? (quarter & 1 ? m[3] : m[1]) : (quarter & 1 ? m[2] : m[0]), leaf_sums(s), leaf_sums(t)};
        Halves hm = halves32(p.m, p.m), hs = halves32(p.s, p.s), ht = halves32(p.t, p.t);
        p = join(Part{hm.first, hs.first, ht.first}, Part{hm.second, hs.second, ht.second});
        hm = halves16(p.m, p.m), hs = halves16(p.s, p.s), ht = halves16(p.t, p.t);
        return join(Part{hm.first, hs.first, ht.first}, Part{hm.second, hs.second, ht.second});
    } else {
        Part p = {m[0], leaf_sum(s[0]), leaf_sum(t[0])};
        if constexpr (LEAVES == 2) p = join(p, Part{m[1], leaf_sum(s[1]), leaf_sum(t[1])});
        return p;
    }
}

__device__ __forceinline__ void put_part(float *states, uint64_t at, const Part &p, uint32_t more = 0) {
    typedef __attribute__((address_space(1))) f32x4 gstate;
    *((gstate *)states + at) = f32x4{p.m, p.s, p.t, bits_f32(more)};
}

// The tile of F's size at columns v0 of shard r and rows n0.
template <int DT, class F, bool DIRECT>
__device__ __forceinline__ void score_tile(const ScoreArgs &p, uint32_t r, uint32_t v0, uint32_t n0, uint32_t rows, const TileMemory &memory,
                                           uint32_t *targets, Part *shared_parts, Part *shared_rests) {
    constexpr int BM = F::kColumns, BN = F::kRows, FM = F::kFM, FN = F::kFN, LEAVES = FM / 2;
    typedef RowProduct<DT, F, DIRECT, 2, F::kWide> Product;
    const WeightShard sh = p.sh.s[r];
    typename Product::A a(static_cast<const uint8_t *>(sh.w) + uint64_t(v0) * uint64_t(sh.stride), sh.stride, sh.width - v0, p.a.kbytes);
    typename Product::B b(static_cast<const uint8_t *>(p.a.x) + uint64_t(n0) * uint64_t(p.a.stride), p.a.stride, rows - n0, p.a.kbytes);
    const uint32_t wave = threadIdx.x / 64, l = threadIdx.x % 64;
    const uint32_t m0 = wave / F::kWN * (FM * 16), w0 = wave % F::kWN * (FN * 16);
    // the rows' tokens as columns of the tile, all others past it
    if (threadIdx.x < BN) {
        const uint32_t n = n0 + threadIdx.x;
        const int64_t tok = p.tokens && n < rows ? p.tokens[p.index ? p.index[n] : n] - int64_t(sh.col0) - int64_t(v0) : -1;
        targets[threadIdx.x] = tok >= 0 && tok < BM && uint32_t(tok) + v0 < sh.width ? uint32_t(tok) : 1u << 30;
    }
    typename Mat<DT>::Acc acc[FM][FN] = {};
    Product::run(a, b, p.a.kbytes, m0, w0, memory, acc);

    // lane l holds columns v0 + m0 + 32 f + 8 (l / 16) + 0 .. 7 of leaf f, row n0 + w0 + 16 j + l % 16
    const uint32_t own = 8 * (l / 16);
    if (v0 + m0 + FM * 16 > sh.width) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v0 + m0 + 32 * (f / 2) + own + 4 * (f % 2) + i >= sh.width)
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[f][j][i] = -kInf;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t n = n0 + w0 + 16 * j + l % 16;
        // the row's token among the wave's columns
        const uint32_t hit = targets[w0 + 16 * j + l % 16] - m0;
        float x[LEAVES][8];
#pragma unroll
        for (int c = 0; c < FM * 4; ++c) x[c / 8][c % 8] = acc[c / 4][j][c % 4];
        const Part part = leaves_of<LEAVES>(x, p.scale);
        Part rest = part;              // the same without the token, where it is among them
        if (__ballot(hit < FM * 16)) {
#pragma unroll
            for (uint32_t c = 0; c < FM * 4; ++c)
                if (hit == 32 * (c / 8) + own + c % 8) {
                    p.target[n] = x[c / 8][c % 8];
                    x[c / 8][c % 8] = -kInf;
                }
            rest = leaves_of<LEAVES>(x, p.scale);
        }
        if constexpr (F::kShare == 1) {
            const uint32_t block = p.sh.block0[r] + (v0 + m0) / kLinearBlock;
            if (l < 16 && n < rows && block < p.sh.block0[r + 1]) {
                put_part(p.states, uint64_t(n) * p.row_step + uint64_t(block) * p.block_step, part);
                if (hit < FM * 16) put_part(p.rests, n, rest, block);
            }
        } else if (l < 16) {
            shared_parts[m0 / (FM * 16) * BN + w0 + 16 * j + l] = part;
            shared_rests[m0 / (FM * 16) * BN + w0 + 16 * j + l] = rest;
        }
    }
    if constexpr (F::kShare > 1) {
        // the waves of a block join their leaves; a tile has one block
        static_assert(BM == int(kLinearBlock), "one block");
        __syncthreads();
        const uint32_t n = n0 + threadIdx.x;
        if (threadIdx.x < BN && n < rows) {
            const auto joined = [&](const Part *of) {
                of += threadIdx.x;
                const Part all = join(of[0], of[BN]);
                return F::kShare == 4 ? join(all, join(of[2 * BN], of[3 * BN])) : all;
            };
            const uint32_t block = p.sh.block0[r] + v0 / kLinearBlock;
            put_part(p.states, uint64_t(n) * p.row_step + uint64_t(block) * p.block_step, joined(shared_parts));
            if (targets[threadIdx.x] < BM) put_part(p.rests, n, joined(shared_rests), block);
        }
    }
}

// The product and the states of its tiles.  Many rows are bound by the matrix units (8192 x 131072 x 4096 bf16, 7173 of them scored:
// 5.6-5.8 ms, 1340-1380 TFLOP/s; the product alone 1520, what a large library product reaches here at the 1.76 GHz
// that its power allows; the states' arithmetic is the rest, eight vector instructions and an exp2 per logit between
// two tiles), few rows by the weights' bytes (64 x 131072 x 4096: 178 us, 6.1 TB/s).  Logits are binary32 sums and
// never rounded to fewer bits.
template <int DT, class F, bool DIRECT>
__global__ __launch_bounds__(F::kThreads, F::kWide ? 2 : 1) void rog_linear_score_kernel(ScoreArgs p) {
    typedef RowProduct<DT, F, DIRECT, 2, F::kWide> Product;
    constexpr uint32_t BM = F::kColumns, BN = F::kRows;
    ROG_TILE_MEMORY(F::kStages, Product::A::kBytes, Product::B::kBytes);
    __shared__ uint32_t targets[BN];
    constexpr uint32_t kParts = F::kTail ? FormQuarter::kShare * FormQuarter::kRows : F::kShare > 1 ? F::kShare * BN : 1;
    __shared__ Part parts[kParts], rests[kParts];
    const uint32_t rows = uniform(p.a.count ? *p.a.count : p.a.rows), tm = p.sh.tile0[p.sh.W], tn = (rows + BN - 1) / BN;
    if constexpr (F::kTail) {
        const Place o = place_of(blockIdx.x, tm, tn);
        if (o.none) return;
        const uint32_t r = shard_of_tile(p.sh, o.at.m), v0 = (o.at.m - p.sh.tile0[r]) * BM, n0 = o.at.n * BN;
        if (o.quarter == 4) {
            score_tile<DT, F, DIRECT>(p, r, v0, n0, rows, memory, targets, parts, rests);
        } else {
            const uint32_t v = v0 + o.quarter % 2 * FormQuarter::kColumns, n = n0 + o.quarter / 2 * FormQuarter::kRows;
            if (v < p.sh.s[r].width && n < rows) score_tile<DT, FormQuarter, DIRECT>(p, r, v, n, rows, memory, targets, parts, rests);
        }
    } else {
        if (blockIdx.x >= tm * tn) return;
        const TileAt at = tile_at(blockIdx.x, tm, tn);
        const uint32_t r = shard_of_tile(p.sh, at.m);
        score_tile<DT, F, DIRECT>(p, r, (at.m - p.sh.tile0[r]) * BM, at.n * BN, rows, memory, targets, parts, rests);
    }
}

// The log probability of a token of logit x beside the others: -log(1 + R), R = sum over them of 2^{(x_j - x) scale}.  A token
// that is nearly sure keeps its digits so (of 1 - p = 10^-4 the sum of all terms holds three).
__device__ __forceinline__ float sure_of(float x, float scale, const Part &rest) {
    if (rest.m == -kInf) return x == -kInf ? -kInf : 0.0f;
    const float d = beyond<true>(x, scale, rest.m);          // exact but for one rounding
    return d > -60.0f ? -log1pf(rest.s * exp2f(-d)) : (d - log2f(rest.s)) * kLn2;
}

// Joins a row's blocks: chunk c of 64 takes every 64th block from the c-th on, one
// after the other, and the chunks are joined in pairs 32, 16, .. 1 apart.  With
// ROWS 1 a wave has a row, its lanes the chunks; with 16 a workgroup has 16 rows
// whose states of a block stand together.  Bound by the chain of its loads, four of which are in flight at a time:
// 1 x 32003 3.8 us, 64 x 131072 8.5, 8192 x 131072 26 (118 MB, 4.5 TB/s).
constexpr uint32_t kJoinWide = 16;
template <uint32_t ROWS>
__global__ __launch_bounds__(ROWS == 1 ? 256 : 64 * ROWS) void rog_linear_join_kernel(JoinArgs p) {
    constexpr uint32_t THREADS = ROWS == 1 ? 256 : 64 * ROWS, EACH = ROWS == 1 ? 4 : ROWS, DEEP = 4;
    __shared__ Part others[ROWS == 1 ? 1 : THREADS], other_rests[ROWS == 1 ? 1 : THREADS];
    typedef const __attribute__((address_space(1))) f32x4 gstate;
    const uint32_t rows = p.count ? *p.count : p.rows, chunk = ROWS == 1 ? threadIdx.x % 64 : threadIdx.x / ROWS;
    const uint32_t n = blockIdx.x * EACH + (ROWS == 1 ? threadIdx.x / 64 : threadIdx.x % ROWS);
    if (blockIdx.x * EACH >= rows) return;
    // all of the row's columns, and all but its token
    Part all = {-kInf, 0, 0}, rest = all;
    uint32_t row = 0;
    int64_t tok = 0;
    if (n < rows) {
        row = p.index ? p.index[n] : n;
        tok = p.tokens ? p.tokens[row] : 0;
        const f32x4 cut = ((gstate *)p.rests)[n];      // of no meaning where there is no such token
        const uint32_t cut_block = p.logp && tok >= 0 && tok < int64_t(p.vocab) ? f32_bits(cut[3]) : 0xFFFFFFFFu;
        gstate *from = (gstate *)p.states + uint64_t(n) * p.row_step;
        // a few blocks' loads at a time; past the last an empty state, which changes nothing
        for (uint32_t b = chunk; b < p.blocks; b += 64 * DEEP) {
            f32x4 v[DEEP];
#pragma unroll
            for (uint32_t i = 0; i < DEEP; ++i) v[i] = b + 64 * i < p.blocks ? from[uint64_t(b + 64 * i) * p.block_step] : f32x4{-kInf, 0, 0, 0};
#pragma unroll
            for (uint32_t i = 0; i < DEEP; ++i) {
                all = join(all, Part{v[i][0], v[i][1], v[i][2]});
                if (b + 64 * i == cut_block) v[i] = cut;
                rest = join(rest, Part{v[i][0], v[i][1], v[i][2]});
            }
        }
    }
    for (uint32_t d = 32; d; d /= 2) {
        if constexpr (ROWS == 1) {
            all = join(all, Part{__shfl_xor(all.m, d), __shfl_xor(all.s, d), __shfl_xor(all.t, d)});
            rest = join(rest, Part{__shfl_xor(rest.m, d), __shfl_xor(rest.s, d), __shfl_xor(rest.t, d)});
        } else {
            __syncthreads();
            if (chunk >= d && chunk < 2 * d) {
                others[threadIdx.x] = all;
                other_rests[threadIdx.x] = rest;
            }
            __syncthreads();
            if (chunk < d) {
                all = join(all, others[threadIdx.x + d * ROWS]);
                rest = join(rest, other_rests[threadIdx.x + d * ROWS]);
            }
        }
    }
    if (chunk || n >= rows) return;
    float logp = 0, entropy = 0, lse = 0;
    if (tok >= 0) {
        const float log_s = log2f(all.s);
        const bool empty = all.m == -kInf, bad = !(all.s == all.s) || all.m == kInf;   // of a NaN, of +inf (also by the scale)
        const float nan = __builtin_nanf("");
        lse = bad ? nan : empty ? -kInf : (all.m + log_s) * kLn2;
        entropy = bad ? nan : empty ? 0.0f : fmaxf(0.0f, (log_s - all.t / all.s) * kLn2);
        if (p.logp) logp = bad || tok >= int64_t(p.vocab) ? nan : empty ? -kInf : sure_of(p.target[n], p.scale, rest);
    }
    if (p.logp) p.logp[row] = logp;
    if (p.entropy) p.entropy[row] = entropy;
    if (p.lse) p.lse[row] = lse;
}

// Packs the scored rows in their order: a workgroup counts those before its ROWS rows, then its waves copy them.  No
// workgroup waits for another, so the tokens are read anew by each (8192 rows of 4096: 25 us for 59 MB each way, 1021
// of 1600 6.6).
constexpr uint32_t kPackThreads = 256;
template <uint32_t ROWS>
__global__ __launch_bounds__(kPackThreads) void rog_linear_pack_kernel(PackArgs p) {
    constexpr uint32_t WAVES = kPackThreads / 64;
    __shared__ uint32_t sums[WAVES];
    __shared__ float most[WAVES];
    const uint32_t row0 = blockIdx.x * ROWS, t = threadIdx.x, wave = t / 64, l = t % 64;
    uint32_t before = 0;
    for (uint32_t i = t; i < row0; i += kPackThreads) before += p.tokens[i] >= 0;
    const uint64_t own = __ballot(l < ROWS && row0 + l < p.rows && p.tokens[row0 + l] >= 0);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) before += __shfl_xor(before, d);
    if (l == 0) sums[wave] = before;
    __syncthreads();
    before = 0;
    for (uint32_t i = 0; i < WAVES; ++i) before += sums[i];
    for (uint32_t i = wave; i < ROWS && row0 + i < p.rows; i += WAVES) {
        const uint32_t row = row0 + i;
        if (own >> i & 1) {
            const uint32_t at_row = before + uint32_t(__popcll(own & ((uint64_t(1) << i) - 1)));
            gbyte *from = (gbyte *)p.x + uint64_t(row) * uint64_t(p.stride);
            __attribute__((address_space(1))) uint8_t *to =
                (__attribute__((address_space(1))) uint8_t *)p.packed + uint64_t(at_row) * p.packed_bytes;
            for (uint32_t at = l * 16; at < p.packed_bytes; at += 4096) {
                vec16 v[4];
#pragma unroll
                for (uint32_t u = 0; u < 4; ++u) v[u] = row_bytes<2>(from, at + u * 1024, p.kbytes);
#pragma unroll
                for (uint32_t u = 0; u < 4; ++u)
                    if (at + u * 1024 < p.packed_bytes) *(gvec16any_out *)(to + at + u * 1024) = v[u];
            }
            if (l == 0) p.index[at_row] = row;
        } else {
            if (p.zero) {
                __attribute__((address_space(1))) uint8_t *to =
                    (__attribute__((address_space(1))) uint8_t *)p.zero + uint64_t(row) * uint64_t(p.zero_stride);
                const uint32_t whole = p.kbytes & ~15u;
                for (uint32_t at = l * 16; at < whole; at += 1024) *(gvec16any_out *)(to + at) = vec16any{0, 0, 0, 0};
                if (whole + l * 2 < p.kbytes) *(__attribute__((address_space(1))) uint16_t *)(to + whole + l * 2) = 0;
            }
            if (l == 0) {
                if (p.logp) p.logp[row] = 0;
                if (p.entropy) p.entropy[row] = 0;
                if (p.lse) p.lse[row] = 0;
            }
        }
    }
    before += uint32_t(__popcll(own));
    if (t == 0 && row0 + ROWS >= p.rows) {
        *p.count = before;
        if (p.parts) *p.parts = weight_parts(before, p.dim_tiles, p.tiles, p.seg_tiles);
    }
    if (!p.g_scale || blockIdx.x) return;
    // one scale of all rows' coefficients, for the products that sum over rows
    float m = 0;
    for (uint32_t i = t; i < p.rows; i += kPackThreads)
        if (p.tokens[i] >= 0)
            m = fmaxf(m, most_of(p.g_logp[i], p.g_entropy ? p.g_entropy[i] : 0.0f, p.inv_t));
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (l == 0) most[wave] = m;
    __syncthreads();
    if (t == 0) {
        for (uint32_t i = 1; i < kPackThreads / 64; ++i) m = fmaxf(m, most[i]);
        *p.g_scale = power_for(m);
    }
}

constexpr float kLog2E = 1.44269504088896341f;

// What a row's coefficients are made of: G = 2^y (c0 + c1 y) with y = x log2(e) / T - at, and g more at the token.
struct RowOf {
    float at, c0, c1, g;
    float uniform;                     // y where the row is uniform over its largest logits: -entropy log2(e)
    float again;                       // binary16: from the row's scale to that of all rows
    uint32_t target;                   // the token as a column of the tile, else past it
};
// |at| from which lse's rounding is looked after, up to 4.5 half steps of it (m's, its sum's with log2 s, three products with
// ln 2 and log2(e)) and what log2 s and the entropy leave: a row that is uniform over its largest logits (sure of one
// token, or masked as a whole) has y = -entropy log2(e) at each of them, so a y that lies within the rounding of that is
// taken to be that, and p is at most 1.  Any other y that happens to lie there moves by less than one more rounding of lse.
constexpr float kLarge = 16384.0f;
__device__ __forceinline__ float settled(float y, float at, float uniform) {
    const bool near = fabsf(y - uniform) <= __builtin_fmaf(fabsf(at), 4.5f * 0x1p-24f, 0x1p-15f);
    return !(fabsf(at) >= kLarge) || at == kInf ? y : near ? uniform : y > 0.0f ? 0.0f : y;
}

template <int DT>
__device__ __forceinline__ RowOf coef_row(const GradArgs &p, uint32_t row, int64_t first, uint32_t columns) {
    const int64_t tok = p.tokens[row];
    const float lse = p.lse[row], h = p.entropy[row];
    float g = p.g_logp[row], gh = p.g_entropy ? p.g_entropy[row] : 0.0f;
    RowOf r;
    // binary16: one copy by a scale of the row's own for d_hidden, one by that of all rows for d_weights
    const float by = DT == ROG_DTYPE_F16 ? power_for(most_of(g, gh, p.inv_t)) : 1.0f;
    r.again = DT == ROG_DTYPE_F16 ? *p.g_scale / by : 1.0f;
    g *= p.inv_t * by;
    gh *= p.inv_t * by;
    if (tok >= int64_t(p.sh.vocab)) g = __builtin_nanf("");
    const bool empty = lse == -kInf;
    if (empty) g = gh = 0.0f;
    r.at = empty ? kInf : lse * kLog2E;
    r.c0 = -__builtin_fmaf(gh, h, g);
    r.c1 = -gh * kLn2;
    r.g = g;
    r.uniform = -h * kLog2E;
    r.target = tok >= first && tok - first < int64_t(columns) ? uint32_t(tok - first) : 1u << 30;
    return r;
}

// The tile of F's size at columns v0 of shard r, which are columns g0 of the piece, and rows n0.  G is rounded to the
// weights' type here, the type that the matrix units take: held in two parts, which would keep 16 bits of it in
// bf16 and 22 in binary16, both products behind it would take twice the instructions, 10 N V D operations in all instead of
// 6, and G's memory and traffic double.  Rounded once it is off by half a step, as the outputs are by theirs (errors against
// 64 bits 2.4-2.7e-3 of the norm in bf16 and 3e-4 in binary16; of binary32 coefficients, with the output's rounding
// alone, 1.7e-3 and 2.1e-4).  Calls of few rows have the same coefficients, so that a row's bits do not depend on how many
// there are.
template <int DT, class F, bool DIRECT>
__device__ __forceinline__ void coef_tile(const GradArgs &p, uint32_t r, uint32_t v0, uint32_t g0, uint32_t n0, uint32_t rows,
                                          const TileMemory &memory, RowOf *row_of) {
    constexpr int BM = F::kColumns, BN = F::kRows, FM = F::kFM, FN = F::kFN, LEAVES = FM / 2;
    typedef RowProduct<DT, F, DIRECT, 2, F::kWide> Product;
    const WeightShard sh = p.sh.s[r];
    if (v0 >= sh.width || n0 >= rows) return;        // nobody reads the coefficients of such a part
    typename Product::A a(static_cast<const uint8_t *>(sh.w) + uint64_t(v0) * uint64_t(sh.stride), sh.stride, sh.width - v0, p.a.kbytes);
    typename Product::B b(static_cast<const uint8_t *>(p.a.x) + uint64_t(n0) * uint64_t(p.a.stride), p.a.stride, rows - n0, p.a.kbytes);
    const uint32_t wave = threadIdx.x / 64, l = threadIdx.x % 64;
    const uint32_t m0 = wave / F::kWN * (FM * 16), w0 = wave % F::kWN * (FN * 16);
    if (threadIdx.x < BN && n0 + threadIdx.x < rows) row_of[threadIdx.x] = coef_row<DT>(p, p.index[n0 + threadIdx.x], int64_t(sh.col0) + v0, BM);
    typename Mat<DT>::Acc acc[FM][FN] = {};
    Product::run(a, b, p.a.kbytes, m0, w0, memory, acc);

    const float scale = p.scale;       // that of the log probabilities
    const uint32_t own = 8 * (l / 16);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t n = n0 + w0 + 16 * j + l % 16;
        const RowOf row = row_of[w0 + 16 * j + l % 16];
        const uint32_t hit = row.target - m0;
        const bool hits = __ballot(hit < FM * 16) != 0, large = __ballot(fabsf(row.at) >= kLarge) != 0;
#pragma unroll
        for (int f = 0; f < LEAVES; ++f) {
            float d[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) d[i] = __builtin_fmaf(acc[2 * f + i / 4][j][i % 4], scale, -row.at);
            if (large)
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) d[i] = settled(d[i], row.at, row.uniform);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) d[i] = exp2_fast(d[i]) * __builtin_fmaf(row.c1, fmaxf(d[i], kFar), row.c0);
            if (hits)
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i)
                    if (hit == 32 * f + own + i) d[i] += row.g;
            if (v0 + m0 + 32 * f + 32 > sh.width)
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i)
                    if (v0 + m0 + 32 * f + own + i >= sh.width) d[i] = 0.0f;
            if (n >= rows) continue;
            vec16 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = narrow_word<DT>(d + 2 * i);
            typedef __attribute__((address_space(1))) vec16 gvec16_out;
            const uint64_t to = uint64_t(n) * uint64_t(p.g_stride) + (uint64_t(g0) + m0 + own + 32 * f) * 2;
            *(gvec16_out *)((uint8_t *)p.g + to) = v;
            if constexpr (DT == ROG_DTYPE_F16) {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] *= row.again;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = narrow_word<DT>(d + 2 * i);
                *(gvec16_out *)((uint8_t *)p.g_all + to) = v;
            }
        }
    }
}

// The logits of a piece once more, and G of them in place of the states: the same product with one exp2 and a write of two bytes
// (binary16: two of them) per logit.  4096 x 32768 of 4096 bf16, 3584 rows scored: 760 us, 1266 TFLOP/s; 893 x 50257 of 1600 binary16 199 us,
// 721; 33 x 32003 of 1024 14.6 us, 4.6 TB/s of weights.
template <int DT, class F, bool DIRECT>
__global__ __launch_bounds__(F::kThreads, F::kWide ? 2 : 1) void rog_linear_coef_kernel(GradArgs p) {
    typedef RowProduct<DT, F, DIRECT, 2, F::kWide> Product;
    constexpr uint32_t BM = F::kColumns, BN = F::kRows, SPLIT = kGradTile / BM;
    ROG_TILE_MEMORY(F::kStages, Product::A::kBytes, Product::B::kBytes);
    __shared__ RowOf row_of[BN];
    const uint32_t rows = uniform(*p.a.count), tm = p.tiles * SPLIT, tn = (rows + BN - 1) / BN;
    TileAt at;
    uint32_t quarter = 4;
    if constexpr (F::kTail) {
        const Place o = place_of(blockIdx.x, tm, tn);
        if (o.none) return;
        at = o.at;
        quarter = o.quarter;
    } else {
        if (blockIdx.x >= tm * tn) return;
        at = tile_at(blockIdx.x, tm, tn);
    }
    const uint32_t tile = p.tile_begin + at.m / SPLIT, r = shard_of_tile(p.sh, tile);
    const uint32_t v0 = (tile - p.sh.tile0[r]) * kGradTile + at.m % SPLIT * BM;
    if (!F::kTail || quarter == 4) {
        coef_tile<DT, F, DIRECT>(p, r, v0, at.m * BM, at.n * BN, rows, memory, row_of);
    } else if constexpr (F::kTail) {
        const uint32_t m = quarter % 2 * FormQuarter::kColumns, n = quarter / 2 * FormQuarter::kRows;
        coef_tile<DT, FormQuarter, DIRECT>(p, r, v0 + m, at.m * BM + m, at.n * BN + n, rows, memory, row_of);
    }
}

template <int DT, bool DIRECT>
hipError_t launch_score(const ScorePlan &p, hipStream_t s) {
    switch (p.form) {
    case kFormWide: return launch(rog_linear_score_kernel<DT, FormWide, DIRECT>, p.grid, FormWide::kThreads, p.args, s);
    case kFormMid: return launch(rog_linear_score_kernel<DT, FormMid, DIRECT>, p.grid, FormMid::kThreads, p.args, s);
    case kFormSome: return launch(rog_linear_score_kernel<DT, FormSome, DIRECT>, p.grid, FormSome::kThreads, p.args, s);
    default:
        return p.grid <= kCus ? launch(rog_linear_score_kernel<DT, FormFewDeep, DIRECT>, p.grid, FormFewDeep::kThreads, p.args, s)
                              : launch(rog_linear_score_kernel<DT, FormFew, DIRECT>, p.grid, FormFew::kThreads, p.args, s);
    }
}

template <int DT, bool DIRECT>
hipError_t launch_coef(const GradPlan &p, const GradArgs &a, uint32_t grid, hipStream_t s) {
    switch (p.form) {
    case kFormWide: return launch(rog_linear_coef_kernel<DT, FormWide, DIRECT>, grid, FormWide::kThreads, a, s);
    case kFormMid: return launch(rog_linear_coef_kernel<DT, FormMid, DIRECT>, grid, FormMid::kThreads, a, s);
    case kFormSome: return launch(rog_linear_coef_kernel<DT, FormSome, DIRECT>, grid, FormSome::kThreads, a, s);
    default:
        return grid <= kCus ? launch(rog_linear_coef_kernel<DT, FormFewDeep, DIRECT>, grid, FormFewDeep::kThreads, a, s)
                            : launch(rog_linear_coef_kernel<DT, FormFew, DIRECT>, grid, FormFew::kThreads, a, s);
    }
}

}  // namespace

hipError_t launch_pack(const PackArgs &a, hipStream_t s) {
    // every workgroup reads the tokens before its rows: few rows each while there are few tokens
    return a.rows <= 16384 ? launch(rog_linear_pack_kernel<8>, (a.rows + 7) / 8, kPackThreads, a, s)
                           : launch(rog_linear_pack_kernel<64>, (a.rows + 63) / 64, kPackThreads, a, s);
}

hipError_t launch_coefficients(const GradPlan &p, const GradArgs &a, uint32_t grid, hipStream_t s) {
    if (p.dtype == ROG_DTYPE_BF16)
        return p.direct ? launch_coef<ROG_DTYPE_BF16, true>(p, a, grid, s) : launch_coef<ROG_DTYPE_BF16, false>(p, a, grid, s);
    return p.direct ? launch_coef<ROG_DTYPE_F16, true>(p, a, grid, s) : launch_coef<ROG_DTYPE_F16, false>(p, a, grid, s);
}

}  // namespace rog

extern "C" {

ROG_API rog_status rog_linear_logprob(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim,
                                      const rog_weight_shard *shards, int W, rog_dtype dtype, float temperature,
                                      const int64_t *tokens, const rog_logprob_out *out, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    rog::ScorePlan p;
    const rog_status st = rog::plan_linear_logprob(hidden, hidden_stride, rows, dim, shards, W, dtype, temperature, tokens, out,
                                                   workspace, workspace_bytes, true, tokens != nullptr, &p);
    if (st != ROG_OK || rows == 0) return st;
    using namespace rog;
    hipError_t e = hipSuccess;
    if (p.packs) e = launch_pack(p.pack, stream);
    if (e == hipSuccess && p.grid) {
        if (dtype == ROG_DTYPE_BF16) e = p.direct ? launch_score<ROG_DTYPE_BF16, true>(p, stream) : launch_score<ROG_DTYPE_BF16, false>(p, stream);
        else e = p.direct ? launch_score<ROG_DTYPE_F16, true>(p, stream) : launch_score<ROG_DTYPE_F16, false>(p, stream);
    }
    if (e == hipSuccess)
        e = p.form == kFormWide ? launch(rog_linear_join_kernel<kJoinWide>, uint32_t((rows + kJoinWide - 1) / kJoinWide), 64 * kJoinWide, p.join, stream)
                                : launch(rog_linear_join_kernel<1>, uint32_t((rows + 3) / 4), 256, p.join, stream);
    return launched(e);
}

}  // extern "C"
