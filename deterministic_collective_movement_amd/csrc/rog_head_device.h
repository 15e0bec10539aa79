// rog_head_device.h -- device helpers of the vocabulary-side kernels: elements
// of a block of logits in a lane's registers, and the partial states of a
// softmax.
#pragma once

#include "rog_device.h"
#include "rog_head.h"

namespace rog {

// Every multiply-add below is written out: the same expression has to give the
// same bits in every kernel that it is inlined into.
#pragma clang fp contract(off)

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// 16 bytes in the global address space at any byte alignment.
typedef const __attribute__((address_space(1))) uint8_t gbyte;
typedef uint32_t vec16any __attribute__((ext_vector_type(4), aligned(1)));
typedef const __attribute__((address_space(1))) vec16any gvec16any;
typedef __attribute__((address_space(1))) vec16any gvec16any_out;

constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float bits_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// 2^x in one instruction (results below 2^-126 are flushed to zero).
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// The larger of two; NaN if one is NaN (v_maximum3_f32).
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Logits of type DT (a rog_dtype) as the kernels hold them.
template <int DT>
struct Logit {
    static constexpr uint32_t kSize = DT == ROG_DTYPE_F32 ? 4 : 2;
    static constexpr uint32_t kPerVec = 16 / kSize;                         // columns per 16-byte vector
    static constexpr uint32_t kVecs = kHeadBlock / 64 / kPerVec;            // vectors per lane of a block
    static constexpr uint32_t kMinusInf = DT == ROG_DTYPE_F32 ? 0xFF800000u // one or two logits of -inf
                                          : DT == ROG_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
};

// Two 2-byte logits, or one binary32, of a 32-bit word.
template <int DT>
__device__ __forceinline__ void widen_word(uint32_t w, float *x) {
    if constexpr (DT == ROG_DTYPE_BF16) {
        x[0] = bits_f32(w << 16);
        x[1] = bits_f32(w & 0xFFFF0000u);
    } else if constexpr (DT == ROG_DTYPE_F16) {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        x[0] = float(h.x);
        x[1] = float(h.y);
    } else {
        x[0] = bits_f32(w);
    }
}

// Rounds once, nearest-even.
template <int DT>
__device__ __forceinline__ uint32_t narrow_word(const float *x) {
    if constexpr (DT == ROG_DTYPE_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[0], x[1]}, bf16x2));
    else if constexpr (DT == ROG_DTYPE_F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[0], x[1]}, f16x2));
    else return f32_bits(x[0]);
}

template <int DT>
__device__ __forceinline__ void widen_vec(const vec16 &v, float *x) {
    constexpr int n = Logit<DT>::kPerVec / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) widen_word<DT>(v[i], x + n * i);
}

// One logit at an element address.
template <int DT>
__device__ __forceinline__ float load_logit(gbyte *p) {
    if constexpr (DT == ROG_DTYPE_F32) return *(const __attribute__((address_space(1))) float *)p;
    else {
        float x[2];
        widen_word<DT>(*(const __attribute__((address_space(1))) uint16_t *)p, x);
        return x[0];
    }
}

// A block of one row: its first column's address, how many columns it has
// (1..2048) and the number of its first column in the row.
struct BlockAt {
    gbyte *p;
    uint32_t n;
    uint32_t col;
    uint32_t shard;
    uint32_t off;       // the first column's number in the shard
    bool shift;         // a full block of 2-byte logits between two 32-bit words
};

__device__ __forceinline__ uint32_t head_group() { return blockIdx.y << kGridRowLog | blockIdx.x; }

// Has the front of the arguments read in one go, into scalar registers and the
// scalar cache, before anything waits for a part of it.
__device__ __forceinline__ void hold_front(const LogprobArgs &a) {
    asm volatile("" ::"s"(a.tokens), "s"(a.rows), "s"(a.units), "s"(a.scale), "s"(a.bound), "s"(a.lse), "s"(a.part), "s"(a.sh.W),
                 "s"(a.sh.blocks), "s"(a.sh.even), "s"(a.sh.s[0].x), "s"(a.sh.s[0].stride), "s"(a.sh.s[0].width));
}
__device__ __forceinline__ void hold_front(const LogprobGradArgs &a) {
    asm volatile("" ::"s"(a.tokens), "s"(a.lse), "s"(a.entropy), "s"(a.g_logp), "s"(a.g_entropy), "s"(a.inv_t),
                 "s"(a.inv_t_rest), "s"(a.groups), "s"(a.sh.W), "s"(a.sh.blocks), "s"(a.sh.even), "s"(a.sh.s[0].x), "s"(a.sh.s[0].stride),
                 "s"(a.sh.s[0].width));
}

// Walks through one row's blocks (of COLUMNS columns), in rising order: the current shard's layout
// stays in scalar registers, and kernel arguments are read only where a shard
// begins.
template <int DT, uint32_t COLUMNS = kHeadBlock>
struct Cursor {
    const HeadShards &h;
    gbyte *base;                       // the row's first column in the shard
    uint32_t row, shard, first, end;   // blocks [first, end) are the shard's
    uint32_t width, col0;

    __device__ __forceinline__ Cursor(const HeadShards &shards, uint32_t r) : h(shards), row(r), shard(0), end(0) {}
    __device__ __forceinline__ void enter(uint32_t r) {
        const Shard &s = h.s[r];
        shard = r;
        width = s.width;
        col0 = s.col0;
        base = (gbyte *)s.x + int64_t(row) * s.stride;
    }
    // To the shard of block b (below the row's blocks, not before the shard that the cursor is in).
    __device__ __forceinline__ void seek(uint32_t b) {
        if (b >= end) {
            if (h.W == 1) {
                first = 0;
                end = h.blocks;
                enter(0);
            } else if (h.even) {
                const uint32_t r = divide(b, h.even_div);
                first = r * h.even;
                end = first + h.even;
                enter(r);
            } else {
                uint32_t r = shard;
                while (h.block0[r + 1] <= b) ++r;
                first = h.block0[r];
                end = h.block0[r + 1];
                enter(r);
            }
        }
    }
    // The n columns of the shard from off on.
    __device__ __forceinline__ BlockAt columns(uint32_t off, uint32_t n) const {
        gbyte *const p = base + uint64_t(off) * Logit<DT>::kSize;
        const bool shift = DT != ROG_DTYPE_F32 && n == COLUMNS && (reinterpret_cast<uintptr_t>((const uint8_t *)p) & 2) != 0;
        return BlockAt{p, n, col0 + off, shard, off, shift};
    }
    __device__ __forceinline__ BlockAt at(uint32_t b) {
        seek(b);
        const uint32_t off = (b - first) * COLUMNS, left = width - off;
        return columns(off, left < COLUMNS ? left : COLUMNS);
    }
};

// A lane's vector i of a block is columns (64 i + lane) * kPerVec and on.  Where
// that runs past the block's end at n, the vector is read from the last place
// where it fits, n - kPerVec: its first elements are then another lane's
// columns (another's whole vector, where nothing of this one is left).  So a
// tail takes the same loads as a full block, no byte past the row is read, and
// element e belongs to the lane iff place + e >= its own first column.  A block
// of fewer columns than one vector is read element by element.
template <int DT>
__device__ __forceinline__ uint32_t own_column(uint32_t i, uint32_t lane) { return (64 * i + lane) * Logit<DT>::kPerVec; }

template <int DT>
__device__ __forceinline__ uint32_t vec_place(uint32_t n, uint32_t i, uint32_t lane) {
    const uint32_t c = own_column<DT>(i, lane), last = n - Logit<DT>::kPerVec;
    return c < last ? c : last;
}

// The n < kPerVec columns of a tiny block, as every lane's vector (-inf behind them).
template <int DT>
__device__ __forceinline__ vec16 load_tiny(gbyte *p, uint32_t n) {
    vec16 v = {Logit<DT>::kMinusInf, Logit<DT>::kMinusInf, Logit<DT>::kMinusInf, Logit<DT>::kMinusInf};
#pragma unroll
    for (uint32_t e = 0; e + 1 < Logit<DT>::kPerVec; ++e) {
        if (e >= n) continue;
        if constexpr (DT == ROG_DTYPE_F32) {
            v[e] = *(const __attribute__((address_space(1))) uint32_t *)(p + e * 4);
        } else {
            const uint32_t h = *(const __attribute__((address_space(1))) uint16_t *)(p + e * 2);
            v[e / 2] = e & 1 ? (v[e / 2] & 0xFFFFu) | h << 16 : (v[e / 2] & 0xFFFF0000u) | h;
        }
    }
    return v;
}

template <int DT>
__device__ __forceinline__ vec16 load_vec(gbyte *p, uint32_t n, uint32_t i, uint32_t lane) {
    if (n < Logit<DT>::kPerVec) return load_tiny<DT>(p, n);
    return *(gvec16any *)(p + vec_place<DT>(n, i, lane) * Logit<DT>::kSize);
}

// A block's vectors as loaded, and the 32-bit word behind them.
template <uint32_t VECS>
struct Loaded {
    vec16 v[VECS];
    uint32_t behind;
};

// Issues the loads of a block.  They are issued whatever the block, so that no
// branch joins registers that loads are still on their way to: a block of less
// than one vector (read where it is used, tiny_state) reads the first bytes of
// the kernel arguments instead, and with `real` false every lane reads the
// block's first bytes.
//
// 16-byte loads at odd multiples of two bytes are slow (4000 x 100003 bf16,
// where every other row begins so: 165 us against 127 for 100002 columns).  A
// full block there (`shift`) is read from the 32-bit word before, two bytes
// early, with one word more behind it (whose other half may lie past the row,
// never past the word); aligned_block puts the columns where they belong.
template <int DT, bool NT, uint32_t VECS>
__device__ __forceinline__ void load_block(const BlockAt &b, uint32_t lane, Loaded<VECS> &l, bool real = true) {
    constexpr uint32_t per = Logit<DT>::kPerVec;
    const bool tiny = b.n < per;
    gbyte *const p = tiny ? (gbyte *)__builtin_amdgcn_kernarg_segment_ptr() : b.p - (b.shift ? 2 : 0);
    const uint32_t last = tiny || !real ? 0 : (b.n - per) * Logit<DT>::kSize;
#pragma unroll
    for (uint32_t i = 0; i < VECS; ++i) {
        const uint32_t c = (64 * i + lane) * 16;
        gvec16any *const q = (gvec16any *)(p + (c < last ? c : last));
        if constexpr (NT) l.v[i] = __builtin_nontemporal_load(q);
        else l.v[i] = *q;
    }
    if constexpr (DT != ROG_DTYPE_F32) {
        typedef const __attribute__((address_space(1))) uint32_t gword;
        if (b.shift) l.behind = *(gword *)(p + (real ? VECS * 1024 : 0));
    }
}

// The vectors of a block as if they had been loaded at their own address: of a
// shifted one, each lane's 16 bytes from the two words they straddle, the last
// of them from the next lane or vector.
template <int DT, uint32_t VECS>
__device__ __forceinline__ void aligned_block(bool shift, Loaded<VECS> &l) {
    if constexpr (DT != ROG_DTYPE_F32) {
        if (!shift) return;
#pragma unroll
        for (uint32_t i = 0; i < VECS; ++i) {
            const uint32_t first = i + 1 < VECS ? uniform(l.v[i + 1 < VECS ? i + 1 : i].x) : uniform(l.behind);
            const uint32_t x = l.v[i].x, y = l.v[i].y, z = l.v[i].z, w = l.v[i].w;
            // lane 63 keeps `first`: wave_shl:1, as from_next_lane
            const uint32_t next = uint32_t(__builtin_amdgcn_update_dpp(int(first), int(x), 0x130, 0xf, 0xf, false));
            l.v[i] = vec16{align_bytes(y, x, 2), align_bytes(z, y, 2), align_bytes(w, z, 2), align_bytes(next, w, 2)};
        }
    }
}

// Whether element e of the lane's vector i, read as above, is the lane's own.
template <int DT>
__device__ __forceinline__ bool owns(uint32_t n, uint32_t i, uint32_t lane, uint32_t e) {
    const uint32_t c = own_column<DT>(i, lane);
    if (n < Logit<DT>::kPerVec) return c + e < n;
    return vec_place<DT>(n, i, lane) + e >= c;
}

// Puts -inf in the place of the elements of a tail that are not the lane's own
// (a block of kPerVec columns or more, its vectors as loaded).
template <int DT>
__device__ __forceinline__ void mask_tail(uint32_t n, uint32_t lane, vec16 (&v)[Logit<DT>::kVecs]) {
    constexpr uint32_t per = Logit<DT>::kPerVec, pack = per / 4;      // elements per word
    const uint32_t last = n - per;
#pragma unroll
    for (uint32_t i = 0; i < Logit<DT>::kVecs; ++i) {
        const uint32_t c = own_column<DT>(i, lane);
        const uint32_t others = c > last ? c - last : 0;       // leading elements that are another lane's
#pragma unroll
        for (uint32_t d = 0; d < 4; ++d) {
            const uint32_t keep = others <= pack * d ? ~0u : pack == 2 && others == 2 * d + 1 ? 0xFFFF0000u : 0u;
            v[i][d] = (v[i][d] & keep) | (Logit<DT>::kMinusInf & ~keep);
        }
    }
}

// The partial state of a softmax over some logits: m their largest (NaN if one
// is NaN), and with z = x * scale, |x| held within `bound`, and R = ref(m):
//     s = sum 2^(z - R),   t = sum 2^(z - R) (z - R).
// R is the rounded product m * scale, and z - R is one fused
// multiply-add, so the rounding of R cancels between s and what is read
// against it.  No logits: m = -inf, s = t = 0.
struct State {
    float m, r, s, t;      // r = ref(m)
};

struct Scaling {
    float scale, bound;
    // The reference for a largest logit m: finite for every m but +inf and NaN.
    __device__ __forceinline__ float ref(float m) const {
        float r = __builtin_amdgcn_fmed3f(m, -bound, bound) * scale;
        r = m < kInf ? r : __builtin_nanf("");
        asm("" : "+v"(r));      // one select here, not one behind every use
        return r;
    }
};

// Logits of a lane as they are used one by one: binary16 stays packed in its
// words (v_fma_mix_f32 widens it on the way), the others are widened first.
template <int DT>
struct Lane32 {
    float x[32];
    __device__ __forceinline__ explicit Lane32(const vec16 (&v)[Logit<DT>::kVecs]) {
#pragma unroll
        for (uint32_t i = 0; i < Logit<DT>::kVecs; ++i) widen_vec<DT>(v[i], x + i * Logit<DT>::kPerVec);
    }
    __device__ __forceinline__ float at(int i) const { return x[i]; }
    __device__ __forceinline__ float largest() const {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) m = max_nan(m, x[i]);
        return m;
    }
    __device__ __forceinline__ float smallest() const {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) m = __builtin_elementwise_minimum(m, x[i]);
        return m;
    }
    __device__ __forceinline__ void raise(float low) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = fmaxf(x[i], low);
    }
};
template <>
struct Lane32<ROG_DTYPE_F16> {
    f16x2 h[16];
    __device__ __forceinline__ explicit Lane32(const vec16 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t word = v[i / 4][i % 4];
            h[i] = __builtin_bit_cast(f16x2, word);
        }
    }
    __device__ __forceinline__ float at(int i) const { return float(i & 1 ? h[i / 2].y : h[i / 2].x); }
    __device__ __forceinline__ float largest() const {
        f16x2 m = h[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) m = __builtin_elementwise_maximum(m, h[i]);
        return max_nan(float(m.x), float(m.y));
    }
    __device__ __forceinline__ float smallest() const {
        f16x2 m = h[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) m = __builtin_elementwise_minimum(m, h[i]);
        return __builtin_elementwise_minimum(float(m.x), float(m.y));
    }
    __device__ __forceinline__ void raise(float) {
        const f16x2 low = {-65504.0f16, -65504.0f16};
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = __builtin_elementwise_max(h[i], low);
    }
};

// The state of a lane's 32 logits of a block.  bound * scale is 2^30: up to
// there the rounding of R stays below 64, so that no term overflows.  Where any
// lane of the wave holds a logit below -bound (-inf, or a mask of the lowest
// finite value; looking for the smallest costs half of raising all), those count
// as -bound: nothing against any reference but their own, and finite, so that
// 0 * (z - R) stays 0.  A row whose largest logit is at a bound or beyond is read
// again (the kernels' extreme rows).
//
// binary16, packed as it is, counts -inf as its lowest value instead: at most
// 2^-64 against a largest logit that is as far above; with one that is nearer
// in some lane, -inf is looked for column by column.  A lane that holds only
// -inf takes a reference of 2^30, against which all of it is nothing.
template <int DT>
__device__ __forceinline__ State state_of(const vec16 (&v)[Logit<DT>::kVecs], const Scaling &c) {
    Lane32<DT> x(v);
    const float m = x.largest();
    const float r = c.ref(m);
    float s[4], t[4], from = r;
    if (__ballot(x.smallest() < -c.bound)) {
        if constexpr (DT == ROG_DTYPE_F16) {
            if (__ballot(m > -kInf && (m + 65504.0f) * c.scale < 64.0f)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float z = x.at(i), y = z > -kInf ? __builtin_fmaf(z, c.scale, -r) : -200.0f, e = exp2_fast(y);
                    s[i & 3] = i < 4 ? e : s[i & 3] + e;
                    t[i & 3] = i < 4 ? e * y : __builtin_fmaf(e, y, t[i & 3]);
                }
                return State{m, r, (s[0] + s[1]) + (s[2] + s[3]), (t[0] + t[1]) + (t[2] + t[3])};
            }
            from = m > -kInf ? r : 1073741824.0f;
        }
        x.raise(-c.bound);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float y = __builtin_fmaf(x.at(i), c.scale, -from);
        const float e = exp2_fast(y);
        s[i & 3] = i < 4 ? e : s[i & 3] + e;
        t[i & 3] = i < 4 ? e * y : __builtin_fmaf(e, y, t[i & 3]);
    }
    return State{m, r, (s[0] + s[1]) + (s[2] + s[3]), (t[0] + t[1]) + (t[2] + t[3])};
}

// The state of a tiny block: the first lane has its columns.
template <int DT>
__device__ __forceinline__ State tiny_state(gbyte *p, uint32_t n, uint32_t lane, const Scaling &c) {
    constexpr uint32_t per = Logit<DT>::kPerVec;
    float x[per];
    widen_vec<DT>(load_tiny<DT>(p, n), x);
    float m = -kInf, s = 0, t = 0;
#pragma unroll
    for (uint32_t e = 0; e < per; ++e) {
        x[e] = lane == 0 ? x[e] : -kInf;
        m = max_nan(m, x[e]);
    }
    const float r = c.ref(m);
#pragma unroll
    for (uint32_t e = 0; e < per; ++e) {
        const float y = __builtin_fmaf(__builtin_amdgcn_fmed3f(x[e], -c.bound, c.bound), c.scale, -r);
        const float q = exp2_fast(y);
        s = s + q;
        t = __builtin_fmaf(q, y, t);
    }
    return State{m, r, s, t};
}

// The state of both sides' logits.  A side without logits leaves the other's
// bits as they are.
__device__ __forceinline__ State join(const State &a, const State &b) {
    const float r = max_nan(a.r, b.r);
    const float da = a.r - r, db = b.r - r;
    const float wa = exp2_fast(da), wb = exp2_fast(db);
    return State{max_nan(a.m, b.m), r, __builtin_fmaf(a.s, wa, b.s * wb),
                 __builtin_fmaf(wa, __builtin_fmaf(a.s, da, a.t), wb * __builtin_fmaf(b.s, db, b.t))};
}

__device__ __forceinline__ State no_state(const Scaling &c) { return State{-kInf, c.ref(-kInf), 0.0f, 0.0f}; }
__device__ __forceinline__ State make_state(float m, float s, float t, const Scaling &c) { return State{m, c.ref(m), s, t}; }

// Reductions over the 64 lanes of a wave, all active: within rows of 16 lanes
// by DPP exchanges (no shared memory), then over the four rows by lane reads.
// The result is uniform.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return bits_f32(uint32_t(__builtin_amdgcn_update_dpp(0, int(f32_bits(x)), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float lane_read(float x, int lane) {
    return bits_f32(uint32_t(__builtin_amdgcn_readlane(int(f32_bits(x)), lane)));
}
template <typename F>
__device__ __forceinline__ float reduce_lanes(float x, F f) {
    x = f(x, dpp<0xB1>(x));      // quad_perm 1,0,3,2
    x = f(x, dpp<0x4E>(x));      // quad_perm 2,3,0,1
    x = f(x, dpp<0x141>(x));     // row_half_mirror
    x = f(x, dpp<0x140>(x));     // row_mirror
    return f(f(lane_read(x, 0), lane_read(x, 16)), f(lane_read(x, 32), lane_read(x, 48)));
}

// Joins the 64 lanes' states: their largest logit first, then two sums.
__device__ __forceinline__ State join_lanes(const State &st, const Scaling &c) {
    const float m = reduce_lanes(st.m, [](float a, float b) { return max_nan(a, b); });
    const float r = c.ref(m), d = st.r - r;
    const float w = exp2_fast(d);
    const auto add = [](float a, float b) { return a + b; };
    return State{m, r, reduce_lanes(st.s * w, add), reduce_lanes(w * __builtin_fmaf(st.s, d, st.t), add)};
}

// Values handed from workgroup to workgroup of one launch: stores and loads at
// device scope, which go past the caches of the eight dies, so that no cache
// has to be written back or emptied around them.
__device__ __forceinline__ void publish(float *p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(double *p, double v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float collect(const float *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double collect(const double *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Called by every thread of a workgroup after its publish() stores: whether
// this is the last of `groups` workgroups to get here, by a counter that is
// zero before and after.  Each wave waits until its stores have reached
// device scope before the barrier that the counting thread passes; the last
// workgroup's collect() loads come after the counter's answer.
__device__ __forceinline__ bool last_to_arrive(uint32_t *counter, uint32_t groups, uint32_t &flag) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        flag = before == groups - 1;
        if (before == groups - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool last = flag != 0;
    asm volatile("" ::: "memory");
    return last;
}

}  // namespace rog
