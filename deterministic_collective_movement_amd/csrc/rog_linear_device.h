// rog_linear_device.h -- tiles of a matrix product through the shared memory and
// the matrix units of gfx950, for the policy head's products.
//
// Both operands of a product come as rows along K (weights [column][K], states
// [row][K]) or as K along rows (states [K = row][element]).  A workgroup takes a
// tile of BM x BN outputs; a slab of both operands is brought into the shared
// memory by loads that go there directly (a lane's 16 bytes land at the wave's
// base + 16 * lane, so a swizzle is a permutation of the global addresses), and
// the waves read their fragments from it.  M is the side whose consecutive
// outputs stand in one lane: the lanes of a quarter wave hold four consecutive
// rows of M for one column of N, and fragments come in pairs whose rows are dealt
// so that a lane holds eight consecutive outputs.
#pragma once

#include "rog_head_device.h"
#include "rog_linear.h"

namespace rog {

#pragma clang fp contract(off)

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lbyte;
typedef __attribute__((address_space(3))) vec16 lvec16;
typedef __attribute__((address_space(3))) s16x4 ls16x4;

constexpr int kTypeI8 = 3;   // beside rog_dtype: 8-bit integers

template <int DT>
struct Mat;
template <>
struct Mat<ROG_DTYPE_BF16> {
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc mma(vec16 a, vec16 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Mat<ROG_DTYPE_F16> {
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc mma(vec16 a, vec16 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Mat<kTypeI8> {
    typedef i32x4 Acc;
    static __device__ __forceinline__ Acc mma(vec16 a, vec16 b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
    }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void *base, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, int(bytes < 0x7fffffffu ? bytes : 0x7fffffffu), kBufferWord3);
}
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every window: reads as zero

// Sixteen bytes of a row of `end` bytes, from byte `at` on; zeros past its end.  Any alignment.
template <int ES>
__device__ __forceinline__ vec16 row_bytes(gbyte *row, uint32_t at, uint32_t end) {
    vec16 v = {0, 0, 0, 0};
    if (at + 16 <= end) {
        v = *(gvec16any *)(row + at);
    } else if (at < end) {
#pragma unroll
        for (uint32_t i = 0; i < 16; i += ES) {
            uint32_t e = 0;
            if (at + i < end) {
                if constexpr (ES == 2) e = *(const __attribute__((address_space(1))) uint16_t *)(row + at + i);
                else e = row[at + i];
            }
            v[i / 4] |= e << (8 * (i % 4));
        }
    }
    return v;
}

// ---------------------------------------------------------------------------
// Operands that come as rows along K
// ---------------------------------------------------------------------------

// A slab of ROWS rows of 128 bytes.  The eight 16-byte units of a row stand in
// the order u ^ swizzle(row), so that the sixteen rows of a fragment read at one
// unit fall on different banks: M's fragments take the rows 8 a + b (a, b < 4) of
// 32 (or four on), N's sixteen consecutive ones.
template <bool M_SIDE>
__device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    return M_SIDE ? (row >> 1 & 1) | (row >> 3 & 3) << 1 : row >> 1 & 7;
}
// The row that lane l holds of fragment f.
template <bool M_SIDE>
__device__ __forceinline__ uint32_t frag_row(uint32_t f, uint32_t l16) {
    return M_SIDE ? 32 * (f / 2) + 8 * (l16 / 4) + 4 * (f & 1) + l16 % 4 : 16 * f + l16;
}

template <bool M_SIDE, int ROWS, int THREADS, bool DIRECT, int ES>
struct RowSlab {
    static constexpr int kBytes = ROWS * int(kSlabBytes);
    static constexpr int kLoads = ROWS * 8 / THREADS;
    static_assert(ROWS * 8 % THREADS == 0, "whole waves");
    const uint8_t *base;
    uint64_t rows_bytes;               // of the rows that there are
    uint32_t kbytes;
    int64_t stride;
    uint32_t voff;                     // the lane's first unit
    uint32_t unit;                     // its place in the slab's rows, in bytes
    // rows_left: rows from `base` on that exist
    __device__ __forceinline__ RowSlab(const void *b, int64_t s, uint32_t rows_left, uint32_t kb)
        : base(static_cast<const uint8_t *>(b)), rows_bytes(uint64_t(rows_left) * uint64_t(s)), kbytes(kb), stride(s) {
        const uint32_t row = threadIdx.x / 8;
        unit = (threadIdx.x % 8 ^ swizzle<M_SIDE>(row)) * 16;
        voff = row * uint32_t(s) + unit;
    }
    // Slab `k` to `to`.  Rows 8 * kWave apart have the same swizzle where THREADS / 8 is a multiple of 32.
    __device__ __forceinline__ void stage(uint8_t *to, uint32_t k) const {
        static_assert(THREADS / 8 % 32 == 0, "one swizzle for all of a lane's rows");
        const uint32_t at = k * kSlabBytes;
        if constexpr (DIRECT) {
            const auto r = window(base, rows_bytes);
            uint32_t v = voff;
            if (at + kSlabBytes > kbytes && at + unit >= kbytes) v = kOutside;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                lbyte *p = (lbyte *)to + (i * THREADS + threadIdx.x / 64 * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16,
                                                         v == kOutside ? v : v + uint32_t(i) * (THREADS / 8) * uint32_t(stride), at, 0, 0);
            }
        } else {
            vec16 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint64_t off = uint64_t(threadIdx.x / 8 + i * (THREADS / 8)) * uint64_t(stride);
                v[i] = off < rows_bytes ? row_bytes<ES>((gbyte *)base + off, at + unit, kbytes) : vec16{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        }
    }
    // Reads fragments of a wave's rows from row0 (a multiple of 32) on: f and the half slab ks are constants,
    // so that a fragment's address is one of two registers and an offset in the instruction.
    struct Reader {
        uint32_t at[2];
        __device__ __forceinline__ explicit Reader(uint32_t row0) {
            const uint32_t l = threadIdx.x % 64, row = frag_row<M_SIDE>(0, l % 16);
            at[0] = (row0 + row) * kSlabBytes + (l / 16 ^ swizzle<M_SIDE>(row)) * 16;
            at[1] = at[0] ^ 64;
        }
        __device__ __forceinline__ vec16 get(const uint8_t *from, int f, int ks) const {
            const int row = M_SIDE ? 32 * (f / 2) + 4 * (f & 1) : 16 * f;
            return *(const lvec16 *)((const lbyte *)from + at[ks] + row * int(kSlabBytes));
        }
    };
};

// ---------------------------------------------------------------------------
// Operands that come as K along rows (two-byte elements)
// ---------------------------------------------------------------------------

// A slab of 64 rows of K, COLS elements each, in units of 16 bytes at
// u ^ 4 (row % 4).  ds_read_b64_tr_b16 gives lane l of a quarter wave the column l
// of four rows of sixteen elements: lane j of the quarter names the 8 bytes of
// row j / 4 that hold its elements 4 (j % 4) and on.
template <bool M_SIDE, int COLS, int THREADS, bool DIRECT>
struct ColSlab {
    static constexpr int kBytes = COLS * int(kSlabBytes);
    static constexpr int kUnits = COLS / 8;              // of a row
    static constexpr int kLoads = 64 * kUnits / THREADS;
    static constexpr int kRows = THREADS / kUnits;       // rows of one load of the workgroup
    static_assert(kRows % 4 == 0, "one swizzle for all of a lane's rows");
    const uint8_t *base;
    uint32_t rows, col_bytes;          // rows of K, bytes of a row from `base` on
    int64_t stride;
    uint32_t row, unit;
    __device__ __forceinline__ ColSlab(const void *b, int64_t s, uint32_t rows_, uint32_t cols_left)
        : base(static_cast<const uint8_t *>(b)), rows(rows_), col_bytes(cols_left * 2), stride(s) {
        row = threadIdx.x / kUnits;
        unit = (threadIdx.x % kUnits ^ 4 * (row % 4)) * 16;
    }
    __device__ __forceinline__ void stage(uint8_t *to, uint32_t k) const {
        const uint32_t left = rows > k * 64 ? rows - k * 64 : 0;
        const uint8_t *from = base + uint64_t(k) * 64 * uint64_t(stride);
        if constexpr (DIRECT) {
            // the last row ends with the columns that are read: nothing past it is in the window
            const auto r = window(from, uint64_t(left < 64 ? left : 64) * uint64_t(stride));
            const uint32_t v = unit < col_bytes ? row * uint32_t(stride) + unit : kOutside;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                lbyte *p = (lbyte *)to + (i * THREADS + threadIdx.x / 64 * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16,
                                                         v == kOutside ? v : v + uint32_t(i) * kRows * uint32_t(stride), 0, 0, 0);
            }
        } else {
            vec16 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                v[i] = row + i * kRows < left ? row_bytes<2>((gbyte *)from + uint64_t(row + i * kRows) * uint64_t(stride), unit, col_bytes)
                                              : vec16{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        }
    }
    // Fragments of a wave's columns from col0 (a multiple of 64) on: the 64 bytes that hold fragments 2 i and
    // 2 i + 1 stand at i ^ (row % 4) of four.
    struct Reader {
        static constexpr int kAts = 4;
        uint32_t at[kAts];
        __device__ __forceinline__ explicit Reader(uint32_t col0) {
            const uint32_t l = threadIdx.x % 64, j = l % 16, k = l / 16 * 8 + j / 4;
            const uint32_t in = M_SIDE ? 16 * (j % 4) : 8 * (j % 4);
#pragma unroll
            for (uint32_t i = 0; i < kAts; ++i) at[i] = k * (COLS * 2) + ((col0 / 32 + i) ^ j / 4) * 64 + in;
        }
        __device__ __forceinline__ vec16 get(const uint8_t *from, int f, int ks) const {
            const int off = ks * 32 * COLS * 2 + (f / 8) * 256 + (f & 1) * (M_SIDE ? 8 : 32);
            const lbyte *p = (const lbyte *)from + at[f / 2 % kAts] + off;
            struct { s16x4 lo, hi; } v = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)p),
                                          __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)(p + 4 * COLS * 2))};
            return __builtin_bit_cast(vec16, v);
        }
    };
};

// ---------------------------------------------------------------------------
// A tile
// ---------------------------------------------------------------------------

// FM x FN fragments of a wave at (m0, n0) of the tile, over `slabs` slabs.
template <int DT, int FM, int FN, class A, class B, class Acc>
__device__ __forceinline__ void multiply(const uint8_t *pa, const uint8_t *pb, const typename A::Reader &ra, const typename B::Reader &rb,
                                         Acc (&acc)[FM][FN]) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        vec16 a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = ra.get(pa, i, ks);
#pragma unroll
        for (int i = 0; i < FN; ++i) b[i] = rb.get(pb, i, ks);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = Mat<DT>::mma(a[i], b[j], acc[i][j]);
    }
}

template <int DT, int FM, int FN, class A, class B, class Acc>
__device__ __forceinline__ void tile_product(const A &a, const B &b, uint32_t slabs, uint32_t m0, uint32_t n0, uint8_t *a0, uint8_t *a1,
                                             uint8_t *b0, uint8_t *b1, Acc (&acc)[FM][FN]) {
    const typename A::Reader ra(m0);
    const typename B::Reader rb(n0);
    if (slabs) {
        a.stage(a0, 0);
        b.stage(b0, 0);
    }
    // One way in and out of the loop: the accumulators stay where they are.  Past the last slab zeros are brought.
    for (uint32_t k = 0; k + 1 < slabs; k += 2) {
        __syncthreads();
        a.stage(a1, k + 1);
        b.stage(b1, k + 1);
        multiply<DT, FM, FN, A, B>(a0, b0, ra, rb, acc);
        __syncthreads();
        a.stage(a0, k + 2);
        b.stage(b0, k + 2);
        multiply<DT, FM, FN, A, B>(a1, b1, ra, rb, acc);
    }
    __syncthreads();
    if (slabs & 1) multiply<DT, FM, FN, A, B>(a0, b0, ra, rb, acc);
}

// Workgroups to tiles: consecutive workgroups go to the eight XCDs in turn, each
// with an L2 of its own, so an XCD takes a run of consecutive tiles, and a run
// goes over groups of kGroup tiles along M for every tile along N, so that the
// tiles in flight on an XCD share their operands.
struct TileAt {
    uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t id, uint32_t tm, uint32_t tn) {
    constexpr uint32_t kXcds = 8, kGroup = 4;
    const uint32_t all = tm * tn, per = all / kXcds, more = all % kXcds;
    const uint32_t x = id % kXcds, t = x * per + (x < more ? x : more) + id / kXcds;
    const uint32_t group = t / (kGroup * tn), in = t % (kGroup * tn);
    const uint32_t gm = tm - group * kGroup < kGroup ? tm - group * kGroup : kGroup;
    return TileAt{group * kGroup + in % gm, in / gm};
}

__device__ __forceinline__ uint32_t shard_of_tile(const WeightShards &h, uint32_t tile) {
    uint32_t r = 0;
    while (tile >= h.tile0[r + 1]) ++r;
    return r;
}

}  // namespace rog
