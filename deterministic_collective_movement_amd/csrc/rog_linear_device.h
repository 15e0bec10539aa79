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

// The same address in all lanes.
__device__ __forceinline__ const uint8_t *uniform(const void *p) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return reinterpret_cast<const uint8_t *>(uintptr_t(uniform(uint32_t(b >> 32))) << 32 | uniform(uint32_t(b)));
}
// The thread's number, to derive anew from what would else be held in registers over a product.
__device__ __forceinline__ uint32_t fresh_thread() {
    uint32_t t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}
// The kernel's one argument, to read anew likewise.
template <class Args>
__device__ __forceinline__ const Args &fresh_args() {
    auto p = (const __attribute__((address_space(4))) Args *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Args *)p;
}
// Bytes from the first of `rows` rows of `row_bytes` to the end of the last: rows may be less than a row apart, or the same.
__device__ __forceinline__ uint32_t extent_of(int32_t rows, uint32_t stride, uint32_t row_bytes) {
    return rows > 0 ? uint32_t(rows - 1) * stride + row_bytes : 0;
}
// A window on [base, base + bytes), the same for all lanes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const uint8_t *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(uniform(base)), 0, int(uniform(bytes)), kBufferWord3);
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
                if constexpr (ES == 4) e = *(const __attribute__((address_space(1))) uint32_t *)(row + at + i);
                else if constexpr (ES == 2) e = *(const __attribute__((address_space(1))) uint16_t *)(row + at + i);
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

// A step of ROWS rows of 64 bytes.  A 16-byte read of a wave goes in four rounds
// of sixteen lanes, each of which can take all 256 bytes of the banks: lanes 0-3,
// 12-15, 20-27; 4-11, 16-19, 28-31; and the same 32 on.  So the four 16-byte units
// of a row stand at u ^ swizzle(row), which puts a round's lanes on sixteen different
// places: N's fragments take sixteen consecutive rows, M's the rows 8 a + b (a, b < 4) of
// 32 (or four on), lane 16 u + 4 a + b unit u.  (u ^ a instead: every read twice
// as long, 8192 x 131072 x 4096 bf16 6.37 ms.)
template <bool M_SIDE>
__device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    const uint32_t a = row >> (M_SIDE ? 3 : 2) & 3;
    return ((a << 1 | a >> 1) & 3) ^ (a & 2);          // 0, 2, 3, 1
}

template <bool M_SIDE, int ROWS, int THREADS, bool DIRECT, int ES>
struct RowSteps {
    static constexpr int kBytes = ROWS * int(kStepBytes);
    static constexpr int kRows = THREADS / 4;            // rows of one load of the workgroup
    static constexpr int kLoads = ROWS / kRows;
    static constexpr int kReads = 1;                     // shared memory instructions of a fragment
    static_assert(ROWS % kRows == 0 && kRows % 32 == 0, "whole waves, one swizzle for all of a lane's rows");
    const uint8_t *base;
    uint32_t rows, bytes;              // rows that there are, and their extent (below 2^31)
    uint32_t kbytes;
    int64_t stride;
    uint32_t voff[kLoads];             // the lane's units
    uint32_t unit;                     // their place in the rows, in bytes
    uint32_t k = 0;                    // the next step
    // rows_left: rows from `base` on that exist
    __device__ __forceinline__ RowSteps(const void *b, int64_t s, uint32_t rows_left, uint32_t kb)
        : base(uniform(b)), rows(uniform(rows_left < ROWS ? rows_left : ROWS)), bytes(uniform(extent_of(rows, uint32_t(s), kb))),
          kbytes(uniform(kb)), stride(s) {
        const uint32_t row = threadIdx.x / 4;
        unit = (threadIdx.x % 4 ^ swizzle<M_SIDE>(row)) * 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) voff[i] = (row + i * kRows) * uint32_t(s) + unit;
    }
    // Brings the next step to `to`, zeros past the rows.
    __device__ __forceinline__ void stage(uint8_t *to) {
        bring<false>(to, k++);         // past the last whole step zeros
    }
    // Brings the last step, which is not whole: zeros past K.
    __device__ __forceinline__ void stage_tail(uint8_t *to) const {
        if (kbytes % 16) bring<true, false>(to, kbytes / kStepBytes);   // a row ends inside a unit
        else bring<true>(to, kbytes / kStepBytes);
    }
    template <bool TAIL, bool STRAIGHT = DIRECT>
    __device__ __forceinline__ void bring(uint8_t *to, uint32_t step) const {
        const uint32_t at = step * kStepBytes;
        if constexpr (STRAIGHT) {
            const auto r = window(base, TAIL || at + kStepBytes <= kbytes ? bytes : 0);
            const bool inside = !TAIL || at + unit < kbytes;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                lbyte *p = (lbyte *)to + (i * THREADS + uniform(threadIdx.x / 64) * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16, inside ? voff[i] : kOutside, at, 0, 0);
            }
        } else {
            vec16 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t row = threadIdx.x / 4 + i * kRows, off = row * uint32_t(stride);
                v[i] = row < rows && (TAIL || at + kStepBytes <= kbytes) ? row_bytes<ES>((gbyte *)base + off, at + unit, kbytes)
                                                                               : vec16{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        }
    }
    // Reads fragments of a wave's rows from row0 (a multiple of 32) on: f is a constant, so that
    // a fragment's address is one register and an offset in the instruction.  The offset has 16
    // bits: HIGH is added to the register for arrays that lie beyond.
    template <uint32_t HIGH>
    struct Reader {
        uint32_t at;
        __device__ __forceinline__ explicit Reader(uint32_t row0) {
            const uint32_t l = threadIdx.x % 64, j = l % 16, row = M_SIDE ? 8 * (j / 4) + j % 4 : j;
            at = (row0 + row) * kStepBytes + (l / 16 ^ swizzle<M_SIDE>(row)) * 16 + HIGH;
            asm("" : "+v"(at));
        }
        __device__ __forceinline__ vec16 get(const uint8_t *from, int f) const {
            const int row = M_SIDE ? 32 * (f / 2) + 4 * (f & 1) : 16 * f;
            return *(const lvec16 *)((const lbyte *)from + (int(at) + row * int(kStepBytes) - int(HIGH)));
        }
        __device__ __forceinline__ void refresh() {}
    };
};

// ---------------------------------------------------------------------------
// Operands that come as K along rows (two-byte elements)
// ---------------------------------------------------------------------------

// A step of 32 rows of K, COLS elements each.  ds_read_b64_tr_b16 gives lane l of a
// quarter wave the column l of four rows of sixteen elements: lane j of the
// quarter names the 8 bytes of row j / 4 that hold its elements 4 (j % 4) and on.
// Half a wave goes at once: rows 0-3 and 8-11 (or 16 on, or four on), 32 bytes
// each, which stand at different places of the 256 bytes of the banks as the
// 32-byte pieces p of a row are at p ^ (2 (row % 4) + (row / 8) % 2).
template <int COLS, int THREADS, bool DIRECT>
struct ColSteps {
    static constexpr int kBytes = COLS * int(kStepBytes);
    static constexpr int kUnits = COLS / 8;              // 16-byte units of a row
    static constexpr int kLoads = 32 * kUnits / THREADS;
    static constexpr int kRows = THREADS / kUnits;       // rows of one load of the workgroup
    static constexpr int kReads = 2;
    static_assert(kRows % 16 == 0 || kRows == 8 || kRows == 4, "see `turn`");
    static_assert(kLoads * THREADS == 32 * kUnits && kUnits >= 16, "whole loads of rows of 256 bytes and more");
    const uint8_t *from;               // of the next step
    int32_t left;                      // rows of K from there on; below 0 past the last step (signed: a scalar has no saturating difference)
    uint32_t col_bytes;                // bytes of a row
    int64_t stride;
    uint32_t row, unit;
    uint32_t voff[kLoads];             // the lane's units
    static __device__ __forceinline__ uint32_t turn(uint32_t row) { return 4 * (row % 4) + 2 * (row / 8 % 2); }   // of units
    __device__ __forceinline__ ColSteps(const void *b, int64_t s, uint32_t rows_, uint32_t cols_left)
        : from(uniform(b)), left(int32_t(uniform(rows_))), col_bytes(uniform((cols_left < COLS ? cols_left : COLS) * 2)), stride(s) {
        row = threadIdx.x / kUnits;
        unit = threadIdx.x % kUnits;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) voff[i] = at(i) < col_bytes ? (row + i * kRows) * uint32_t(s) + at(i) : kOutside;
    }
    // The bytes of the lane's unit in row `row + i * kRows` of a step.
    __device__ __forceinline__ uint32_t at(int i) const { return (unit ^ turn(row + uint32_t(i) * kRows)) * 16; }
    // Brings the next step to `to`, zeros past the rows.
    __device__ __forceinline__ void stage(uint8_t *to) {
        if constexpr (DIRECT) {
            // a row past the last is past the window; in the last, nothing past the columns is read
            const auto r = window(from, extent_of(left < 32 ? left : 32, uint32_t(stride), col_bytes));
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                lbyte *p = (lbyte *)to + (i * THREADS + uniform(threadIdx.x / 64) * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16, voff[i], 0, 0, 0);
            }
        } else {
            vec16 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                v[i] = int32_t(row + i * kRows) < left ? row_bytes<2>((gbyte *)from + uint64_t(row + i * kRows) * uint64_t(stride), at(i), col_bytes)
                                              : vec16{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        }
        from += 32 * uint32_t(stride);
        left -= 32;
    }
    __device__ __forceinline__ void stage_tail(uint8_t *to) { stage(to); }   // K ends with a row
    // Fragments (sixteen consecutive columns) of a wave's columns from col0 on, a multiple of its fragments' columns
    // (4, 8 or more fragments): bits 5 to 7 of an address are the low ones of its fragment's number, turned.
    template <uint32_t HIGH>
    struct Reader {
        uint32_t lane;                 // fragment 0
        __device__ __forceinline__ explicit Reader(uint32_t col0) {
            const uint32_t l = threadIdx.x % 64, j = l % 16, k = l / 16 * 8 + j / 4;
            lane = k * (COLS * 2) + (col0 * 2 ^ turn(k) * 16) + 8 * (j % 4) + HIGH;
        }
        __device__ __forceinline__ vec16 get(const uint8_t *from, int f) const {
            const uint32_t at = (lane ^ f % 8 * 32) + f / 8 * 256;
            const lbyte *p = (const lbyte *)from + (int(at) - int(HIGH));
            struct { s16x4 lo, hi; } v = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)p),
                                          __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)(p + 4 * COLS * 2))};
            return __builtin_bit_cast(vec16, v);
        }
        // The fragments' addresses are made anew in every step: kept, they take the registers that hold fragments.
        __device__ __forceinline__ void refresh() { asm volatile("" : "+v"(lane)); }
    };
};

// Lanes 32 apart, and lanes 16 apart: of a pair of registers the lower lanes' values in first, the upper lanes' in
// second, in both halves: (a, b) gives a's halves to the lower lanes and b's to the upper ones.
struct Halves {
    float first, second;
};
__device__ __forceinline__ Halves halves32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(f32_bits(a), f32_bits(b), false, false);
    return Halves{bits_f32(r[0]), bits_f32(r[1])};
}
__device__ __forceinline__ Halves halves16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(f32_bits(a), f32_bits(b), false, false);
    return Halves{bits_f32(r[0]), bits_f32(r[1])};
}

// Two fragments of sixteen consecutive rows of M each, a and b, in a lane of quarter q rows 4 q and on of each: has
// the lane hold eight consecutive ones, from row 8 * eight_of(q) of the 32 on, in a and then b.
__device__ __forceinline__ void pair_up(float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(f32_bits(a), f32_bits(b), false, false);
    a = bits_f32(r[0]);
    b = bits_f32(r[1]);
}
__device__ __forceinline__ uint32_t eight_of(uint32_t quarter) { return quarter / 2 + quarter % 2 * 2; }

// ---------------------------------------------------------------------------
// A tile
// ---------------------------------------------------------------------------

// Waits until at most LOADS loads of this wave are in flight and its shared memory accesses are done, then for the other waves.
template <int LOADS>
__device__ __forceinline__ void arrive() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((LOADS & 15) | 7 << 4 | (LOADS >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// The order of a step's instructions: loads to the shared memory and reads from it dealt among the matrix instructions.
template <int N, int LOADS, int READS, int I>
struct Deal {
    static __device__ __forceinline__ void slot() {
        constexpr int kMfma = 8, kVmem = 16, kLds = 256, kSlots = LOADS + READS;
        constexpr int kCount = N * (I + 1) / kSlots - N * I / kSlots;
        if constexpr (kCount > 0) __builtin_amdgcn_sched_group_barrier(kMfma, kCount, 0);
        __builtin_amdgcn_sched_group_barrier(I * LOADS / kSlots != (I + 1) * LOADS / kSlots ? kVmem : kLds, 1, 0);
        if constexpr (I + 1 < kSlots) Deal<N, LOADS, READS, I + 1>::slot();
    }
};

constexpr int kStages = 4;

// The shared memory of a tile: arrays of their own, so that the compiler can tell a
// load in flight to one from a read of another (through one array it waits for all).
#define ROG_STAGE_MEMORY(STAGES, I, A, B) __shared__ __attribute__((aligned(16))) uint8_t a##I[(STAGES) > I ? (A) : 16], b##I[(STAGES) > I ? (B) : 16]
#define ROG_TILE_MEMORY(STAGES, A, B)                                                                           \
    ROG_STAGE_MEMORY(STAGES, 0, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 1, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 2, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 3, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 4, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 5, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 6, A, B);                                                                          \
    ROG_STAGE_MEMORY(STAGES, 7, A, B);                                                                          \
    const TileMemory memory = {{a0, a1, a2, a3, a4, a5, a6, a7}, {b0, b1, b2, b3, b4, b5, b6, b7}}
struct TileMemory {
    uint8_t *a[8], *b[8];
};

// FM x FN fragments of a wave at (m0, n0) of the tile, over `steps` whole steps of K and, if `tail`, a last one that is not.
// While a step is multiplied from registers, the next one's fragments are read,
// and up to three further steps are in flight to the shared memory: a step's
// memory is free as soon as every wave has its fragments.
template <int DT, int FM, int FN, class A, class B>
struct Tile {
    typedef typename Mat<DT>::Acc Acc;
    vec16 fa[2][FM], fb[2][FN];

    static constexpr uint32_t kHigh = A::kBytes * kStages >= 65536 ? 65536 : 0;
    typedef typename A::template Reader<0> ReadA;
    typedef typename B::template Reader<kHigh> ReadB;

    __device__ __forceinline__ void read(const ReadA &ra, const ReadB &rb, const uint8_t *pa, const uint8_t *pb, int set) {
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[set][i] = ra.get(pa, i);
#pragma unroll
        for (int i = 0; i < FN; ++i) fb[set][i] = rb.get(pb, i);
    }
    __device__ __forceinline__ void multiply(int set, Acc (&acc)[FM][FN]) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = Mat<DT>::mma(fa[set][i], fb[set][j], acc[i][j]);
    }
    // With FOURS steps past the last whole one are multiplied as zeros, up to a multiple of four (less to hold in registers).
    template <bool FOURS = false>
    __device__ __forceinline__ void run(A &a, B &b, uint32_t steps, bool tail, uint32_t m0, uint32_t n0, const TileMemory &mem,
                                        Acc (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)   // the compiler's host pass loses some kernels' stubs over what is in here
        constexpr int kEach = A::kLoads + B::kLoads;
        ReadA ra(m0);
        ReadB rb(n0);
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            a.stage(mem.a[i]);
            b.stage(mem.b[i]);
        }
        arrive<3 * kEach>();
        read(ra, rb, mem.a[0], mem.b[0], 0);
        // One way in and out of the loop, so that the accumulators stay where they are.
        for (uint32_t k = 0; FOURS ? k < steps : k + 4 <= steps; k += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                arrive<2 * kEach>();
                a.stage(mem.a[i]);
                b.stage(mem.b[i]);
                ra.refresh();
                rb.refresh();
                read(ra, rb, mem.a[(i + 1) % 4], mem.b[(i + 1) % 4], (i + 1) % 2);
                multiply(i % 2, acc);
                Deal<FM * FN, kEach, FM * A::kReads + FN * B::kReads, 0>::slot();
            }
        }
        const uint32_t rest = FOURS ? 0 : steps % 4;
        if (rest > 0) multiply(0, acc);
        arrive<0>();
        if (rest > 1) {
            read(ra, rb, mem.a[1], mem.b[1], 1);
            multiply(1, acc);
        }
        if (rest > 2) {
            read(ra, rb, mem.a[2], mem.b[2], 0);
            multiply(0, acc);
        }
        if (tail) {
            a.stage_tail(mem.a[3]);
            b.stage_tail(mem.b[3]);
            arrive<0>();
            read(ra, rb, mem.a[3], mem.b[3], 1);
            multiply(1, acc);
        }
#else
        (void)a, (void)b, (void)steps, (void)tail, (void)m0, (void)n0, (void)mem, (void)acc;
#endif
    }
};

// ---------------------------------------------------------------------------
// Tiles of few rows: bound by the weights' bytes
// ---------------------------------------------------------------------------

// A step of ROWS rows of 128 bytes, a line each.  Two rows are the 256 bytes of the
// banks: the eight 16-byte units u of a row stand at u ^ turn(row), where a read's
// rounds of sixteen lanes (see swizzle()) meet every place once.
template <bool M_SIDE, int ROWS, int THREADS, bool DIRECT, int ES>
struct RowLines {
    static constexpr int kBytes = ROWS * 128;
    static constexpr int kRows = THREADS / 8;
    static constexpr int kLoads = ROWS / kRows;
    static_assert(ROWS % kRows == 0, "whole waves");
    static __device__ __forceinline__ uint32_t turn(uint32_t row) {
        // the row's place among the sixteen of its fragment, halved
        const uint32_t q = M_SIDE ? (row >> 1 & 1) | (row >> 3 & 3) << 1 : row >> 1 & 7;
        return (q & 1) | (q >> 2 & 1) << 1 | ((q >> 1 ^ q >> 2) & 1) << 2;
    }
    const uint8_t *base;
    uint32_t rows, bytes, kbytes;
    int64_t stride;
    uint32_t at = 0;                   // of the next step in the rows
    __device__ __forceinline__ RowLines(const void *b, int64_t s, uint32_t rows_left, uint32_t kb)
        : base(uniform(b)), rows(uniform(rows_left < ROWS ? rows_left : ROWS)), bytes(uniform(extent_of(rows, uint32_t(s), kb))),
          kbytes(uniform(kb)), stride(s) {}
    // Brings the next step to `to`, zeros past the rows and past K.
    __device__ __forceinline__ void stage(uint8_t *to) {
        // A step in which a row ends inside 16 bytes goes through registers.  Its loads are waited for, and
        // with them all before them, so that counting loads in flight stays right.
        if (DIRECT && !(kbytes % 16 && at < kbytes && at + 128 > kbytes)) bring<true>(to);
        else bring<false>(to);
        at += 128;
    }
    template <bool STRAIGHT>
    __device__ __forceinline__ void bring(uint8_t *to) const {
        const uint32_t row = threadIdx.x / 8;
        if constexpr (STRAIGHT) {
            const auto r = window(base, bytes);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t unit = (threadIdx.x % 8 ^ turn(row + i * kRows)) * 16;
                const uint32_t v = at + unit < kbytes ? (row + i * kRows) * uint32_t(stride) + unit : kOutside;
                lbyte *p = (lbyte *)to + (i * THREADS + uniform(threadIdx.x / 64) * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16, v, at < kbytes ? at : 0, 0, 0);
            }
        } else {
            vec16 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t unit = (threadIdx.x % 8 ^ turn(row + i * kRows)) * 16, off = (row + i * kRows) * uint32_t(stride);
                v[i] = row + i * kRows < rows ? row_bytes<ES>((gbyte *)base + off, at + unit, kbytes) : vec16{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        }
    }
    // Fragment f, half ks of the step, of a wave's rows from row0 (a multiple of 32) on.
    static __device__ __forceinline__ vec16 get(const uint8_t *from, uint32_t row0, int f, int ks) {
        const uint32_t l = threadIdx.x % 64, j = l % 16, row = M_SIDE ? 8 * (j / 4) + j % 4 : j;
        const uint32_t first = (row0 + row) * 128 + ((ks * 4 + l / 16) ^ turn(row)) * 16;
        return *(const lvec16 *)((const lbyte *)from + first + (M_SIDE ? 32 * (f / 2) + 4 * (f & 1) : 16 * f) * 128);
    }
};

// A step of 64 rows of K, 64 elements (a line) each.  As ColSteps, with two rows in the 256 bytes of the banks: the
// 32-byte pieces p of a row are at p ^ turn(row).
template <int THREADS, bool DIRECT>
struct ColLines {
    static constexpr int kBytes = 64 * 128;
    static constexpr int kRows = THREADS / 8, kLoads = 64 / kRows;
    static __device__ __forceinline__ uint32_t turn(uint32_t row) { return (row >> 1 & 1) | (row >> 3 & 1) << 1; }
    const uint8_t *from;               // of the next step
    int32_t left;                      // rows of K from there on; below 0 past the last step (signed: a scalar has no saturating difference)
    uint32_t col_bytes;                // bytes of a row
    int64_t stride;
    __device__ __forceinline__ ColLines(const void *b, int64_t s, uint32_t rows, uint32_t cols_left)
        : from(uniform(b)), left(int32_t(uniform(rows))), col_bytes(uniform((cols_left < 64 ? cols_left : 64) * 2)), stride(s) {}
    __device__ __forceinline__ void stage(uint8_t *to) {
        const uint32_t row = threadIdx.x / 8;
        const auto r = window(from, extent_of(left < 64 ? left : 64, uint32_t(stride), col_bytes));
        vec16 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t k = row + i * kRows, at = (threadIdx.x % 8 ^ 2 * turn(k)) * 16;
            if constexpr (DIRECT) {
                lbyte *p = (lbyte *)to + (i * THREADS + uniform(threadIdx.x / 64) * 64) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)p, 16,
                                                         at < col_bytes ? k * uint32_t(stride) + at : kOutside, 0, 0, 0);
            } else {
                v[i] = int32_t(k) < left ? row_bytes<2>((gbyte *)from + uint64_t(k) * uint64_t(stride), at, col_bytes) : vec16{0, 0, 0, 0};
            }
        }
        if constexpr (!DIRECT)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *(lvec16 *)((lbyte *)to + (i * THREADS + threadIdx.x) * 16) = v[i];
        from += 64 * uint32_t(stride);
        left -= 64;
    }
    static __device__ __forceinline__ vec16 get(const uint8_t *from, uint32_t col0, int f, int ks) {
        const uint32_t l = threadIdx.x % 64, j = l % 16, k = ks * 32 + l / 16 * 8 + j / 4;
        const lbyte *p = (const lbyte *)from + k * 128 + ((col0 / 16 + f) ^ turn(k)) * 32 + 8 * (j % 4);
        struct { s16x4 lo, hi; } v = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)p),
                                      __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4 *)(p + 4 * 128))};
        return __builtin_bit_cast(vec16, v);
    }
};

// FM x FN fragments of a wave at (m0, n0) over `lines` steps of 128 bytes of K, GROUP of them at a time, up to
// STAGES - GROUP in flight.
template <int DT, int FM, int FN, int STAGES, int GROUP, class A, class B>
struct Stream {
    typedef typename Mat<DT>::Acc Acc;
    static_assert(STAGES % GROUP == 0 && STAGES >= 2 * GROUP, "whole groups");
    static __device__ __forceinline__ void run(A &a, B &b, uint32_t lines, uint32_t m0, uint32_t n0, const TileMemory &mem, Acc (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)   // as in Tile
        constexpr int kEach = A::kLoads + B::kLoads;
#pragma unroll
        for (int i = 0; i < STAGES - GROUP; ++i) {
            a.stage(mem.a[i]);
            b.stage(mem.b[i]);
        }
        // past the last step zeros are multiplied, which leaves the sums as they are
        for (uint32_t k = 0; k < lines; k += STAGES) {
#pragma unroll
            for (int i = 0; i < STAGES; i += GROUP) {
                arrive<(STAGES - 2 * GROUP) * kEach>();
                vec16 fa[2 * GROUP][FM], fb[2 * GROUP][FN];
#pragma unroll
                for (int g = 0; g < 2 * GROUP; ++g) {
#pragma unroll
                    for (int f = 0; f < FM; ++f) fa[g][f] = A::get(mem.a[i + g / 2], m0, f, g % 2);
#pragma unroll
                    for (int f = 0; f < FN; ++f) fb[g][f] = B::get(mem.b[i + g / 2], n0, f, g % 2);
                }
#pragma unroll
                for (int g = 0; g < GROUP; ++g) {
                    a.stage(mem.a[(i + g + STAGES - GROUP) % STAGES]);
                    b.stage(mem.b[(i + g + STAGES - GROUP) % STAGES]);
                }
#pragma unroll
                for (int g = 0; g < 2 * GROUP; ++g)
#pragma unroll
                    for (int f = 0; f < FM; ++f)
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[f][j] = Mat<DT>::mma(fa[g][f], fb[g][j], acc[f][j]);
            }
        }
        arrive<0>();
#else
        (void)a, (void)b, (void)lines, (void)m0, (void)n0, (void)mem, (void)acc;
#endif
    }
};

// A product of rows and rows (weights and states) in the form F.
template <int DT, class F, bool DIRECT, int ES, bool WIDE>
struct RowProduct;
template <int DT, class F, bool DIRECT, int ES>
struct RowProduct<DT, F, DIRECT, ES, true> {
    typedef RowSteps<true, F::kColumns, F::kThreads, DIRECT, ES> A;
    typedef RowSteps<false, F::kRows, F::kThreads, DIRECT, ES> B;
    template <class Acc>
    static __device__ __forceinline__ void run(A &a, B &b, uint32_t kbytes, uint32_t m0, uint32_t n0, const TileMemory &mem, Acc &acc) {
        Tile<DT, F::kFM, F::kFN, A, B>().run(a, b, kbytes / kStepBytes, kbytes % kStepBytes != 0, m0, n0, mem, acc);
    }
};
template <int DT, class F, bool DIRECT, int ES>
struct RowProduct<DT, F, DIRECT, ES, false> {
    typedef RowLines<true, F::kColumns, F::kThreads, DIRECT, ES> A;
    typedef RowLines<false, F::kRows, F::kThreads, DIRECT, ES> B;
    template <class Acc>
    static __device__ __forceinline__ void run(A &a, B &b, uint32_t kbytes, uint32_t m0, uint32_t n0, const TileMemory &mem, Acc &acc) {
        Stream<DT, F::kFM, F::kFN, F::kStages, 1, A, B>::run(a, b, (kbytes + 127) / 128, m0, n0, mem, acc);
    }
};

// The power of two that brings `most` into [2^14, 2^15): binary16 holds coefficients of at most `most` after it.
__device__ __forceinline__ float power_for(float most) {
    int e = 0;
    if (most > 0 && most < kInf) e = 14 - (int(f32_bits(most) >> 23) - 127);
    e = e > 100 ? 100 : e < -100 ? -100 : e;
    return __builtin_ldexpf(1.0f, e);
}
// The largest |G| that a row can have: p |log p| is at most 1 / e, p H at most log V < 21.5.
__device__ __forceinline__ float most_of(float g, float gh, float inv_t) {
    return (fabsf(g) + 22.0f * fabsf(gh)) * inv_t;
}

// Workgroups to tiles: consecutive workgroups go to the eight XCDs in turn, each
// with an L2 of its own, so an XCD takes a run of consecutive tiles, and a run
// goes over groups of kGroup tiles along M for every tile along N, so that the
// tiles in flight on an XCD share their operands.
struct TileAt {
    uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t id, uint32_t tm, uint32_t tn) {
    constexpr uint32_t kXcds = 8, kGroup = 8;
    const uint32_t all = tm * tn, per = all / kXcds, more = all % kXcds;
    const uint32_t x = id % kXcds, t = x * per + (x < more ? x : more) + id / kXcds;
    const uint32_t group = t / (kGroup * tn), in = t % (kGroup * tn);
    const uint32_t gm = tm - group * kGroup < kGroup ? tm - group * kGroup : kGroup;
    return TileAt{group * kGroup + in % gm, in / gm};
}

// A workgroup's tile of the wide form: the tiles past the last whole round of the
// CUs are dealt out in quarters where they are few (kTailSplit).
struct Place {
    TileAt at;
    uint32_t quarter;                  // 4: the whole tile
    bool none;
};
__device__ __forceinline__ Place place_of(uint32_t id, uint32_t tm, uint32_t tn) {
    const uint32_t all = tm * tn, over = all % kCus, whole = over <= kTailSplit ? all - over : all;
    if (id < whole) return Place{tile_at(id, tm, tn), 4, false};
    const uint32_t q = id - whole;
    if (whole == all || q >= 4 * over) return Place{TileAt{0, 0}, 4, true};
    return Place{tile_at(whole + q / 4, tm, tn), q % 4, false};
}

__device__ __forceinline__ uint32_t shard_of_tile(const WeightShards &h, uint32_t tile) {
    uint32_t r = 0;
    while (tile >= h.tile0[r + 1]) ++r;
    return r;
}

// Host: enqueues a kernel of one argument structure, and what a call answers then.
template <class Args>
inline hipError_t launch(void (*kernel)(Args), uint32_t grid, uint32_t threads, const Args &args, hipStream_t stream) {
    void *list[] = {const_cast<Args *>(&args)};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(threads), list, 0, stream);
}

inline rog_status launched(hipError_t e) {
    if (e == hipSuccess) return ROG_OK;
    g_last_hip_error = int(e);
    return ROG_ERR_LAUNCH;
}

}  // namespace rog
