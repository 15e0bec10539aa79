// rog_logprob.hip -- HIP kernels of the token log probabilities for gfx950
// (CDNA4) and the C entry points that launch them.
//
// Per row of V logits x_j, z_j = x_j log2(e) / T, in one pass over the row:
// every lane keeps the partial states (m, s, t) of its columns (rog_head_device.h),
// states are joined in a fixed order, and with M, S, T' of the whole row
//     L = log2 S,  lse = M / T + (L - (M log2(e) / T - ref(M))) ln 2,
//     logp = ((z_token - ref(M)) - L) ln 2,  entropy = (L - T' / S) ln 2.
// M / T is rounded together with the rest, once, so that lse is off by half a
// unit in its last place and what the sums leave, however large M is.
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

// Orders logits as unsigned numbers; -0 counts as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = f32_bits(x + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) {
    return bits_f32(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
constexpr uint32_t kOrderMinusInf = 0x007FFFFFu;   // order_of(-inf)

// The threads that finish one row together: a workgroup or one wave.
template <int THREADS>
struct Team {
    static constexpr uint32_t kThreads = THREADS;
    static constexpr uint32_t kTeamWaves = THREADS / 64;
    static constexpr uint32_t kSlots = THREADS == 64 ? kUnitBlocks : kTeamWaves * kTopSlots;     // table rows of 64 lanes
    static constexpr uint32_t kEntries = kSlots * 64;
    static constexpr uint32_t kListCap = THREADS == 64 ? 128 : 512;             // candidates held at once
    static __device__ __forceinline__ uint32_t id() { return THREADS == 64 ? threadIdx.x & 63 : threadIdx.x; }
    static __device__ __forceinline__ void sync() {
        if constexpr (THREADS == 64) {
            // a wave's shared-memory accesses complete in order; keep the compiler from moving them
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        } else {
            __syncthreads();
        }
    }
};

struct Shared {
    float m[64], s[64], t[64];   // the states of units 64 apart, joined
    float lane_m[kWaves][64];    // the lanes' largest logits, by wave
    float lane_s[kWaves][64], lane_t[kWaves][64];   // split: with them, the states of a unit's blocks
    float row[4];                // m, s, t and log2 s of the row, written by the first wave
    uint32_t equal;              // extreme rows: columns that equal the largest
    uint32_t last;
};
// Where a row's blocks are, for lanes that each look for another: per shard for a
// workgroup's row, per block for a wave's (at most four).
template <int THREADS>
struct Places {
    uint64_t x[kMaxPeers];         // element (0, 0)
    int64_t stride[kMaxPeers];
    uint32_t width[kMaxPeers], col0[kMaxPeers], block0[kMaxPeers];
    // by one wave, lane r bringing shard r; the LDS writes wait for the kernel arguments
    __device__ __forceinline__ void fill(const LogprobArgs &a, uint32_t lane) {
        if (lane < a.sh.W) {
            const Shard &s = a.sh.s[lane];
            x[lane] = reinterpret_cast<uint64_t>(s.x);
            stride[lane] = s.stride;
            width[lane] = s.width;
            col0[lane] = s.col0;
            block0[lane] = a.sh.block0[lane];
        }
    }
    template <int DT>
    __device__ __forceinline__ BlockAt at(const LogprobArgs &a, uint32_t row, uint32_t b) const {
        uint32_t r = 0, first = 0;
        if (a.sh.even) {
            r = divide(b, a.sh.even_div);
            first = r * a.sh.even;
        } else {                   // the last shard that begins at or before block b
            for (uint32_t step = kMaxPeers / 2; step; step /= 2)
                if (step < a.sh.W && r + step < a.sh.W && block0[r + step] <= b) r += step;
            first = block0[r];
        }
        const uint32_t off = (b - first) * kHeadBlock, left = width[r] - off;
        return BlockAt{(gbyte *)(x[r] + uint64_t(int64_t(row) * stride[r]) + uint64_t(off) * Logit<DT>::kSize),
                       left < kHeadBlock ? left : kHeadBlock, col0[r] + off, r, off, false};
    }
};
template <>
struct Places<64> {
    uint64_t p[kUnitBlocks];
    uint32_t n[kUnitBlocks], col[kUnitBlocks];
    __device__ __forceinline__ void set(uint32_t b, const BlockAt &at) {
        p[b] = reinterpret_cast<uint64_t>((const uint8_t *)at.p);
        n[b] = at.n;
        col[b] = at.col;
    }
    template <int DT>
    __device__ __forceinline__ BlockAt at(const LogprobArgs &, uint32_t, uint32_t b) const {
        return BlockAt{(gbyte *)p[b], n[b], col[b], 0, 0, false};
    }
};

template <typename T>
struct SharedTop {
    float tab[T::kEntries];    // [slot][lane]: largest logit of the slot's blocks in the lane's columns
    uint64_t list[T::kListCap];
    uint64_t floor_key;        // a later floor, as found by one lane
    uint32_t hit_count, count;
    uint16_t hits[T::kEntries];
    Places<int(T::kThreads)> places;
};
struct Nothing {};
template <typename T, bool TOP> struct SharedFor { typedef Nothing type; };
template <typename T> struct SharedFor<T, true> { typedef SharedTop<T> type; };

constexpr float kMaxFinite = 3.40282347e38f;

// What a row comes to: the reference of its largest logit m, l = log2 S, and
// lse in nats, held in the finite range, so that a row masked with the lowest
// finite values does not read as one masked with -inf.
struct Row {
    float r, l, m, lse;
    bool extreme;
    // m / T + x: 1 / T in two parts, one rounding of the size of the result
    __device__ __forceinline__ float above_largest(float x, const LogprobArgs &a) const {
        return __builtin_fmaf(m, a.inv_t, __builtin_fmaf(m, a.inv_t_rest, x));
    }
    // log probability of a logit of the row
    __device__ __forceinline__ float logp(float x, const LogprobArgs &a) const {
        if (extreme) return (x - m) * a.inv_t - l * kLn2;
        if (x < -a.bound) return __builtin_fmaf(x, a.inv_t, -lse);      // x * scale may overflow
        return (__builtin_fmaf(x, a.scale, -r) - l) * kLn2;
    }
};

// Block j (in its order) of the blocks that wave w of a workgroup takes.
__device__ __forceinline__ uint32_t wave_block(uint32_t w, uint32_t j) { return j * kChunkUnits + w; }

// The block that table row `slot` holds at place i (of 1 << slot_shift).
template <typename T>
__device__ __forceinline__ uint32_t slot_block(uint32_t slot, uint32_t i, uint32_t shift) {
    if constexpr (T::kThreads == 64) return slot;
    else return wave_block(slot / kTopSlots, ((slot % kTopSlots) << shift) + i);
}

// The first floor of the candidates, the same in every lane of a wave: the K-th
// largest of the 64 lanes' largest logits, bit by bit, to 16 bits (the rest
// zero: a little lower).
__device__ __forceinline__ uint64_t first_floor(float lane_m, uint32_t K) {
    const uint32_t o = order_of(lane_m);
    uint32_t k = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t higher = k | 1u << bit;
        k = uint32_t(__popcll(__ballot(o >= higher))) >= K ? higher : k;
    }
    if (k <= kOrderMinusInf) k = kOrderMinusInf + 1;      // -inf is no alternative
    return uint64_t(k) << 32;
}

// The table's entries that reach a floor.  Counts are zero before.
template <typename T>
__device__ __forceinline__ void find_hits(uint64_t floor_key, SharedTop<T> &top) {
    const float floor_x = from_order(uint32_t(floor_key >> 32));
#pragma unroll
    for (uint32_t e = T::id(); e < T::kEntries; e += T::kThreads)
        if (top.tab[e] >= floor_x) top.hits[atomicAdd(&top.hit_count, 1u)] = uint16_t(e);
}

// Lists the candidates for a row's K best alternatives from its table, and
// returns how many: every column that reaches the floor, so K at least where
// the row has as many.  Called by the whole team, after find_hits with this
// floor and a sync; leaves the list in sync.
template <int DT, typename T>
__device__ __forceinline__ uint32_t list_candidates(const LogprobArgs &a, uint32_t row, uint64_t floor_key, SharedTop<T> &top) {
    constexpr uint32_t per = Logit<DT>::kPerVec;
    const uint32_t tid = T::id(), K = a.top_k;
    const uint32_t shift = T::kThreads == 64 ? 0 : a.slot_shift;
    const uint32_t vecs_shift = shift + (Logit<DT>::kVecs == 8 ? 3 : 2);
    for (;;) {
        const float floor_x = from_order(uint32_t(floor_key >> 32));
        const uint64_t tasks = uint64_t(top.hit_count) << vecs_shift;
        for (uint64_t q = tid; q < tasks; q += T::kThreads) {
            const uint32_t e = top.hits[q >> vecs_shift], i = uint32_t(q) & ((1u << vecs_shift) - 1);
            const uint32_t b = slot_block<T>(e / 64, i / Logit<DT>::kVecs, shift), el = e % 64, vi = i % Logit<DT>::kVecs;
            if (b >= a.sh.blocks) continue;
            const BlockAt at = top.places.template at<DT>(a, row, b);
            float x[per];
            widen_vec<DT>(load_vec<DT>(at.p, at.n, vi, el), x);
            const uint32_t col = at.col + (at.n < per ? 0 : vec_place<DT>(at.n, vi, el));
#pragma unroll
            for (uint32_t k = 0; k < per; ++k) {
                const uint64_t key = uint64_t(order_of(x[k])) << 32 | uint32_t(~(col + k));
                if (x[k] >= floor_x && owns<DT>(at.n, vi, el, k) && key >= floor_key) {
                    const uint32_t place = atomicAdd(&top.count, 1u);
                    if (place < T::kListCap) top.list[place] = key;
                }
            }
        }
        T::sync();
        const uint32_t n = top.count;
        if (n <= T::kListCap) return n;
        T::sync();
        // More columns reach the floor than the list holds (many equal logits):
        // the K-th best of those listed is a higher floor that K columns reach.
        // It rises with every turn, since the list holds more than K.
        for (uint32_t q = tid; q < T::kListCap; q += T::kThreads) {
            const uint64_t key = top.list[q];
            uint32_t above = 0;
            for (uint32_t k = 0; k < T::kListCap; ++k) above += top.list[k] > key;
            if (above == K - 1) top.floor_key = key;
        }
        if (tid == 0) top.hit_count = top.count = 0;
        T::sync();
        floor_key = top.floor_key;
        find_hits<T>(floor_key, top);
        T::sync();
    }
}

// Writes the K best of the n candidates, each at the place of its rank.
template <typename T>
__device__ __forceinline__ void write_alternatives(const LogprobArgs &a, uint32_t row, uint32_t n, const Row &v, const SharedTop<T> &top) {
    const uint32_t tid = T::id(), K = a.top_k;
    for (uint32_t q = tid; q < n; q += T::kThreads) {
        const uint64_t key = top.list[q];
        uint32_t above = 0;
#pragma unroll 8
        for (uint32_t k = 0; k < n; ++k) above += top.list[k] > key;
        if (above < K) {
            const float x = from_order(uint32_t(key >> 32));
            const uint64_t o = uint64_t(row) * K + above;
            if (a.top_ids) a.top_ids[o] = ~uint32_t(key);
            if (a.top_logp) a.top_logp[o] = v.logp(x, a);
        }
    }
    for (uint32_t q = n + tid; q < K; q += T::kThreads) {
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

// The logit of column `tok` of a row; 0 for a column past the end.  Read at the
// start of a kernel and used at its end.
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobArgs &a, uint32_t row, int64_t token) {
    if (token >= int64_t(a.vocab)) return 0.0f;
    const uint32_t tok = uint32_t(token);
    uint32_t r = 0;
    while (r + 1 < a.sh.W && a.sh.s[r + 1].col0 <= tok) ++r;
    const Shard &s = a.sh.s[r];
    return load_logit<DT>((gbyte *)s.x + int64_t(row) * s.stride + uint64_t(tok - s.col0) * Logit<DT>::kSize);
}

// How many of a wave's share of a row's columns equal x: blocks first, first + step, ...
template <int DT>
__device__ __forceinline__ uint32_t count_equal(const LogprobArgs &a, uint32_t row, uint32_t first, uint32_t step, uint32_t lane, float x) {
    uint32_t n = 0;
    Cursor<DT> cur(a.sh, row);
    for (uint32_t b = first; b < a.sh.blocks; b += step) {
        const BlockAt at = cur.at(b);
#pragma unroll 1
        for (uint32_t k = lane; k < at.n; k += 64) n += load_logit<DT>(at.p + k * Logit<DT>::kSize) == x;
    }
    return n;
}

// A row's numbers from the joined state of its lanes: called by the whole team,
// with the same `all`.  equal: shared, zero.
template <int DT, typename T, bool TOP>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, uint32_t row, int64_t tok, float tx, const State &all, float log_s,
                                           uint64_t floor_key, uint32_t &equal, typename SharedFor<T, TOP>::type &top) {
    const uint32_t tid = T::id();
    const float nan = __builtin_nanf("");
    const bool token = tok < int64_t(a.vocab);      // tok < 0 never comes here, except for tokens == NULL
    if (!(all.m < kInf)) {
        write_plain_row(a, row, tid, T::kThreads, nan, nan, nan, nan);
        return;
    }
    if (all.m == -kInf) {
        write_plain_row(a, row, tid, T::kThreads, token ? -kInf : nan, 0.0f, -kInf, -kInf);
        return;
    }
    uint32_t candidates = 0;
    if constexpr (TOP) candidates = list_candidates<DT, T>(a, row, floor_key, top);
    Row v;
    v.r = all.r;
    v.l = log_s;
    v.m = all.m;
    v.lse = v.above_largest((v.l - __builtin_fmaf(v.m, a.scale, -v.r)) * kLn2, a);
    v.extreme = false;
    float entropy = (v.l - all.t / all.s) * kLn2;
    if (DT != ROG_DTYPE_F16 && fabsf(all.m) >= a.bound) {
        // Logits this large lie so far apart that any but the largest has
        // probability 0: the row is uniform over the columns that equal it.
        atomicAdd(&equal, count_equal<DT>(a, row, tid / 64, T::kTeamWaves, tid & 63, all.m));
        T::sync();
        v.extreme = true;
        v.l = log2f(float(equal));
        entropy = v.l * kLn2;
        v.lse = __builtin_amdgcn_fmed3f(v.above_largest(entropy, a), -kMaxFinite, kMaxFinite);
    }
    if (tid == T::kThreads - 1) {      // in the last wave, where the first one ranks the alternatives
        if (a.lse) a.lse[row] = v.lse;
        if (a.entropy) a.entropy[row] = entropy;
        if (a.logp) a.logp[row] = token ? v.logp(tx, a) : nan;
    }
    if constexpr (TOP) write_alternatives<T>(a, row, candidates, v, top);
}

// The same from the units' states and the lanes' maxima in shared memory, by a
// workgroup.
template <int DT, bool TOP>
__device__ __forceinline__ void finish_units(const LogprobArgs &a, uint32_t row, int64_t tok, float tx, Shared &sh,
                                             typename SharedFor<Team<kHeadThreads>, TOP>::type &top) {
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const Scaling c{a.scale, a.bound};
    uint64_t floor_key = 0;
    if constexpr (TOP) {
        floor_key = first_floor(fmaxf(fmaxf(sh.lane_m[0][lane], sh.lane_m[1][lane]), fmaxf(sh.lane_m[2][lane], sh.lane_m[3][lane])),
                                a.top_k);
        find_hits<Team<kHeadThreads>>(floor_key, top);
    }
    if (tid < 64) {
        const State all = join_lanes(make_state(sh.m[lane], sh.s[lane], sh.t[lane], c), c);
        if (tid == 0) {
            sh.row[0] = all.m;
            sh.row[1] = all.s;
            sh.row[2] = all.t;
            sh.row[3] = log2f(all.s);
            sh.equal = 0;
        }
    }
    __syncthreads();
    finish_row<DT, Team<kHeadThreads>, TOP>(a, row, tok, tx, make_state(sh.row[0], sh.row[1], sh.row[2], c), sh.row[3], floor_key,
                                            sh.equal, top);
}

// The state of a block of n columns at p from its vectors.
template <int DT>
__device__ __forceinline__ State block_state(gbyte *p, uint32_t n, bool shift, Loaded<Logit<DT>::kVecs> &x, uint32_t lane,
                                             const Scaling &c) {
    if (n < Logit<DT>::kPerVec) return tiny_state<DT>(p, n, lane, c);
    aligned_block<DT>(shift, x);
    if (n < kHeadBlock) mask_tail<DT>(n, lane, x.v);
    return state_of<DT>(x.v, c);
}

// Some of a row's blocks, taken one after the other by one wave with the next
// block's loads in flight: blocks first, first + step, ... of which there are
// `count`.  (Two or three blocks ahead took as long on long rows and 5-15 %
// more where a row has few blocks.)  The first loads go out in the constructor,
// before anything else is known of the row; each(use) calls use(j, state).
template <int DT, bool NT>
struct BlockStream {
    Cursor<DT> cur;
    BlockAt at;
    Loaded<Logit<DT>::kVecs> v;
    uint32_t next, step, count;

    __device__ __forceinline__ BlockStream(const LogprobArgs &a, uint32_t row, uint32_t first, uint32_t by, uint32_t n, uint32_t lane)
        : cur(a.sh, row), next(first + by), step(by), count(n) {
        if (count) {
            at = cur.at(first);
            load_block<DT, NT>(at, lane, v);
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(uint32_t lane, const Scaling &c, F use) {
#pragma unroll 1
        for (uint32_t j = 0; j < count; ++j) {
            const uint32_t n = at.n;
            gbyte *const p = at.p;
            const bool shift = at.shift;
            Loaded<Logit<DT>::kVecs> x = v;
            const bool more = j + 1 < count;
            if (more) at = cur.at(next);
            next += step;
            load_block<DT, NT>(at, lane, v, more);
            use(j, block_state<DT>(p, n, shift, x, lane, c));
        }
    }
};

__device__ __forceinline__ int64_t row_token(const LogprobArgs &a, uint32_t row) { return a.tokens ? a.tokens[row] : 0; }

// One workgroup per row: wave w takes unit w of every chunk, the next block's
// loads in flight while it works on one.
//
// Bound by HBM on many long rows: 4096 x 131072 bf16 over eight shards (1.07 GB)
// take 163-170 us = 6.3-6.6 TB/s, every logit fetched once (counted: 1.002 times
// the bytes), some 8.2 vector instructions an element of which one in ten is an
// exp2: the vector units are busy for about half of that time.  On fewer rows the
// start and the joins show: 893 scored rows of 1021 x 50257 binary16 (90 MB)
// 20.3 us = 4.4 TB/s, 509 x 32003 binary32 with 8 alternatives (65 MB) 16.0.
// Alternatives cost 4000 x 32000 bf16 51 us instead of 45 (8) and 56 (32).
template <int DT, bool TOP, bool NT>
__global__ __launch_bounds__(kHeadThreads) void rog_logprob_row_kernel(LogprobArgs) {
    typedef Team<kHeadThreads> T;
    const LogprobArgs &a = launch_args<LogprobArgs>();
    hold_front(a);
    __shared__ Shared sh;
    __shared__ typename SharedFor<T, TOP>::type top;
    const uint32_t tid = threadIdx.x, lane = tid & 63, w = uniform(tid / 64);
    const Scaling c{a.scale, a.bound};
    const uint32_t row = head_group();
    if (row >= a.rows) return;
    // the loads first: the token only says whether they count
    const uint32_t mine = a.sh.blocks > w ? (a.sh.blocks - w + kChunkUnits - 1) / kChunkUnits : 0;
    BlockStream<DT, NT> blocks(a, row, wave_block(w, 0), kChunkUnits, mine, lane);
    const int64_t tok = row_token(a, row);
    if (tok < 0) {
        write_plain_row(a, row, tid, kHeadThreads, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const float tx = token_logit<DT>(a, row, tok);
    // this wave's places in the tables
    if (lane % kWaves == w) {
        sh.m[lane] = -kInf;
        sh.s[lane] = sh.t[lane] = 0.0f;
    }
    if constexpr (TOP) {
        for (uint32_t e = 0; e < kTopSlots; ++e) top.tab[(w * kTopSlots + e) * 64 + lane] = -kInf;
        if (tid == 0) top.hit_count = top.count = 0;
        if (w == 3) top.places.fill(a, lane);
    }
    State unit = no_state(c);
    float lane_m = -kInf;
    blocks.each(lane, c, [&](uint32_t j, const State &st) {
        if constexpr (TOP) {
            float &e = top.tab[(w * kTopSlots + (j >> a.slot_shift)) * 64 + lane];
            e = max_nan(e, st.m);
            lane_m = max_nan(lane_m, st.m);
        }
        unit = j % kUnitBlocks == 0 ? st : join(unit, st);
        if (j % kUnitBlocks == kUnitBlocks - 1 || j + 1 == mine) {
            State all = join_lanes(unit, c);
            const uint32_t u = j / kUnitBlocks * kChunkUnits + w, slot = u % 64;
            if (u >= 64) all = join(make_state(sh.m[slot], sh.s[slot], sh.t[slot], c), all);
            if (lane == 0) {
                sh.m[slot] = all.m;
                sh.s[slot] = all.s;
                sh.t[slot] = all.t;
            }
        }
    });
    if constexpr (TOP) sh.lane_m[w][lane] = lane_m;
    __syncthreads();
    finish_units<DT, TOP>(a, row, tok, tx, sh, top);
}

// A row over several workgroups, a unit each, a block per wave; the last one of
// the row to finish joins the units' states.
//
// Bound by the chain of latencies, not by bytes: one row of 131072 bf16 columns
// takes 5.1 us, 8.3-8.7 with 5 alternatives.  The chain: kernel arguments 0.6 us, a
// block's loads and sums 1.2, states published and counted 0.7, collected 1,
// joined 1; for alternatives the candidates' columns again 1.7 and their ranks
// 0.6 (the rest is the launch itself).  A workgroup adds some 3 ns: 64 such rows
// take 8.5 us, with 20 alternatives 13.4, over eight shards and masked 14.4.  A wave
// per unit in place of a block per wave took 64 rows 9.4 us.
template <int DT, bool TOP>
__global__ __launch_bounds__(kHeadThreads) void rog_logprob_split_kernel(LogprobArgs) {
    typedef Team<kHeadThreads> T;
    const LogprobArgs &a = launch_args<LogprobArgs>();
    hold_front(a);
    __shared__ Shared sh;
    __shared__ typename SharedFor<T, TOP>::type top;
    const uint32_t tid = threadIdx.x, lane = tid & 63, w = uniform(tid / 64);
    const Scaling c{a.scale, a.bound};
    const uint32_t group = head_group();
    const uint32_t row = group / a.units, u = group % a.units;
    if (row >= a.rows) return;
    const uint32_t first = u / kChunkUnits * kChunkBlocks + u % kChunkUnits, b = first + w * kChunkUnits;
    // the loads first: the token only says whether they count
    Loaded<Logit<DT>::kVecs> v;
    BlockAt at;
    if (b < a.sh.blocks) {
        at = Cursor<DT>(a.sh, row).at(b);
        load_block<DT, false>(at, lane, v);
    }
    const int64_t tok = row_token(a, row);
    if (tok < 0) {
        if (u == 0) write_plain_row(a, row, tid, kHeadThreads, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const float tx = token_logit<DT>(a, row, tok);
    float *const states = a.part + uint64_t(row) * a.units * kUnitFloats;   // [unit][4]
    float *const maxima = states + a.units * 4;                             // [unit][entry][lane]
    // entries of a unit in the table: as many as its blocks, or fewer, wider ones
    const uint32_t entry_shift = min(a.slot_shift, 2u), entry_log = 2 - entry_shift, entries = 1u << entry_log;
    State st = no_state(c);
    if (b < a.sh.blocks) st = block_state<DT>(at.p, at.n, at.shift, v, lane, c);
    sh.lane_m[w][lane] = st.m;
    sh.lane_s[w][lane] = st.s;
    sh.lane_t[w][lane] = st.t;
    __syncthreads();
    if (w == 0) {
        State unit = st;
#pragma unroll
        for (uint32_t i = 1; i < kUnitBlocks; ++i)
            if (first + i * kChunkUnits < a.sh.blocks)
                unit = join(unit, make_state(sh.lane_m[i][lane], sh.lane_s[i][lane], sh.lane_t[i][lane], c));
        const State all = join_lanes(unit, c);
        if (lane < 3) publish(states + u * 4 + lane, lane == 0 ? all.m : lane == 1 ? all.s : all.t);
    } else if (TOP && w == 1) {
        for (uint32_t e = 0; e < entries; ++e) {
            float m = sh.lane_m[e << entry_shift][lane];
            for (uint32_t i = 1; i < 1u << entry_shift; ++i) m = max_nan(m, sh.lane_m[(e << entry_shift) + i][lane]);
            publish(maxima + (u * entries + e) * 64 + lane, m);
        }
    }
    if (!last_to_arrive(a.counters + row * kCounterStride, a.units, sh.last)) return;
    // one round trip: the first 64 units' states, and of the maxima as many as the table has entries
    float jm = -kInf, js = 0.0f, jt = 0.0f;
    if (w == 0 && lane < a.units) {
        jm = collect(states + lane * 4);
        js = collect(states + lane * 4 + 1);
        jt = collect(states + lane * 4 + 2);
    }
    if constexpr (TOP) {
        float lane_m = -kInf;
        const uint32_t all = a.chunks * entries;      // this wave's units' entries
        const bool alone = a.slot_shift <= 2;         // one entry per slot of the table
        if (!alone) {
            for (uint32_t e = 0; e < kTopSlots; ++e) top.tab[(w * kTopSlots + e) * 64 + lane] = -kInf;
        }
        for (uint32_t k0 = 0; k0 < all || k0 == 0; k0 += kTopSlots) {
            float m[kTopSlots];
#pragma unroll
            for (uint32_t i = 0; i < kTopSlots; ++i) {
                const uint32_t k = k0 + i, q = (k >> entry_log) * kChunkUnits + w;
                m[i] = -kInf;
                if (k < all && q < a.units) m[i] = collect(maxima + (q * entries + (k & (entries - 1))) * 64 + lane);
            }
#pragma unroll
            for (uint32_t i = 0; i < kTopSlots; ++i) {
                lane_m = max_nan(lane_m, m[i]);
                if (alone) {
                    top.tab[(w * kTopSlots + i) * 64 + lane] = m[i];
                } else if (k0 + i < all) {
                    float &slot = top.tab[(w * kTopSlots + (((k0 + i) << entry_shift) >> a.slot_shift)) * 64 + lane];
                    slot = max_nan(slot, m[i]);
                }
            }
        }
        sh.lane_m[w][lane] = lane_m;
        if (w == 1) top.places.fill(a, lane);
        if (tid == 0) top.hit_count = top.count = 0;
    }
    if (w == 0) {
        State joined = make_state(jm, js, jt, c);
        for (uint32_t q = lane + 64; q < a.units; q += 64)
            joined = join(joined, make_state(collect(states + q * 4), collect(states + q * 4 + 1), collect(states + q * 4 + 2), c));
        sh.m[lane] = joined.m;
        sh.s[lane] = joined.s;
        sh.t[lane] = joined.t;
    }
    __syncthreads();
    finish_units<DT, TOP>(a, row, tok, tx, sh, top);
}

// One wave per row of at most four blocks: a single unit.  Four rows to a
// workgroup share nothing.  Bound by HBM and the launch: 8627 x 8192 bf16 (141 MB,
// streamed) take 26.2 us = 5.4 TB/s, of which some 5 us are the launch's start and
// end; 10000 x 8192 29 us, with 8 alternatives 35.8.
template <int DT, bool TOP, bool NT>
__global__ __launch_bounds__(64 * kWaveRows) void rog_logprob_wave_kernel(LogprobArgs) {
    typedef Team<64> T;
    const LogprobArgs &a = launch_args<LogprobArgs>();
    hold_front(a);
    __shared__ uint32_t equal[kWaveRows];
    __shared__ typename SharedFor<T, TOP>::type top[kWaveRows];
    const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64);
    const Scaling c{a.scale, a.bound};
    const uint32_t row = head_group() * kWaveRows + w;
    if (row >= a.rows) return;
    BlockStream<DT, NT> blocks(a, row, 0, 1, a.sh.blocks, lane);
    const int64_t tok = row_token(a, row);
    if (tok < 0) {
        write_plain_row(a, row, lane, 64, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const float tx = token_logit<DT>(a, row, tok);
    State unit = no_state(c);
    if constexpr (TOP) {
        Cursor<DT> cur(a.sh, row);
        for (uint32_t b = 0; b < a.sh.blocks; ++b) {
            const BlockAt at = cur.at(b);
            if (lane == 0) top[w].places.set(b, at);
        }
    }
    blocks.each(lane, c, [&](uint32_t b, const State &st) {
        if constexpr (TOP) top[w].tab[b * 64 + lane] = st.m;
        unit = b == 0 ? st : join(unit, st);
    });
    if constexpr (TOP) {
        for (uint32_t b = a.sh.blocks; b < kUnitBlocks; ++b) top[w].tab[b * 64 + lane] = -kInf;
    }
    const State all = join_lanes(unit, c);
    uint64_t floor_key = 0;
    if (lane == 0) equal[w] = 0;
    if constexpr (TOP) {
        if (lane == 0) top[w].hit_count = top[w].count = 0;
        T::sync();
        floor_key = first_floor(unit.m, a.top_k);
        find_hits<T>(floor_key, top[w]);
    }
    T::sync();
    finish_row<DT, T, TOP>(a, row, tok, tx, all, log2f(all.s), floor_key, equal[w], top[w]);
}

template <typename K>
const void *kfn(K *k) { return reinterpret_cast<const void *>(k); }

template <int DT>
const void *logprob_kernel(const LogprobPlan &p) {
    const bool top = p.args.top_ids || p.args.top_logp, nt = p.nt_loads;
    switch (p.info.form) {
    case ROG_LOGPROB_SPLIT: return top ? kfn(&rog_logprob_split_kernel<DT, true>) : kfn(&rog_logprob_split_kernel<DT, false>);
    case ROG_LOGPROB_WAVE:
        return top ? (nt ? kfn(&rog_logprob_wave_kernel<DT, true, true>) : kfn(&rog_logprob_wave_kernel<DT, true, false>))
                   : (nt ? kfn(&rog_logprob_wave_kernel<DT, false, true>) : kfn(&rog_logprob_wave_kernel<DT, false, false>));
    default:
        return top ? (nt ? kfn(&rog_logprob_row_kernel<DT, true, true>) : kfn(&rog_logprob_row_kernel<DT, true, false>))
                   : (nt ? kfn(&rog_logprob_row_kernel<DT, false, true>) : kfn(&rog_logprob_row_kernel<DT, false, false>));
    }
}

rog_status launch_logprob(LogprobPlan &p, hipStream_t stream) {
    const void *k = p.dtype == ROG_DTYPE_BF16  ? logprob_kernel<ROG_DTYPE_BF16>(p)
                    : p.dtype == ROG_DTYPE_F16 ? logprob_kernel<ROG_DTYPE_F16>(p)
                                               : logprob_kernel<ROG_DTYPE_F32>(p);
    void *params[] = {&p.args};
    const hipError_t e = hipLaunchKernel(k, head_grid(p.info.grid), dim3(p.info.block), params, 0, stream);
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
