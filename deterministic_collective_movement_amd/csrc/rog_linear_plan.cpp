// rog_linear_plan.cpp -- argument validation, tiles and workspaces of the policy
// head's products.  Pure host code: no HIP calls, so every decision here can be
// checked on a machine without a GPU.
#include <math.h>

#include <algorithm>

#include "rog_head_checks.h"
#include "rog_linear.h"

namespace rog {
namespace {

constexpr uint64_t kMaxGroups = uint64_t(1) << 22;   // workgroups of a launch (of 512 threads, below 2^32 work-items)
constexpr float kMinTemperature = 1.0f / 1024, kMaxTemperature = 1024.0f;
constexpr double kLog2E = 1.4426950408889634;

// Bytes behind a row of coefficients, whose own are a multiple of 512: with rows 2^16 bytes apart a tile's
// rows fall on few of the memory's channels (4096 rows of 65536 x 4096: 5.78 ms without, 5.24 with 256,
// 5.29 / 5.51 / 5.32 with 128 / 512 / 1024).
constexpr uint64_t kRowPad = 256;
// Large tiles up to which 128 x 128 ones are taken instead: half of the CUs or fewer would be at work (200 rows of
// 32000 x 2048 56.5 us with 125 large tiles, 50.1 with 500; 600 rows of 16000 x 2048 60 with 189, 68 with 625).
constexpr uint64_t kMidTiles = 128;

inline bool product_type(rog_dtype t) { return t == ROG_DTYPE_BF16 || t == ROG_DTYPE_F16; }
inline uint64_t up(uint64_t v, uint64_t unit) { return ceil_div(v, unit) * unit; }

// A matrix of `rows` rows of `width` elements: address, stride and extent; `bytes` gets its stride in bytes (one row
// has none).
rog_status check_matrix(const void *p, int64_t stride, uint64_t rows, uint64_t width, uint32_t es, bool spread, int64_t *bytes) {
    if (stride < 0) return ROG_ERR_INVALID_ARGUMENT;
    if (rows && width && (!p || addr(p) % es)) return ROG_ERR_INVALID_ARGUMENT;
    if (rows <= 1) stride = 0;
    if (spread && rows > 1 && uint64_t(stride) < width) return ROG_ERR_INVALID_ARGUMENT;
    if (uint64_t(stride) >= kMaxLinearStride / es) return ROG_ERR_TOO_LARGE;
    *bytes = stride * es;
    return fits(addr(p), rows, uint64_t(*bytes), width * es) ? ROG_OK : ROG_ERR_TOO_LARGE;
}

// Loads of 16 bytes go straight to the shared memory from rows that begin on 4 bytes.
bool aligned(const void *p, uint64_t stride_bytes) { return (addr(p) | stride_bytes) % 4 == 0; }

template <class Shard>
rog_status lay_weights(const Shard *shards, int W, int64_t dim, uint32_t es, bool addresses, WeightShards *h, bool *direct) {
    if (!shards || W < 1 || W > kMaxPeers || dim < 1) return ROG_ERR_INVALID_ARGUMENT;
    if (uint64_t(dim) >= kMaxDim) return ROG_ERR_TOO_LARGE;
    uint64_t v = 0;
    for (int r = 0; r < W; ++r) {
        if (shards[r].width < 0) return ROG_ERR_INVALID_ARGUMENT;
        if (uint64_t(shards[r].width) >= kMaxVocab || v + uint64_t(shards[r].width) >= kMaxVocab) return ROG_ERR_TOO_LARGE;
        int64_t stride = 0;
        if (addresses) {
            const rog_status st = check_matrix(shards[r].weight, shards[r].row_stride, uint64_t(shards[r].width), uint64_t(dim), es, false, &stride);
            if (st != ROG_OK) return st;
        }
        h->s[r] = WeightShard{shards[r].weight, stride, uint32_t(shards[r].width), uint32_t(v)};
        if (shards[r].width && !aligned(shards[r].weight, uint64_t(stride))) *direct = false;
        v += uint64_t(shards[r].width);
    }
    h->W = uint32_t(W);
    h->vocab = uint32_t(v);
    return ROG_OK;
}

void lay_tiles(WeightShards *h, uint32_t tile) {
    uint32_t t = 0, b = 0;
    for (uint32_t r = 0; r < h->W; ++r) {
        h->tile0[r] = t;
        h->block0[r] = b;
        t += uint32_t(ceil_div(h->s[r].width, tile));
        b += uint32_t(ceil_div(h->s[r].width, kLinearBlock));
    }
    h->tile0[h->W] = t;
    h->block0[h->W] = b;
}

// The tile for so many rows.
int32_t form_of(uint64_t rows, const WeightShards &h) {
    if (rows <= FormSome::kRows) return rows <= FormFew::kRows ? kFormFew : kFormSome;
    uint64_t wide = 0;
    for (uint32_t r = 0; r < h.W; ++r) wide += ceil_div(h.s[r].width, FormWide::kColumns);
    wide *= ceil_div(rows, FormWide::kRows);
    return rows <= FormMid::kRows || wide <= kMidTiles ? kFormMid : kFormWide;
}
constexpr uint32_t kFormColumns[] = {FormFew::kColumns, FormSome::kColumns, FormMid::kColumns, FormWide::kColumns};
constexpr uint32_t kFormRows[] = {FormFew::kRows, FormSome::kRows, FormMid::kRows, FormWide::kRows};
uint32_t tile_columns(int32_t form) { return kFormColumns[form]; }
uint32_t tile_rows(int32_t form) { return kFormRows[form]; }

// Workgroups for so many tiles: the wide form deals some of them out in quarters, by the rows that there turn out to be.
uint64_t groups_of(uint64_t tiles, int32_t form) { return form == kFormWide && tiles ? tiles + 3 * kTailSplit : tiles; }

// Cubes of 256 rows x 256 columns x 256 elements up to which the mid form is taken, and the same for up to 128 rows.  There the
// crossing lies between 1000 and 3000 cubes, lower for narrow states (us, mid and wide: 128 x 28672 x 1024, 448 cubes,
// 77 and 118; 70 x 50257 x 1000 binary16, 788, 126 and 123; 100 x 32000 x 2048, 1000, 121 and 210; 70 x 50257 x 1600
// binary16, 1379, 166 and 148; 128 x 50257 x 2048, 1576, 216 and 260; 100 x 32000 x 4096, 2000, 275 and 312;
// 128 x 131072 x 1024, 2048, 294 and 248; 100 x 50257 x 4096, 3152, 431 and 345; 100 x 131072 x 2048, 4096, 561 and 475).
constexpr uint64_t kMidCubes = 224, kMidCubesFew = 1024;
// Rows from which the scored ones are packed: few rows are one tile whether scored or not, and a launch is 4 us more;
// of many the tiles of rows that do not count are saved (8192 x 4096: 25 us, where every eighth row that does not count
// takes an eighth of 6.5 ms with it).
constexpr uint64_t kPackFrom = 65;

// A workspace, laid out front to back: behind the arrival counters of the other operators, which stay zero.
struct Layout {
    uint64_t at = kHeadCounterBytes;
    uint64_t take(uint64_t bytes) {
        const uint64_t p = at;
        at = up(at + bytes, 256);
        return p;
    }
};
template <class T>
T *in(void *workspace, uint64_t at) { return reinterpret_cast<T *>(static_cast<char *>(workspace) + at); }

Strip matrix(const void *p, uint64_t rows, int64_t stride_bytes, uint64_t row_bytes) {
    return Strip{addr(p), rows, uint64_t(stride_bytes), row_bytes};
}

}  // namespace

rog_status plan_linear_logprob(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim, const rog_weight_shard *shards, int W,
                               rog_dtype dtype, float temperature, const int64_t *tokens, const rog_logprob_out *out, void *workspace,
                               size_t workspace_bytes, bool addresses, bool has_tokens, ScorePlan *p) {
    if (!product_type(dtype)) return ROG_ERR_INVALID_ARGUMENT;
    if (!(temperature >= kMinTemperature && temperature <= kMaxTemperature)) return ROG_ERR_INVALID_ARGUMENT;
    ScoreArgs &a = p->args;
    p->direct = true;
    rog_status st = lay_weights(shards, W, dim, 2, addresses, &a.sh, &p->direct);
    if (st != ROG_OK) return st;
    if (rows >= kMaxVocab) return ROG_ERR_TOO_LARGE;
    int64_t h_stride = 0;
    if (addresses) st = check_matrix(hidden, hidden_stride, rows, uint64_t(dim), 2, false, &h_stride);
    if (st != ROG_OK) return st;
    p->form = form_of(rows, a.sh);
    p->packs = has_tokens && rows >= kPackFrom;
    lay_tiles(&a.sh, tile_columns(p->form));
    const uint64_t kbytes = uint64_t(dim) * 2, packed = up(kbytes, kPackUnit);
    if (!p->packs && !aligned(hidden, uint64_t(h_stride))) p->direct = false;
    const uint64_t groups = groups_of(a.sh.tile0[W] * ceil_div(rows, tile_rows(p->form)), p->form);
    // the join has 64 threads per row, of whole workgroups of 16 rows: a dispatch counts work-items in 32 bits
    if (groups >= kMaxGroups || up(rows, 16) * 64 >= uint64_t(1) << 32) return ROG_ERR_TOO_LARGE;
    p->grid = uint32_t(groups);
    const uint32_t blocks = a.sh.block0[W], rows_pad = uint32_t(up(rows, 16));
    // a row's states together where a wave joins a row, else a block's
    a.row_step = p->form == kFormWide ? 1 : blocks;
    a.block_step = p->form == kFormWide ? rows_pad : 1;
    Layout w;
    const uint64_t target = w.take(rows * 4), rests = w.take(rows * 16), states = w.take(uint64_t(blocks) * rows_pad * 16);
    const uint64_t index = w.take(p->packs ? rows * 4 : 0), count = w.take(p->packs ? 4 : 0), rows_at = w.take(p->packs ? rows * packed : 0);
    p->workspace_bytes = rows ? w.at : 0;
    if (rows == 0 || !addresses) return ROG_OK;

    if (!out || out->top_logp || out->top_ids || (out->logp && !tokens)) return ROG_ERR_INVALID_ARGUMENT;
    if (addr(tokens) % 8 || (addr(out->logp) | addr(out->entropy) | addr(out->lse)) % 4) return ROG_ERR_INVALID_ARGUMENT;
    if (!workspace || addr(workspace) % 16 || workspace_bytes < p->workspace_bytes) return ROG_ERR_INVALID_ARGUMENT;
    const Strip outs[4] = {flat(out->logp, out->logp ? rows * 4 : 0), flat(out->entropy, out->entropy ? rows * 4 : 0),
                           flat(out->lse, out->lse ? rows * 4 : 0), flat(workspace, p->workspace_bytes)};
    for (int i = 0; i < 4; ++i) {
        if (outs[i].at > UINTPTR_MAX - outs[i].width) return ROG_ERR_TOO_LARGE;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ROG_ERR_OVERLAP;
        if (tokens && overlap(outs[i], flat(tokens, rows * 8))) return ROG_ERR_OVERLAP;
        if (overlap(outs[i], matrix(hidden, rows, h_stride, kbytes))) return ROG_ERR_OVERLAP;
        for (int r = 0; r < W; ++r)
            if (overlap(outs[i], matrix(a.sh.s[r].w, a.sh.s[r].width, a.sh.s[r].stride, kbytes))) return ROG_ERR_OVERLAP;
    }
    a.a = LinearRows{hidden, h_stride, nullptr, uint32_t(rows), uint32_t(kbytes)};
    a.tokens = tokens;
    a.index = nullptr;
    a.scale = float(kLog2E / double(temperature));
    a.target = in<float>(workspace, target);
    a.rests = in<float>(workspace, rests);
    a.states = in<float>(workspace, states);
    if (p->packs) {
        p->pack = PackArgs{};
        p->pack.x = hidden;
        p->pack.stride = h_stride;
        p->pack.tokens = tokens;
        p->pack.rows = uint32_t(rows);
        p->pack.kbytes = uint32_t(kbytes);
        p->pack.packed_bytes = uint32_t(packed);
        p->pack.index = in<uint32_t>(workspace, index);
        p->pack.count = in<uint32_t>(workspace, count);
        p->pack.packed = in<void>(workspace, rows_at);
        p->pack.logp = out->logp;
        p->pack.entropy = out->entropy;
        p->pack.lse = out->lse;
        a.a = LinearRows{p->pack.packed, int64_t(packed), p->pack.count, uint32_t(rows), uint32_t(kbytes)};
        a.index = p->pack.index;
    }
    p->join = JoinArgs{tokens, a.index, a.a.count, a.target, a.rests, a.states, out->logp, out->entropy, out->lse, uint32_t(rows), a.row_step,
                       a.block_step, a.sh.vocab, blocks, a.scale};
    return ROG_OK;
}

rog_status plan_linear_grad(const void *hidden, int64_t hidden_stride, size_t rows, int64_t dim, const rog_weight_shard *shards, int W,
                            rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse, const float *entropy,
                            const float *g_logp, const float *g_entropy, void *d_hidden, int64_t d_hidden_stride,
                            const rog_grad_shard *d_weights, void *workspace, size_t workspace_bytes, bool addresses, GradPlan *p) {
    if (!product_type(dtype)) return ROG_ERR_INVALID_ARGUMENT;
    if (!(temperature >= kMinTemperature && temperature <= kMaxTemperature)) return ROG_ERR_INVALID_ARGUMENT;
    GradArgs &a = p->coef;
    BackArgs &k = p->back;
    p->dtype = dtype;
    p->direct = true;
    rog_status st = lay_weights(shards, W, dim, 2, addresses, &a.sh, &p->direct);
    if (st != ROG_OK) return st;
    if (a.sh.vocab == 0) return ROG_ERR_INVALID_ARGUMENT;
    if (rows >= kMaxVocab) return ROG_ERR_TOO_LARGE;
    int64_t h_stride = 0;
    if (addresses) st = check_matrix(hidden, hidden_stride, rows, uint64_t(dim), 2, false, &h_stride);
    if (st != ROG_OK) return st;
    lay_tiles(&a.sh, kGradTile);
    const uint64_t kbytes = uint64_t(dim) * 2, packed = up(kbytes, kPackUnit);
    p->form = rows > FormSome::kRows ? kFormWide : rows > FormFew::kRows ? kFormSome : kFormFew;
    // Little work is spread wider in the small tiles, and up to 128 rows leave half of a large one empty (us, mid and
    // wide: 544 x 5830 x 128 40 and 51, 243 x 1020 x 384 30 and 45, 1024 x 16000 x 256 85 and 66,
    // 100 x 32000 x 2048 121 and 207, 128 x 131072 x 4096 1112 and 865).
    if (p->form == kFormWide && ceil_div(rows, 256) * a.sh.tile0[W] * ceil_div(uint64_t(dim), 256) <= (rows <= 128 ? kMidCubesFew : kMidCubes))
        p->form = kFormMid;
    const uint32_t bn = p->form == kFormWide ? 256 : 64;
    k = BackArgs{};
    k.sh = a.sh;
    k.dim = uint32_t(dim);
    k.dim_pad = uint32_t(up(uint64_t(dim), 64));
    k.dim_tiles = uint32_t(ceil_div(uint64_t(dim), 256));
    k.row_tiles = uint32_t(ceil_div(rows, bn));
    // Segments go by the width of the states alone, so that the sums' order does: a segment's sums go through memory,
    // which costs large batches of narrow states most, while short segments are short chains for small batches (us, of
    // half these tiles and of these: 8192 x 32000 x 320 911 and 854, 544 x 5830 x 128 37 and 40).
    k.seg_tiles = dim >= 2048 ? 32 : dim >= 512 ? 16 : 8;
    uint32_t segs = 0;
    for (int r = 0; r < W; ++r) {
        k.seg0[r] = segs;
        segs += uint32_t(ceil_div(a.sh.tile0[r + 1] - a.sh.tile0[r], k.seg_tiles));
    }
    k.seg0[W] = segs;
    // A tile's sums stay with one workgroup for all of a piece's segments where there are enough tiles for that (us, from
    // 64 and from 128 tiles: 8192 x 50257 x 768, of 96, 2636 and 2374).
    p->running = p->form == kFormWide && uint64_t(k.dim_tiles) * k.row_tiles >= 128;
    // Pieces are runs of whole segments: as many as the bytes allow.
    p->piece_tiles = piece_tiles(rows, k.seg_tiles);
    // Count them as lay_piece() walks.
    p->pieces = 0;
    uint32_t most_tiles = 0, most_segs = 0;
    for (uint32_t s = 0; s < segs;) {
        uint32_t t = 0, n = 0;
        for (int r = 0; r < W && s < segs; ++r)
            while (s >= k.seg0[r] && s < k.seg0[r + 1]) {
                const uint32_t left = a.sh.tile0[r + 1] - a.sh.tile0[r] - (s - k.seg0[r]) * k.seg_tiles, here = std::min(left, k.seg_tiles);
                if (n && t + here > p->piece_tiles) goto full;
                t += here;
                ++n;
                ++s;
            }
    full:
        most_tiles = std::max(most_tiles, t);
        most_segs = std::max(most_segs, n);
        ++p->pieces;
    }
    const uint64_t coef_groups = uint64_t(most_tiles) * k.row_tiles * 2 + 3 * kTailSplit;   // of any form's at most
    const uint64_t back_groups = uint64_t(p->running ? 1 : most_segs) * k.dim_tiles * 4 * k.row_tiles + uint64_t(k.dim_tiles) * most_tiles * 4 + kCus;
    // The weights' sums over many rows are cut where their tiles leave CUs idle, into the more the more rows are scored.
    k.splits = weight_parts(uint32_t(rows), k.dim_tiles, a.sh.tile0[W], k.seg_tiles);
    if (coef_groups >= kMaxGroups || back_groups >= kMaxGroups) return ROG_ERR_TOO_LARGE;
    Layout w;
    const uint64_t index = w.take(rows * 4), count = w.take(4), g_scale = w.take(4), parts = w.take(4), rows_at = w.take(rows * packed);
    const uint64_t g_row = uint64_t(most_tiles) * kGradTile * 2 + kRowPad, g_bytes = rows * g_row;
    const uint64_t g = w.take(g_bytes), g_all = dtype == ROG_DTYPE_F16 ? w.take(g_bytes) : g;
    const uint64_t seg_floats = rows * uint64_t(k.dim_pad);
    const uint64_t part = w.take(p->running ? 0 : seg_floats * 4 * most_segs), running = w.take(p->running || p->pieces > 1 ? seg_floats * 4 : 0);
    const uint64_t split_floats = uint64_t(most_tiles) * kGradTile * k.dim_pad, dw_part = w.take(k.splits > 1 ? split_floats * 4 * k.splits : 0);
    p->workspace_bytes = rows ? w.at : 0;
    if (rows == 0 || !addresses) return ROG_OK;

    if (!tokens || !lse || !entropy || !g_logp || !d_weights || addr(tokens) % 8 ||
        (addr(lse) | addr(entropy) | addr(g_logp) | addr(g_entropy)) % 4)
        return ROG_ERR_INVALID_ARGUMENT;
    int64_t d_stride = 0;
    st = check_matrix(d_hidden, d_hidden_stride, rows, uint64_t(dim), 2, true, &d_stride);
    if (st != ROG_OK) return st;
    if (!workspace || addr(workspace) % 16 || workspace_bytes < p->workspace_bytes) return ROG_ERR_INVALID_ARGUMENT;
    const Strip work = flat(workspace, p->workspace_bytes), dh = matrix(d_hidden, rows, d_stride, kbytes);
    if (work.at > UINTPTR_MAX - work.width) return ROG_ERR_TOO_LARGE;
    const Strip x = matrix(hidden, rows, h_stride, kbytes);
    const Strip vectors[5] = {flat(lse, rows * 4), flat(entropy, rows * 4), flat(g_logp, rows * 4),
                              flat(g_entropy, g_entropy ? rows * 4 : 0), flat(tokens, rows * 8)};
    if (overlap(work, dh) || overlap(work, x) || overlap(dh, x)) return ROG_ERR_OVERLAP;
    for (const Strip &v : vectors)
        if (overlap(work, v) || overlap(dh, v)) return ROG_ERR_OVERLAP;
    for (int r = 0; r < W; ++r) {
        const uint64_t width = a.sh.s[r].width;
        if (width) {
            st = check_matrix(d_weights[r].grad, d_weights[r].row_stride, width, uint64_t(dim), 2, true, &k.dw_stride[r]);
            if (st != ROG_OK) return st;
        }
        k.dw[r] = d_weights[r].grad;
        const Strip dw = matrix(k.dw[r], width, k.dw_stride[r], kbytes), wr = matrix(a.sh.s[r].w, width, a.sh.s[r].stride, kbytes);
        if (overlap(dw, work) || overlap(dw, dh) || overlap(dw, x) || overlap(wr, work) || overlap(wr, dh)) return ROG_ERR_OVERLAP;
        for (const Strip &v : vectors)
            if (overlap(dw, v)) return ROG_ERR_OVERLAP;
        for (int q = 0; q < W; ++q)
            if (overlap(dw, matrix(a.sh.s[q].w, a.sh.s[q].width, a.sh.s[q].stride, kbytes)) ||
                (q < r && overlap(dw, matrix(k.dw[q], a.sh.s[q].width, k.dw_stride[q], kbytes))))
                return ROG_ERR_OVERLAP;
    }

    PackArgs &c = p->pack;
    c = PackArgs{};
    c.x = hidden;
    c.stride = h_stride;
    c.tokens = tokens;
    c.rows = uint32_t(rows);
    c.kbytes = uint32_t(kbytes);
    c.packed_bytes = uint32_t(packed);
    c.index = in<uint32_t>(workspace, index);
    c.count = in<uint32_t>(workspace, count);
    c.packed = in<void>(workspace, rows_at);
    c.zero = d_hidden;
    c.zero_stride = d_stride;
    c.parts = k.splits > 1 ? in<uint32_t>(workspace, parts) : nullptr;
    c.dim_tiles = k.dim_tiles;
    c.tiles = a.sh.tile0[W];
    c.seg_tiles = k.seg_tiles;
    c.g_logp = g_logp;
    c.g_entropy = g_entropy;
    c.g_scale = dtype == ROG_DTYPE_F16 ? in<float>(workspace, g_scale) : nullptr;
    c.inv_t = float(1.0 / double(temperature));
    a.a = LinearRows{c.packed, int64_t(packed), c.count, uint32_t(rows), uint32_t(kbytes)};
    a.tokens = tokens;
    a.index = c.index;
    a.lse = lse;
    a.entropy = entropy;
    a.g_logp = g_logp;
    a.g_entropy = g_entropy;
    a.g_scale = c.g_scale;
    a.inv_t = c.inv_t;
    a.scale = float(kLog2E / double(temperature));
    a.g = in<void>(workspace, g);
    a.g_all = in<void>(workspace, g_all);
    a.g_stride = int64_t(g_row);
    k.a = a.a;
    k.index = a.index;
    k.g_logp = g_logp;
    k.g_entropy = g_entropy;
    k.g_scale = a.g_scale;
    k.inv_t = c.inv_t;
    k.g = a.g;
    k.g_all = a.g_all;
    k.g_stride = a.g_stride;
    k.part = in<float>(workspace, p->running ? running : part);
    k.part_seg = p->running ? 0 : seg_floats;
    k.parts = c.parts;
    k.dw_part = in<float>(workspace, dw_part);
    k.dw_part_split = split_floats;
    // along rows, where a row's end inside 16 bytes would be read past, only whole ones
    p->direct_back = p->direct && kbytes % 16 == 0;
    k.d_hidden = d_hidden;
    k.d_stride = d_stride;
    if (!p->running) {
        if (ceil_div(rows * (k.dim_pad / 8), 256) >= uint64_t(1) << 24) return ROG_ERR_TOO_LARGE;
        p->join = BackJoinArgs{k.part, in<float>(workspace, running), k.part_seg, 0, k.dim_pad, k.dim, 0, 0, k.index, c.count,
                               g_logp, g_entropy, c.inv_t, uint32_t(rows), d_hidden, k.d_stride};
    }
    a.tile_begin = a.tiles = k.seg_begin = k.segs = 0;
    return ROG_OK;
}

PieceGrid lay_piece(GradPlan *p, uint32_t i) {
    GradArgs &a = p->coef;
    BackArgs &k = p->back;
    const uint32_t W = a.sh.W, segs = k.seg0[W];
    uint32_t s = k.seg_begin + k.segs;          // where the last piece ended
    k.tile_begin = a.tile_begin + a.tiles;
    k.seg_begin = s;
    k.segs = k.tiles = 0;
    for (uint32_t r = 0; r < W && s < segs; ++r)
        while (s >= k.seg0[r] && s < k.seg0[r + 1]) {
            const uint32_t left = a.sh.tile0[r + 1] - a.sh.tile0[r] - (s - k.seg0[r]) * k.seg_tiles, here = std::min(left, k.seg_tiles);
            if (k.segs && k.tiles + here > p->piece_tiles) goto full;
            k.tiles += here;
            ++k.segs;
            ++s;
        }
full:
    k.first = i == 0;
    k.last = s == segs;
    a.tile_begin = k.tile_begin;
    a.tiles = k.tiles;
    PieceGrid g = {};
    if (p->form == kFormWide) {
        g.coefficients = uint32_t(groups_of(uint64_t(k.tiles) * k.row_tiles, p->form));
        g.states = (p->running ? 1 : k.segs) * k.dim_tiles * k.row_tiles;
        g.weights = k.dim_tiles * k.tiles;
    } else {
        g.coefficients = k.tiles * 2 * uint32_t(ceil_div(k.a.rows, tile_rows(p->form)));
        g.states = k.segs * uint32_t(ceil_div(k.dim, 64)) * k.row_tiles;
        g.weights = uint32_t(ceil_div(k.dim, 128)) * k.tiles * 2;
    }
    g.weights *= k.splits;
    if (k.splits > 1) g.weights_join = uint32_t(ceil_div(uint64_t(k.tiles) * kGradTile * (k.dim_pad / 8), 256));
    if (!p->running) {
        p->join.segs = k.segs;
        p->join.first = k.first;
        p->join.last = k.last;
        g.join = uint32_t(ceil_div(k.a.rows * uint64_t(k.dim_pad / 8), 256));
    }
    return g;
}

rog_status plan_quantize(const void *x, int64_t row_stride, size_t rows, int64_t dim, rog_dtype dtype, int8_t *q, int64_t q_stride,
                         float *scale, QuantizeArgs *a) {
    if (!known(dtype) || dim < 1) return ROG_ERR_INVALID_ARGUMENT;
    if (rows >= uint64_t(1) << 23 || uint64_t(dim) >= kMaxDim) return ROG_ERR_TOO_LARGE;
    const uint32_t es = esize(dtype);
    int64_t x_bytes = 0, q_bytes = 0;
    rog_status st = check_matrix(x, row_stride, rows, uint64_t(dim), es, false, &x_bytes);
    if (st == ROG_OK) st = check_matrix(q, q_stride, rows, uint64_t(dim), 1, true, &q_bytes);
    if (st != ROG_OK || rows == 0) return st;
    if (!scale || addr(scale) % 4) return ROG_ERR_INVALID_ARGUMENT;
    const Strip xs = matrix(x, rows, x_bytes, uint64_t(dim) * es), qs = matrix(q, rows, q_bytes, uint64_t(dim)), s = flat(scale, rows * 4);
    if (s.at > UINTPTR_MAX - s.width) return ROG_ERR_TOO_LARGE;
    if (overlap(xs, qs) || overlap(xs, s) || overlap(qs, s)) return ROG_ERR_OVERLAP;
    *a = QuantizeArgs{x, x_bytes, q, q_bytes, scale, uint32_t(rows), uint32_t(dim)};
    return ROG_OK;
}

rog_status plan_linear_i8(const int8_t *q, int64_t q_stride, const float *scale, size_t rows, int64_t dim, const rog_i8_shard *shards, int W,
                          rog_dtype out_dtype, const rog_grad_shard *out, LinearI8Plan *p) {
    LinearI8Args &a = p->args;
    p->direct = true;
    p->grid = 0;
    if (!known(out_dtype)) return ROG_ERR_INVALID_ARGUMENT;
    rog_status st = lay_weights(shards, W, dim, 1, true, &a.sh, &p->direct);
    if (st != ROG_OK) return st;
    if (rows >= kMaxVocab) return ROG_ERR_TOO_LARGE;
    int64_t q_bytes = 0;
    st = check_matrix(q, q_stride, rows, uint64_t(dim), 1, false, &q_bytes);
    if (st != ROG_OK || rows == 0) return st;
    if (!scale || addr(scale) % 4 || !out) return ROG_ERR_INVALID_ARGUMENT;
    const uint32_t os = esize(out_dtype);
    const Strip qs = matrix(q, rows, q_bytes, uint64_t(dim)), ss = flat(scale, rows * 4);
    for (int r = 0; r < W; ++r) {
        const uint64_t width = a.sh.s[r].width;
        a.scale[r] = shards[r].scale;
        a.out[r] = out[r].grad;
        a.out_stride[r] = 0;
        if (!width) continue;
        if (!shards[r].scale || addr(shards[r].scale) % 4 || !out[r].grad || addr(out[r].grad) % os || out[r].row_stride < 0 ||
            (rows > 1 && uint64_t(out[r].row_stride) < width))
            return ROG_ERR_INVALID_ARGUMENT;
        if (uint64_t(out[r].row_stride) >= uint64_t(1) << 48) return ROG_ERR_TOO_LARGE;
        a.out_stride[r] = out[r].row_stride * os;
        if (!fits(addr(a.out[r]), rows, uint64_t(a.out_stride[r]), width * os)) return ROG_ERR_TOO_LARGE;
    }
    for (int r = 0; r < W; ++r) {
        const Strip o = matrix(a.out[r], rows, a.out_stride[r], uint64_t(a.sh.s[r].width) * os);
        if (overlap(o, qs) || overlap(o, ss)) return ROG_ERR_OVERLAP;
        for (int s = 0; s < W; ++s)
            if (overlap(o, matrix(a.sh.s[s].w, a.sh.s[s].width, a.sh.s[s].stride, uint64_t(dim))) ||
                overlap(o, flat(a.scale[s], uint64_t(a.sh.s[s].width) * 4)) ||
                (s < r && overlap(o, matrix(a.out[s], rows, a.out_stride[s], uint64_t(a.sh.s[s].width) * os))))
                return ROG_ERR_OVERLAP;
    }
    p->form = form_of(rows, a.sh);
    lay_tiles(&a.sh, tile_columns(p->form));
    if (!aligned(q, uint64_t(q_bytes))) p->direct = false;
    const uint64_t groups = groups_of(a.sh.tile0[W] * ceil_div(rows, tile_rows(p->form)), p->form);
    if (groups >= kMaxGroups) return ROG_ERR_TOO_LARGE;
    p->grid = uint32_t(groups);
    a.a = LinearRows{q, q_bytes, nullptr, uint32_t(rows), uint32_t(dim)};
    a.row_scale = scale;
    return ROG_OK;
}

}  // namespace rog

extern "C" {

ROG_API rog_status rog_linear_logprob_plan(const rog_weight_shard *shards, int W, size_t rows, int64_t dim, rog_dtype dtype, int tokens,
                                           rog_linear_plan_info *info) {
    if (!info) return ROG_ERR_INVALID_ARGUMENT;
    rog::ScorePlan p;
    const rog_status st = rog::plan_linear_logprob(nullptr, 0, rows, dim, shards, W, dtype, 1.0f, nullptr, nullptr, nullptr, 0, false,
                                                   tokens != 0, &p);
    if (st != ROG_OK) return st;
    *info = rog_linear_plan_info{rows ? rog::tile_columns(p.form) : 0, rows ? rog::tile_rows(p.form) : 0, rows ? 1u : 0u,
                                 rows ? 1u + (p.grid != 0) + p.packs : 0u, p.workspace_bytes};
    return ROG_OK;
}

ROG_API rog_status rog_linear_logprob_grad_plan(const rog_weight_shard *shards, int W, size_t rows, int64_t dim, rog_dtype dtype,
                                                rog_linear_plan_info *info) {
    if (!info) return ROG_ERR_INVALID_ARGUMENT;
    rog::GradPlan p;
    const rog_status st = rog::plan_linear_grad(nullptr, 0, rows, dim, shards, W, dtype, 1.0f, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                nullptr, 0, nullptr, nullptr, 0, false, &p);
    if (st != ROG_OK) return st;
    *info = rog_linear_plan_info{rows ? rog::kGradTile : 0, rows ? (p.form == rog::kFormWide ? 256u : 64u) : 0, rows ? p.pieces : 0,
                                 rows ? 1 + (p.form == rog::kFormWide ? 2 + !p.running : 4) * p.pieces + (p.back.splits > 1) * p.pieces : 0, p.workspace_bytes};
    return ROG_OK;
}

}  // extern "C"
