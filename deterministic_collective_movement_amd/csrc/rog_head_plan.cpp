// rog_head_plan.cpp -- argument validation, launch forms and workspace sizes of
// the vocabulary-side operators (token log probabilities, their gradient, the
// policy loss).  Pure host code: no HIP calls, so every decision here can be
// checked on a machine without a GPU.
#include <math.h>

#include <algorithm>

#include "rog_head_checks.h"

namespace rog {
namespace {

constexpr uint64_t kMaxGroups = uint64_t(1) << 31;   // workgroups of one launch
constexpr float kMinTemperature = 1.0f / 1024, kMaxTemperature = 1024.0f;
constexpr double kLog2E = 1.4426950408889634;

// 1 / temperature as a binary32 number and the rest, to 2^-48 of it together.
void invert(float temperature, float *inv, float *rest) {
    const double t = 1.0 / double(temperature);
    *inv = float(t);
    *rest = float(t - double(*inv));
}

// Shared checks of the logits, and their layout into the kernel arguments.
// heads: columns by which the blocks of each shard may begin early (NULL: none do).
rog_status lay_shards(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype, bool addresses,
                      uint32_t block, const uint32_t *heads, HeadShards *h, uint32_t *vocab, uint32_t *blocks) {
    if (!shards || W < 1 || W > kMaxPeers || !known(dtype)) return ROG_ERR_INVALID_ARGUMENT;
    const uint32_t es = esize(dtype);
    uint64_t v = 0, b = 0;
    for (int r = 0; r < W; ++r) {
        const rog_logit_shard &s = shards[r];
        if (s.width < 0) return ROG_ERR_INVALID_ARGUMENT;
        if (addresses) {
            if (s.row_stride < 0) return ROG_ERR_INVALID_ARGUMENT;
            if (rows && s.width && (!s.logits || addr(s.logits) % es)) return ROG_ERR_INVALID_ARGUMENT;
        }
        if (uint64_t(s.width) >= kMaxVocab || v + uint64_t(s.width) >= kMaxVocab) return ROG_ERR_TOO_LARGE;
        Shard &o = h->s[r];
        o = Shard{s.logits, 0, uint32_t(s.width), uint32_t(v)};
        h->block0[r] = uint32_t(b);
        v += uint64_t(s.width);
        b += s.width ? ceil_div(uint64_t(s.width) + (heads ? heads[r] : 0), block) : 0;
        if (addresses) {
            if (uint64_t(s.row_stride) >= uint64_t(1) << 48) return ROG_ERR_TOO_LARGE;
            o.stride = s.row_stride * es;
            if (!fits(addr(s.logits), rows, uint64_t(o.stride), uint64_t(s.width) * es)) return ROG_ERR_TOO_LARGE;
        }
    }
    h->block0[W] = uint32_t(b);
    h->W = uint32_t(W);
    h->blocks = uint32_t(b);
    h->even = h->block0[1];
    for (int r = 1; r < W; ++r)
        if (h->block0[r + 1] - h->block0[r] != h->even) h->even = 0;
    h->even_div = make_divider(std::max(h->even, 1u));
    *vocab = uint32_t(v);
    *blocks = uint32_t(b);
    return rows >= kMaxVocab ? ROG_ERR_TOO_LARGE : ROG_OK;
}

// Units that have blocks, of a row of more than one.
inline uint32_t units_of(uint32_t blocks) {
    const uint32_t rest = blocks % kChunkBlocks;
    return blocks / kChunkBlocks * kChunkUnits + std::min(rest, kChunkUnits);
}
inline uint32_t chunks_of(uint32_t blocks) { return uint32_t(ceil_div(blocks, kChunkBlocks)); }

// Launch form, grid and workspace of rog_logprob.
rog_status choose_form(uint32_t blocks, size_t rows, int top_k, rog_logprob_form form, rog_head_plan_info *info) {
    if (form < ROG_LOGPROB_AUTO || form > ROG_LOGPROB_WAVE || top_k < 0 || top_k > kMaxTopK)
        return ROG_ERR_INVALID_ARGUMENT;
    const uint32_t units = units_of(blocks);
    const bool wave = blocks <= kUnitBlocks, may_split = rows <= kHeadCounters && !wave;
    const uint64_t split_rows = top_k ? kSplitRowsTop : kSplitRows;
    if (form == ROG_LOGPROB_AUTO)
        form = wave ? ROG_LOGPROB_WAVE
               : may_split && rows * units + kSplitCost <= split_rows * units ? ROG_LOGPROB_SPLIT : ROG_LOGPROB_ROW;
    if ((form == ROG_LOGPROB_SPLIT && !may_split) || (form == ROG_LOGPROB_WAVE) != wave) return ROG_ERR_INVALID_ARGUMENT;
    const uint64_t groups = form == ROG_LOGPROB_SPLIT  ? rows * uint64_t(units)
                            : form == ROG_LOGPROB_WAVE ? ceil_div(rows, kWaveRows) : rows;
    if (groups >= kMaxGroups) return ROG_ERR_TOO_LARGE;
    info->form = rows ? form : ROG_LOGPROB_AUTO;
    info->blocks = blocks;
    info->workspace_bytes = rows && form == ROG_LOGPROB_SPLIT
                                ? kHeadCounterBytes + rows * units * kUnitFloats * sizeof(float) : 0;
    info->block = form == ROG_LOGPROB_WAVE ? 64 * kWaveRows : kHeadThreads;
    info->grid = uint32_t(groups);
    return ROG_OK;
}

}  // namespace

rog_status plan_logprob(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype, float temperature,
                        const int64_t *tokens, int top_k, const rog_logprob_out *out, void *workspace,
                        size_t workspace_bytes, rog_logprob_form form, bool check_workspace, LogprobPlan *p) {
    LogprobArgs &a = p->args;
    uint32_t vocab = 0, blocks = 0;
    if (!out || !(temperature >= kMinTemperature && temperature <= kMaxTemperature)) return ROG_ERR_INVALID_ARGUMENT;
    rog_status st = lay_shards(shards, W, rows, dtype, true, kHeadBlock, nullptr, &a.sh, &vocab, &blocks);
    if (st != ROG_OK) return st;
    st = choose_form(blocks, rows, top_k, form, &p->info);
    if (st != ROG_OK || rows == 0) return st;

    if (out->logp && !tokens) return ROG_ERR_INVALID_ARGUMENT;
    if (addr(tokens) % 8 || addr(out->top_ids) % 8) return ROG_ERR_INVALID_ARGUMENT;
    if ((addr(out->logp) | addr(out->entropy) | addr(out->lse) | addr(out->top_logp)) % 4) return ROG_ERR_INVALID_ARGUMENT;
    const uint64_t need = p->info.workspace_bytes;
    if (check_workspace && need && (!workspace || addr(workspace) % 16 || workspace_bytes < need))
        return ROG_ERR_INVALID_ARGUMENT;

    Strip outs[6];
    int n_out = 0;
    const auto add = [&](const void *q, uint64_t bytes) { if (q && bytes) outs[n_out++] = flat(q, bytes); };
    add(out->logp, rows * 4);
    add(out->entropy, rows * 4);
    add(out->lse, rows * 4);
    add(out->top_logp, rows * uint64_t(top_k) * 4);
    add(out->top_ids, rows * uint64_t(top_k) * 8);
    if (need) add(workspace, need);
    for (int i = 0; i < n_out; ++i) {
        if (outs[i].at > UINTPTR_MAX - outs[i].width) return ROG_ERR_TOO_LARGE;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return ROG_ERR_OVERLAP;
        if (tokens && overlap(outs[i], flat(tokens, rows * 8))) return ROG_ERR_OVERLAP;
        for (int r = 0; r < W; ++r)
            if (overlap(outs[i], Strip{addr(a.sh.s[r].x), rows, uint64_t(a.sh.s[r].stride), uint64_t(a.sh.s[r].width) * esize(dtype)}))
                return ROG_ERR_OVERLAP;
    }

    a.tokens = tokens;
    a.logp = out->logp;
    a.entropy = out->entropy;
    a.lse = out->lse;
    a.top_logp = top_k ? out->top_logp : nullptr;
    a.top_ids = top_k ? out->top_ids : nullptr;
    a.counters = static_cast<uint32_t *>(workspace);
    a.part = need ? reinterpret_cast<float *>(static_cast<char *>(workspace) + kHeadCounterBytes) : nullptr;
    a.scale = float(kLog2E / double(temperature));
    invert(temperature, &a.inv_t, &a.inv_t_rest);
    a.bound = float(ldexp(double(temperature) / kLog2E, 30));
    a.rows = uint32_t(rows);
    a.chunks = chunks_of(blocks);
    a.units = units_of(blocks);
    a.top_k = uint32_t(top_k);
    a.slot_shift = 0;
    while ((a.chunks * kUnitBlocks - (blocks ? 1 : 0)) >> a.slot_shift >= kTopSlots) ++a.slot_shift;
    a.vocab = vocab;
    p->dtype = dtype;
    p->nt_loads = rows * uint64_t(vocab) * esize(dtype) >= ROG_HEAD_NT_MIN_BYTES;
    return ROG_OK;
}

rog_status plan_logprob_grad(const rog_logit_shard *shards, const rog_grad_shard *grads, int W, size_t rows,
                             rog_dtype dtype, float temperature, const int64_t *tokens, const float *lse,
                             const float *entropy, const float *g_logp, const float *g_entropy,
                             LogprobGradPlan *p) {
    LogprobGradArgs &a = p->args;
    uint32_t vocab = 0, blocks = 0;
    p->grid = 0;
    if (!grads || !(temperature >= kMinTemperature && temperature <= kMaxTemperature)) return ROG_ERR_INVALID_ARGUMENT;
    // Pieces begin with the gradient's 128-byte lines: as many columns early as a row's first line may hold of others.
    const uint32_t size = known(dtype) ? esize(dtype) : 4;
    uint32_t heads[kMaxPeers] = {};
    for (int r = 0; r < W && r < kMaxPeers; ++r) {
        const uint64_t places = addr(grads[r].grad) | uint64_t(grads[r].row_stride) * size | 128;
        heads[r] = uint32_t(128 - (places & -places)) / size;
    }
    rog_status st = lay_shards(shards, W, rows, dtype, true, kGradPieceBytes / size, heads, &a.sh, &vocab, &blocks);
    if (st != ROG_OK) return st;
    if (rows == 0 || vocab == 0) return ROG_OK;
    if (!tokens || !lse || !entropy || !g_logp || addr(tokens) % 8 ||
        (addr(lse) | addr(entropy) | addr(g_logp) | addr(g_entropy)) % 4)
        return ROG_ERR_INVALID_ARGUMENT;
    const uint32_t es = esize(dtype);
    for (int r = 0; r < W; ++r) {
        const uint64_t width = uint64_t(a.sh.s[r].width) * es;
        a.g[r] = grads[r].grad;
        a.g_stride[r] = 0;
        if (!width) continue;
        if (!grads[r].grad || addr(grads[r].grad) % es || grads[r].row_stride < 0 ||
            (rows > 1 && uint64_t(grads[r].row_stride) < a.sh.s[r].width))
            return ROG_ERR_INVALID_ARGUMENT;
        if (uint64_t(grads[r].row_stride) >= uint64_t(1) << 48) return ROG_ERR_TOO_LARGE;
        a.g_stride[r] = grads[r].row_stride * es;
        if (!fits(addr(a.g[r]), rows, uint64_t(a.g_stride[r]), width)) return ROG_ERR_TOO_LARGE;
    }
    const float *const vectors[4] = {lse, entropy, g_logp, g_entropy};
    for (int r = 0; r < W; ++r) {
        const Strip g{addr(a.g[r]), rows, uint64_t(a.g_stride[r]), uint64_t(a.sh.s[r].width) * es};
        for (int q = 0; q < W; ++q) {
            const Strip x{addr(a.sh.s[q].x), rows, uint64_t(a.sh.s[q].stride), uint64_t(a.sh.s[q].width) * es};
            const bool in_place = q == r && g.at == x.at && (rows == 1 || g.stride == x.stride);
            if (!in_place && overlap(g, x)) return ROG_ERR_OVERLAP;
            if (q < r && overlap(g, Strip{addr(a.g[q]), rows, uint64_t(a.g_stride[q]), uint64_t(a.sh.s[q].width) * es}))
                return ROG_ERR_OVERLAP;
        }
        for (const float *v : vectors)
            if (v && overlap(g, flat(v, rows * 4))) return ROG_ERR_OVERLAP;
        if (overlap(g, flat(tokens, rows * 8))) return ROG_ERR_OVERLAP;
    }
    a.tokens = tokens;
    a.lse = lse;
    a.entropy = entropy;
    a.g_logp = g_logp;
    a.g_entropy = g_entropy;
    invert(temperature, &a.inv_t, &a.inv_t_rest);
    a.vocab = vocab;
    a.pieces_div = make_divider(blocks);
    const uint64_t pieces = uint64_t(blocks) * rows;
    if (pieces >= kMaxGroups) return ROG_ERR_TOO_LARGE;
    a.groups = p->grid = uint32_t(pieces);
    p->nt_loads = rows * uint64_t(vocab) * es >= ROG_HEAD_NT_MIN_BYTES;
    p->dtype = dtype;
    return ROG_OK;
}

namespace {
// Tiles per workgroup and workgroups: the order of the sums hangs on them, so
// both go by n alone.
struct PolicySplit {
    uint64_t tiles, groups;
};
PolicySplit policy_split(uint64_t n) {
    const uint64_t all = std::max<uint64_t>(1, ceil_div(n, kPolicyTile)), tiles = ceil_div(all, kPolicyGroups);
    return PolicySplit{tiles, ceil_div(all, tiles)};
}
size_t policy_workspace(uint64_t n) {
    const uint64_t g = policy_split(n).groups;
    return g <= 1 ? 0 : kHeadCounterBytes + g * 4 * sizeof(double);
}
}  // namespace

rog_status plan_policy(const rog_policy_in *in, size_t n, const rog_policy_params *k, const rog_policy_out *out,
                       void *workspace, size_t workspace_bytes, PolicyPlan *p) {
    PolicyArgs &a = p->args;
    if (!in || !k || !out || !out->stats) return ROG_ERR_INVALID_ARGUMENT;
    if (!(k->clip_low >= 0 && k->clip_low <= 1) || !(k->clip_high >= 0) || !isfinite(k->kl_coef) ||
        !isfinite(k->entropy_coef) || !isfinite(k->grad_scale))
        return ROG_ERR_INVALID_ARGUMENT;
    if (n >= size_t(1) << 34) return ROG_ERR_TOO_LARGE;
    if (n && (!in->logp || !in->old_logp || !in->advantage)) return ROG_ERR_INVALID_ARGUMENT;
    if (out->g_entropy && !in->entropy) return ROG_ERR_INVALID_ARGUMENT;
    const float *const ins[6] = {in->logp, in->old_logp, in->advantage, in->weight, in->ref_logp, in->entropy};
    const float *const outs[3] = {out->stats, out->g_logp, out->g_entropy};
    for (const float *q : ins)
        if (addr(q) % 4) return ROG_ERR_INVALID_ARGUMENT;
    const size_t need = policy_workspace(n);
    if (need && (!workspace || addr(workspace) % 16 || workspace_bytes < need)) return ROG_ERR_INVALID_ARGUMENT;
    if (need)
        for (const float *q : ins)
            if (q && overlap(flat(workspace, need), flat(q, n * 4))) return ROG_ERR_OVERLAP;
    for (int i = 0; i < 3; ++i) {
        if (!outs[i]) continue;
        if (addr(outs[i]) % 4) return ROG_ERR_INVALID_ARGUMENT;
        const Strip o = flat(outs[i], i == 0 ? 16 : n * 4);
        if (!fits(o.at, 1, 0, o.width)) return ROG_ERR_TOO_LARGE;
        for (const float *q : ins) {
            if (!q || (i != 0 && q == outs[i])) continue;   // in place: every thread reads its tokens before it writes them
            if (!fits(addr(q), 1, 0, n * 4)) return ROG_ERR_TOO_LARGE;
            if (overlap(o, flat(q, n * 4))) return ROG_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (outs[j] && overlap(o, flat(outs[j], j == 0 ? 16 : n * 4))) return ROG_ERR_OVERLAP;
        if (need && overlap(o, flat(workspace, need))) return ROG_ERR_OVERLAP;
    }
    a.logp = in->logp;
    a.old_logp = in->old_logp;
    a.adv = in->advantage;
    a.weight = in->weight;
    a.ref = in->ref_logp;
    a.entropy = in->entropy;
    a.stats = out->stats;
    a.g_logp = out->g_logp;
    a.g_entropy = out->g_entropy;
    a.counter = static_cast<uint32_t *>(workspace);
    a.part = need ? reinterpret_cast<double *>(static_cast<char *>(workspace) + kHeadCounterBytes) : nullptr;
    a.n = n;
    a.lo = float(log1p(-double(k->clip_low)));
    a.hi = float(log1p(double(k->clip_high)));
    a.ratio_lo = float(exp(double(a.lo)));
    a.ratio_hi = float(exp(double(a.hi)));
    a.kl_coef = k->kl_coef;
    a.entropy_coef = k->entropy_coef;
    a.grad_scale = k->grad_scale;
    a.w_all = n ? float(1.0 / double(n)) : 0.0f;
    a.tiles = uint32_t(policy_split(n).tiles);   // n < 2^34: at most 2^15
    a.groups = uint32_t(policy_split(n).groups);
    return ROG_OK;
}

}  // namespace rog

extern "C" {

ROG_API rog_status rog_logprob_plan(const rog_logit_shard *shards, int W, size_t rows, rog_dtype dtype, int top_k,
                                    rog_logprob_form form, rog_head_plan_info *info) {
    if (!info) return ROG_ERR_INVALID_ARGUMENT;
    rog::HeadShards h;
    uint32_t vocab = 0, blocks = 0;
    const rog_status st = rog::lay_shards(shards, W, rows, dtype, false, rog::kHeadBlock, nullptr, &h, &vocab, &blocks);
    return st != ROG_OK ? st : rog::choose_form(blocks, rows, top_k, form, info);
}

ROG_API size_t rog_policy_loss_workspace_bytes(size_t n) { return rog::policy_workspace(n); }

ROG_API int rog_max_top_k(void) { return rog::kMaxTopK; }

ROG_API int rog_logprob_max_split_rows(void) { return int(rog::kHeadCounters); }

}  // extern "C"
