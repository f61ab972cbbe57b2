// rr_loss.cpp -- the C ABI of the sharded losses (rr.h): argument validation,
// the division of the workspace, and the launches of each call.  Everything is
// rejected before any HIP call; nothing is allocated on the device.
#include "rr_loss.h"

#include <math.h>

#include <algorithm>

#include "rr_call.h"

namespace {

using namespace rr;

rr_status check_tokens(int64_t rows)
{
    if (rows < 0 || rows > RR_MAX_ROUTE_ROWS)
        return set_error(RR_EINVAL, "rows=%lld outside [0, RR_MAX_ROUTE_ROWS]", (long long)rows);
    return RR_OK;
}

rr_status check_vocab(const rr_vocab *v, int64_t rows)
{
    if (!v)
        return set_error(RR_EINVAL, "vocabulary descriptor is null");
    if (v->total < 1 || v->total > INT32_MAX)
        return set_error(RR_EINVAL, "total=%lld outside [1, 2^31)", (long long)v->total);
    if (v->vocab < 0 || v->first < 0 || v->first > v->total || v->vocab > v->total - v->first)
        return set_error(RR_EINVAL, "shard [first=%lld, + vocab=%lld) outside [0, total=%lld)",
                         (long long)v->first, (long long)v->vocab, (long long)v->total);
    if (v->vocab > RR_MAX_VOCAB)
        return set_error(RR_EINVAL, "vocab=%lld above RR_MAX_VOCAB", (long long)v->vocab);
    if (v->dim < 1 || v->dim > RR_MAX_DIM)
        return set_error(RR_EINVAL, "dim=%d outside [1, RR_MAX_DIM]", v->dim);
    if (v->topk < 1 || v->topk > RR_MAX_TOPK)
        return set_error(RR_EINVAL, "topk=%d outside [1, RR_MAX_TOPK]", v->topk);
    if (!isfinite(v->scale))
        return set_error(RR_EINVAL, "scale is not finite");
    if (rows < 0 || rows > RR_MAX_ROWS)
        return set_error(RR_EINVAL, "rows=%lld outside [0, RR_MAX_ROWS]", (long long)rows);
    if (v->vocab * v->dim > RR_MAX_PLANE || rows * v->vocab > RR_MAX_PLANE)
        return set_error(RR_EINVAL, "rows=%lld, vocab=%lld, dim=%d: vocab * dim or rows * vocab above RR_MAX_PLANE",
                         (long long)rows, (long long)v->vocab, v->dim);
    return RR_OK;
}

Product logits_product(const rr_vocab *v, int dtype, int64_t rows, const void *x, const void *w)
{
    return Product{w, x, v->dim, v->dim, int32_t(v->vocab), int32_t(rows), v->dim, dtype == RR_BF16};
}

// The workspace of rr_vocab_grad.  dz is held for one piece of the vocabulary
// at a time.
struct GradSpace {
    int64_t piece, ldd, ldv, lda;
    int32_t pieces, x_splits, w_splits;
    float2 *row;
    char *x, *w, *dz;    // x without the rows that have no gradient; a piece of w, if not in 16-byte chunks
    float *dx, *dw;      // parts of the gradients' sums
    int64_t bytes;
};

// Bytes of one piece of dz.
constexpr int64_t kPieceBytes = int64_t(1) << 28;

GradSpace grad_space(const rr_vocab *v, int dtype, int64_t rows, void *base)
{
    const int64_t es = elem_size(dtype);
    GradSpace s{};
    const int64_t most = std::max<int64_t>(kPieceBytes / (std::max<int64_t>(rows, 1) * es) / 256 * 256, 256);
    const int64_t pieces = (v->vocab + most - 1) / most;
    s.piece = pieces ? std::min(round_up((v->vocab + pieces - 1) / pieces, 256), v->vocab) : 0;
    s.ldd = round_up(v->dim, 16 / es);
    s.ldv = round_up(s.piece, 64);
    s.lda = round_up(v->dim, 4);
    s.pieces = s.piece ? int32_t((v->vocab + s.piece - 1) / s.piece) : 0;
    // one number of parts for every piece, as dx's sums go on from piece to piece
    const int32_t bf16 = dtype == RR_BF16, n = int32_t(rows), c = int32_t(s.piece);
    s.x_splits = product_splits(Product{nullptr, nullptr, s.ldd, s.ldv, v->dim, n, c, bf16}, false);
    s.w_splits = product_splits(Product{nullptr, nullptr, s.ldd, s.ldv, v->dim, c, n, bf16}, true);
    Carver space(base);
    s.row = static_cast<float2 *>(space.take(rows * 8));
    s.x = static_cast<char *>(space.take(rows * s.ldd * es));
    s.w = static_cast<char *>(space.take(s.piece * s.ldd * es));
    s.dz = static_cast<char *>(space.take(rows * s.ldv * es));
    s.dx = static_cast<float *>(space.take(s.x_splits * rows * s.lda * 4));
    s.dw = static_cast<float *>(space.take(s.w_splits > 1 ? s.w_splits * s.piece * s.lda * 4 : 0));
    s.bytes = space.used();
    return s;
}

int64_t stats_bytes(const rr_vocab *v, int dtype, int64_t rows)
{
    return round_up(stats_parts(logits_product(v, dtype, rows, nullptr, nullptr)) * rows * 8, 256);
}

rr_status check_router(const rr_router *r)
{
    if (!r)
        return set_error(RR_EINVAL, "router descriptor is null");
    if (r->experts < 1 || r->experts > RR_MAX_EXPERTS)
        return set_error(RR_EINVAL, "experts=%d outside [1, RR_MAX_EXPERTS]", r->experts);
    if (r->topk < 1 || r->topk > std::min(r->experts, RR_MAX_ROUTE_TOPK))
        return set_error(RR_EINVAL, "topk=%d outside [1, min(experts, RR_MAX_ROUTE_TOPK)]", r->topk);
    return RR_OK;
}

int64_t route_bytes(const rr_router *r, int64_t rows)
{
    const int32_t blocks = route_blocks(rows, r->experts);
    return blocks > 1 ? round_up(int64_t(blocks) * (r->experts + 1) * 4, 256) + int64_t(blocks) * r->experts * 4 : 0;
}

// The arguments both combining calls share.
rr_status check_combine(const rr_vocab *v, int64_t rows, const int64_t *index, const float *const *stats,
                        const float *const *picked, int nShards, Buffers &b)
{
    const rr_status st = check_vocab(v, rows);
    if (st != RR_OK)
        return st;
    if (nShards < 1 || nShards > RR_MAX_SHARDS)
        return set_error(RR_EINVAL, "nShards=%d outside [1, RR_MAX_SHARDS]", nShards);
    if (!stats || !picked)
        return set_error(RR_EINVAL, "an array of shard pointers is null");
    b.in(index, rows * v->topk * 8, 8, "index");
    for (int i = 0; i < nShards; ++i)
        b.in(stats[i], rows * 8, 8, "stats").in(picked[i], rows * v->topk * 4, 4, "picked");
    return RR_OK;
}

CombineArgs combine_args(const rr_vocab *v, int64_t rows, const int64_t *index, const float *const *stats,
                         const float *const *picked, int nShards, float *lse, float *logit, float *loss)
{
    CombineArgs a{};
    for (int i = 0; i < nShards; ++i) {
        a.stats[i] = reinterpret_cast<const float2 *>(stats[i]);
        a.picked[i] = picked[i];
    }
    a.shards = nShards;
    a.rows = int32_t(rows);
    a.topk = v->topk;
    a.total = v->total;
    a.scale = v->scale;
    a.index = index;
    a.lse = lse;
    a.logit = logit;
    a.loss = loss;
    return a;
}

}  // namespace

extern "C" {

int64_t rr_vocab_workspace(const rr_vocab *v, int dtype, int64_t rows, int grad)
{
    if (check_vocab(v, rows) != RR_OK || check_dtype(dtype) != RR_OK)
        return -1;
    set_ok();
    const int64_t n = stats_bytes(v, dtype, rows);
    return grad ? std::max(n, grad_space(v, dtype, rows, nullptr).bytes) : n;
}

rr_status rr_vocab_stats(const rr_vocab *v, int dtype, int64_t rows, const void *x, const void *w,
                         const int64_t *index, float *stats, float *picked, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    rr_status st = check_vocab(v, rows);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), need = stats_bytes(v, dtype, rows);
    if ((st = check_workspace(workspace_bytes, need)) != RR_OK)
        return st;
    Buffers b;
    b.in(x, rows * v->dim * es, es, "x").in(w, v->vocab * v->dim * es, es, "w");
    b.in(index, rows * v->topk * 8, 8, "index");
    b.out(stats, rows * 8, 8, "stats").out(picked, rows * v->topk * 4, 4, "picked");
    b.out(workspace, need, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();

    Launches l(stream);
    StatsArgs a{};
    a.p = logits_product(v, dtype, rows, x, w);
    a.scale = v->scale;
    a.part = static_cast<float2 *>(workspace);
    if (v->vocab > 0)
        l.add(launch_stats, a);
    l.add(launch_stats_done, StatsDoneArgs{a.part, x, w, index, reinterpret_cast<float2 *>(stats), picked, v->first,
                                           int32_t(stats_parts(a.p)), a.p.nj, v->topk, a.p.ni, v->dim, a.p.bf16,
                                           v->scale});
    return l.finish();
}

rr_status rr_vocab_cross_entropy(const rr_vocab *v, int64_t rows, const int64_t *index,
                                 const float *const *stats, const float *const *picked, int nShards,
                                 float *lse, float *logit, float *loss, void *stream)
{
    Buffers b;
    rr_status st = check_combine(v, rows, index, stats, picked, nShards, b);
    if (st != RR_OK)
        return st;
    if (v->topk != 1)
        return set_error(RR_EINVAL, "topk=%d: cross entropy has one target per row", v->topk);
    b.out(lse, rows * 4, 4, "lse").out(logit, rows * 4, 4, "logit").out(loss, rows * 4, 4, "loss");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_cross_entropy, combine_args(v, rows, index, stats, picked, nShards, lse, logit, loss));
    return l.finish();
}

rr_status rr_vocab_distill(const rr_vocab *v, int dtype, int64_t rows, const int64_t *index,
                           const void *teacher, const float *const *stats, const float *const *picked,
                           int nShards, float *lse, float *logit, float *prob, float *loss, void *stream)
{
    rr_status st = check_dtype(dtype);
    if (st != RR_OK)
        return st;
    Buffers b;
    if ((st = check_combine(v, rows, index, stats, picked, nShards, b)) != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), n = rows * v->topk;
    b.in(teacher, n * es, es, "teacher");
    b.out(lse, rows * 4, 4, "lse").out(logit, n * 4, 4, "logit").out(prob, n * 4, 4, "prob");
    b.out(loss, rows * 4, 4, "loss");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();
    CombineArgs a = combine_args(v, rows, index, stats, picked, nShards, lse, logit, loss);
    a.teacher = teacher;
    a.prob = prob;
    a.bf16 = dtype == RR_BF16;
    Launches l(stream);
    l.add(launch_distill, a);
    return l.finish();
}

rr_status rr_vocab_grad(const rr_vocab *v, int dtype, int64_t rows, const void *x, const void *w,
                        const int64_t *index, const float *lse, const float *logit, const float *prob,
                        const float *grad, void *dx, void *dw, void *workspace, int64_t workspace_bytes,
                        void *stream)
{
    rr_status st = check_vocab(v, rows);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st != RR_OK)
        return st;
    if (!prob && v->topk != 1)
        return set_error(RR_EINVAL, "topk=%d: cross entropy (prob is null) has one target per row", v->topk);
    const int64_t es = elem_size(dtype), wbytes = v->vocab * v->dim * es, xbytes = rows * v->dim * es;
    const GradSpace s = grad_space(v, dtype, rows, workspace);
    if ((st = check_workspace(workspace_bytes, s.bytes)) != RR_OK)
        return st;
    Buffers b;
    b.in(x, xbytes, es, "x").in(w, wbytes, es, "w").in(index, rows * v->topk * 8, 8, "index");
    b.in(lse, rows * 4, 4, "lse").in(logit, rows * v->topk * 4, 4, "logit").in(grad, rows * 4, 4, "grad");
    if (prob)
        b.in(prob, rows * v->topk * 4, 4, "prob");
    b.out(dx, xbytes, es, "dx").out(dw, wbytes, es, "dw").out(workspace, s.bytes, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;

    const int32_t bf16 = dtype == RR_BF16, dim = v->dim, n = int32_t(rows);
    Launches l(stream);
    if (rows == 0) {
        // no row contributes: dw is zero
        if (v->vocab > 0)
            l.add(launch_gather, GathersArgs{GatherArgs{}, GatherArgs{nullptr, dw, v->vocab, s.lda, dim, 0}, bf16});
        return l.finish();
    }
    const RowsArgs of_rows{index, lse, prob, grad, n, v->topk, v->total, v->scale, s.row};
    const bool copy_x = !in_chunks(x, dim, es), copy_w = !in_chunks(w, dim, es);
    const bool whole = s.pieces == 1 && s.x_splits == 1, parts = s.w_splits > 1;  // of dx, of dw
    const AlignArgs x_copy{x, s.x, rows, s.ldd, dim};
    const void *xc = copy_x ? s.x : x;
    const int64_t ldx = copy_x ? s.ldd : dim, ldw = copy_w ? s.ldd : dim;
    if (v->vocab == 0)
        l.add(launch_gather, GathersArgs{GatherArgs{nullptr, dx, rows, s.lda, dim, 0}, GatherArgs{}, bf16});
    for (int64_t v0 = 0; v0 < v->vocab; v0 += s.piece) {
        const bool first = v0 == 0, last = v0 + s.piece >= v->vocab;
        const int32_t c = int32_t(std::min(s.piece, v->vocab - v0));
        const void *wp = static_cast<const char *>(w) + v0 * dim * es, *wc = copy_w ? s.w : wp;
        char *dwp = static_cast<char *>(dw) + v0 * dim * es;
        if (copy_w || (first && (copy_x || prob)))
            l.add(launch_prepare, PrepareArgs{of_rows, first && copy_x ? x_copy : AlignArgs{},
                                              copy_w ? AlignArgs{wp, s.w, c, s.ldd, dim} : AlignArgs{},
                                              first && prob, bf16});
        l.add(launch_dz, DzArgs{Product{wc, xc, ldw, ldx, c, n, dim, bf16}, of_rows, logit, v->first + v0, s.dz, s.ldv,
                                first && !copy_x ? x_copy : AlignArgs{}});
        if (prob)
            l.add(launch_targets, TargetArgs{index, logit, prob, s.row, n, v->topk, c, bf16, v->first + v0, s.dz, s.ldv});
        l.add(launch_stores, StoresArgs{
            StoreArgs{Product{wc, s.dz, ldw, s.ldv, dim, n, c, bf16}, whole ? dx : nullptr, dim, whole ? nullptr : s.dx,
                      s.lda, s.x_splits, !first},
            StoreArgs{Product{s.x, s.dz, s.ldd, s.ldv, dim, c, n, bf16}, parts ? nullptr : dwp, dim,
                      parts ? s.dw : nullptr, s.lda, s.w_splits, 0}});
        if (parts || (last && !whole))
            l.add(launch_gather, GathersArgs{
                last && !whole ? GatherArgs{s.dx, dx, rows, s.lda, dim, s.x_splits} : GatherArgs{},
                parts ? GatherArgs{s.dw, dwp, c, s.lda, dim, s.w_splits} : GatherArgs{}, bf16});
    }
    return l.finish();
}

int64_t rr_route_workspace(const rr_router *r, int64_t rows)
{
    if (check_router(r) != RR_OK || check_tokens(rows) != RR_OK)
        return -1;
    set_ok();
    return route_bytes(r, rows);
}

rr_status rr_route(const rr_router *r, int dtype, int64_t rows, const void *logits, const uint8_t *keep,
                   int32_t *choice, float *weight, float *lse, int32_t *counts, float *prob_sum,
                   void *workspace, int64_t workspace_bytes, void *stream)
{
    rr_status st = check_router(r);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_tokens(rows);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), need = route_bytes(r, rows), e = r->experts;
    if ((st = check_workspace(workspace_bytes, need)) != RR_OK)
        return st;
    Buffers b;
    b.in(logits, rows * e * es, es, "logits");
    if (keep)
        b.in(keep, rows, 1, "keep");
    b.out(choice, rows * r->topk * 4, 4, "choice").out(weight, rows * r->topk * 4, 4, "weight");
    b.out(lse, rows * 4, 4, "lse").out(counts, (e + 1) * 4, 4, "counts").out(prob_sum, e * 4, 4, "prob_sum");
    b.out(workspace, need, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;
    const int32_t blocks = route_blocks(rows, r->experts);
    RouteArgs a{logits, keep, choice, weight, lse, counts, prob_sum, rows,
                r->experts, r->topk, r->renormalize ? 1 : 0, dtype == RR_BF16, blocks};
    Launches l(stream);
    if (blocks <= 1) {
        l.add(launch_route, a);
        return l.finish();
    }
    a.counts = static_cast<int32_t *>(workspace);
    a.prob_sum = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up(int64_t(blocks) * (e + 1) * 4, 256));
    l.add(launch_route, a);
    l.add(launch_route_sum, RouteSumArgs{a.counts, a.prob_sum, counts, prob_sum, blocks, r->experts});
    return l.finish();
}

rr_status rr_balance_loss(const rr_router *r, const int32_t *const *counts, const float *const *prob_sum,
                          int nRanks, float *loss, float *slope, void *stream)
{
    rr_status st = check_router(r);
    if (st != RR_OK)
        return st;
    if (nRanks < 1 || nRanks > RR_MAX_SHARDS)
        return set_error(RR_EINVAL, "nRanks=%d outside [1, RR_MAX_SHARDS]", nRanks);
    if (!counts || !prob_sum)
        return set_error(RR_EINVAL, "an array of rank pointers is null");
    const int64_t e = r->experts;
    Buffers b;
    BalanceArgs a{};
    for (int i = 0; i < nRanks; ++i) {
        b.in(counts[i], (e + 1) * 4, 4, "counts").in(prob_sum[i], e * 4, 4, "prob_sum");
        a.counts[i] = counts[i];
        a.prob_sum[i] = prob_sum[i];
    }
    b.out(loss, 4, 4, "loss").out(slope, e * 4, 4, "slope");
    if ((st = b.check()) != RR_OK)
        return st;
    a.ranks = nRanks;
    a.experts = r->experts;
    a.topk = r->topk;
    a.loss = loss;
    a.slope = slope;
    Launches l(stream);
    l.add(launch_balance, a);
    return l.finish();
}

rr_status rr_route_grad(const rr_router *r, int dtype, int64_t rows, const void *logits, const uint8_t *keep,
                        const int32_t *choice, const float *weight, const float *lse, const float *slope,
                        const float *grad_loss, const float *grad_weight, void *dlogits, void *stream)
{
    rr_status st = check_router(r);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_tokens(rows);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), e = r->experts, n = rows * r->topk;
    Buffers b;
    b.in(logits, rows * e * es, es, "logits");
    if (keep)
        b.in(keep, rows, 1, "keep");
    b.in(choice, n * 4, 4, "choice").in(weight, n * 4, 4, "weight").in(lse, rows * 4, 4, "lse");
    b.in(slope, e * 4, 4, "slope").in(grad_loss, 4, 4, "grad_loss").in(grad_weight, n * 4, 4, "grad_weight");
    b.out(dlogits, rows * e * es, es, "dlogits");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_route_grad, RouteGradArgs{logits, keep, choice, weight, lse, slope, grad_loss, grad_weight, dlogits,
                                           rows, r->experts, r->topk, r->renormalize ? 1 : 0, dtype == RR_BF16});
    return l.finish();
}

}  // extern "C"
