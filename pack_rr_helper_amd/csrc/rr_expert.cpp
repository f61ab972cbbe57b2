// rr_expert.cpp -- the C ABI of the expert layer and the clipping (rr.h): argument
// validation, the division of workspaces, and the launches of each call.
// Everything is rejected before any HIP call; nothing is allocated on the device.
#include "rr_expert.h"

#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "rr_call.h"

namespace {

using namespace rr;

rr_status check_group_router(const rr_group_router *r)
{
    if (!r)
        return set_error(RR_EINVAL, "router descriptor is null");
    if (r->experts < 1 || r->experts > RR_MAX_EXPERTS)
        return set_error(RR_EINVAL, "experts=%d outside [1, RR_MAX_EXPERTS]", r->experts);
    if (r->groups < 1 || r->groups > RR_MAX_GROUPS || r->experts % r->groups != 0)
        return set_error(RR_EINVAL, "groups=%d outside [1, RR_MAX_GROUPS] or no divisor of experts=%d", r->groups, r->experts);
    if (r->top_groups < 1 || r->top_groups > r->groups)
        return set_error(RR_EINVAL, "top_groups=%d outside [1, groups=%d]", r->top_groups, r->groups);
    const int32_t size = r->experts / r->groups;
    if (r->group_best < 1 || r->group_best > std::min(2, size))
        return set_error(RR_EINVAL, "group_best=%d outside [1, min(2, experts / groups)]", r->group_best);
    if (r->topk < 1 || r->topk > std::min(r->top_groups * size, RR_MAX_ROUTE_TOPK))
        return set_error(RR_EINVAL, "topk=%d outside [1, min(top_groups * experts / groups, RR_MAX_ROUTE_TOPK)]", r->topk);
    if (r->score != RR_SOFTMAX && r->score != RR_SIGMOID)
        return set_error(RR_EINVAL, "unknown score %d", r->score);
    if (!isfinite(r->scale))
        return set_error(RR_EINVAL, "scale is not finite");
    return RR_OK;
}

rr_status check_tokens(int64_t rows)
{
    if (rows < 0 || rows > RR_MAX_ROUTE_ROWS)
        return set_error(RR_EINVAL, "rows=%lld outside [0, RR_MAX_ROUTE_ROWS]", (long long)rows);
    return RR_OK;
}

int64_t group_bytes(const rr_group_router *r, int64_t rows)
{
    const int64_t blocks = group_route_blocks(rows, r->experts, r->groups);
    return blocks > 1 ? blocks * (r->experts + 1) * 4 : 0;
}

rr_status check_experts(const rr_experts *e)
{
    if (!e)
        return set_error(RR_EINVAL, "experts descriptor is null");
    if (e->experts < 1 || e->experts > RR_MAX_EXPERTS)
        return set_error(RR_EINVAL, "experts=%d outside [1, RR_MAX_EXPERTS]", e->experts);
    if (e->first < 0 || e->first > 1 << 30)
        return set_error(RR_EINVAL, "first=%d outside [0, 2^30]", e->first);
    if (e->topk < 1 || e->topk > RR_MAX_ROUTE_TOPK)
        return set_error(RR_EINVAL, "topk=%d outside [1, RR_MAX_ROUTE_TOPK]", e->topk);
    if (e->rows < 0 || e->rows > RR_MAX_CHOICES / e->topk)
        return set_error(RR_EINVAL, "rows=%lld, topk=%d: rows * topk outside [0, RR_MAX_CHOICES]", (long long)e->rows, e->topk);
    return RR_OK;
}

rr_status check_width(const char *what, int32_t n)
{
    if (n < 1 || n > RR_MAX_WIDTH)
        return set_error(RR_EINVAL, "%s=%d outside [1, RR_MAX_WIDTH]", what, n);
    return RR_OK;
}

// An expert's last positions are not all in use: RR_QUANT_BLOCK - 1 at the most.
int64_t capacity_of(const rr_experts *e)
{
    const int64_t n = e->rows * e->topk;
    return round_up(n + std::min<int64_t>(e->experts, n) * (RR_QUANT_BLOCK - 1), RR_QUANT_BLOCK);
}

int64_t slots_bytes(const rr_experts *e)
{
    const int64_t blocks = slots_blocks(e->rows * e->topk);
    return blocks > 1 ? blocks * e->experts * 4 : 0;
}

int64_t quantized_ld(int64_t n) { return round_up(n, RR_QUANT_BLOCK); }
int64_t quantized_lds(int64_t n) { return round_up(quantized_ld(n) / RR_QUANT_BLOCK, 4); }
int64_t blocks_of(int64_t n) { return quantized_ld(n) / RR_QUANT_BLOCK; }

Eight eight(const void *values, const void *powers, int64_t n)
{
    return Eight{static_cast<unsigned char *>(const_cast<void *>(values)),
                 static_cast<unsigned char *>(const_cast<void *>(powers)), quantized_ld(n), quantized_lds(n)};
}

// A division by d as a multiplication: 2^shift is the least power not below d.
void divide_by(int32_t d, uint32_t *mul, uint32_t *shift)
{
    *shift = 0;
    while ((1 << *shift) < d)
        ++*shift;
    *mul = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << *shift) - uint64_t(d)) / uint64_t(d) + 1);
}

// What one buffer resource can address: a little less than 2^31 bytes, as offsets
// past the end stand for rows that are not there.
constexpr int64_t kReach = (INT64_C(1) << 31) - (INT64_C(1) << 20);

rr_status check_tensors(int dtype, int nTensors, const int64_t *count, int64_t *total)
{
    rr_status st = check_dtype(dtype);
    if (st != RR_OK)
        return st;
    if (nTensors < 0 || nTensors > RR_MAX_TENSORS)
        return set_error(RR_EINVAL, "nTensors=%d outside [0, RR_MAX_TENSORS]", nTensors);
    if (nTensors > 0 && !count)
        return set_error(RR_EINVAL, "count is null");
    int64_t n = 0;
    for (int i = 0; i < nTensors; ++i) {
        if (count[i] < 0 || count[i] > (INT64_C(1) << 40) - n)
            return set_error(RR_EINVAL, "count[%d]=%lld: below 0 or above 2^40 elements in all", i, (long long)count[i]);
        n += count[i];
    }
    *total = n;
    return RR_OK;
}

// f(table, whether it is the first) for the launches that the tensors take, at least one.
template <typename F>
void each_launch(int32_t vectors, int dtype, int nTensors, const void *const *in, void *const *out, const int64_t *count, F f)
{
    const auto from = [&](auto *const *p, int i, int64_t done) { return p ? p[i] + done * elem_size(dtype) : nullptr; };
    const char *const *src = reinterpret_cast<const char *const *>(in);
    char *const *dst = reinterpret_cast<char *const *>(out);
    bool first = true;
    int i = 0;
    int64_t done = 0;    // of tensor i, of which one launch may take a part
    do {
        ClipTable t{};
        t.bf16 = dtype == RR_BF16;
        t.vectors = vectors;
        for (; i < nTensors; ++i, done = 0) {
            done += t.add(from(src, i, done), from(dst, i, done), count[i] - done);
            if (done < count[i])
                break;
        }
        f(t, first);
        first = false;
    } while (i < nTensors);
}

// Whether one workgroup sums a call's tensors, which saves a launch: up to 64 tiles of
// 4 KiB, four for each of its waves (40000 fp32 elements in 14 tensors, with the
// clipping, 12.7 us instead of 14.5 us).
bool small(int dtype, int nTensors, const int64_t *count)
{
    int32_t launches = 0, tiles = 0;
    each_launch(kSmallVectors, dtype, nTensors, nullptr, nullptr, count, [&](const ClipTable &t, bool) {
        ++launches;
        tiles = t.tiles;
    });
    return launches == 1 && tiles <= 64;
}

// Parts of one call's sum; one: none.
int64_t square_parts(int dtype, int nTensors, const int64_t *count)
{
    if (small(dtype, nTensors, count))
        return 1;
    int64_t parts = 0;
    each_launch(kSquareVectors, dtype, nTensors, nullptr, nullptr, count, [&](const ClipTable &t, bool) { parts += t.blocks(); });
    return parts;
}

struct Range {
    uintptr_t lo, hi;
    int index;       // of the tensor, -1 for another buffer
};

// A written range that overlaps another; those that are only read do not overlap
// each other here, so that neighbours in order are all there is to look at.
rr_status check_ranges(std::vector<Range> &r)
{
    std::sort(r.begin(), r.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i].lo < r[i - 1].hi)
            return set_error(RR_EALIAS, "a written buffer overlaps another (tensors %d and %d; -1: no tensor)",
                             r[i - 1].index, r[i].index);
    return RR_OK;
}

rr_status add_range(std::vector<Range> &r, const void *p, int64_t bytes, int64_t align, const char *what, int index)
{
    if (bytes <= 0)
        return RR_OK;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (!p)
        return set_error(RR_EINVAL, "%s of tensor %d is null", what, index);
    if (lo % uintptr_t(align))
        return set_error(RR_EINVAL, "%s of tensor %d (%p) is not aligned to %lld bytes", what, index, p, (long long)align);
    r.push_back(Range{lo, lo + uintptr_t(bytes), index});
    return RR_OK;
}

// Ranges that are only read may overlap: joined to such that do not.
void join_read(std::vector<Range> &r)
{
    std::sort(r.begin(), r.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    std::vector<Range> kept;
    kept.reserve(r.size());
    for (const Range &x : r) {
        if (!kept.empty() && x.lo < kept.back().hi)
            kept.back().hi = std::max(kept.back().hi, x.hi);
        else
            kept.push_back(x);
    }
    r.swap(kept);
}

}  // namespace

extern "C" {

int64_t rr_group_route_workspace(const rr_group_router *r, int64_t rows)
{
    if (check_group_router(r) != RR_OK || check_tokens(rows) != RR_OK)
        return -1;
    set_ok();
    return group_bytes(r, rows);
}

rr_status rr_group_route(const rr_group_router *r, int dtype, int64_t rows, const void *logits,
                         const float *bias, const uint8_t *keep, int32_t *choice, float *weight,
                         float *logit, float *lse, int32_t *counts, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    rr_status st = check_group_router(r);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_tokens(rows);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), need = group_bytes(r, rows), e = r->experts, n = rows * r->topk;
    if ((st = check_workspace(workspace_bytes, need)) != RR_OK)
        return st;
    const bool softmax = r->score == RR_SOFTMAX;
    Buffers b;
    b.in(logits, rows * e * es, es, "logits");
    if (bias)
        b.in(bias, e * 4, 4, "bias");
    if (keep)
        b.in(keep, rows, 1, "keep");
    b.out(choice, n * 4, 4, "choice").out(weight, n * 4, 4, "weight").out(logit, n * 4, 4, "logit");
    if (softmax && lse)
        b.out(lse, rows * 4, 4, "lse");
    b.out(counts, (e + 1) * 4, 4, "counts").out(workspace, need, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;
    const int32_t blocks = group_route_blocks(rows, r->experts, r->groups);
    int32_t *part = blocks > 1 ? static_cast<int32_t *>(workspace) : counts;
    Launches l(stream);
    l.add(launch_group_route, GroupRouteArgs{logits, bias, keep, choice, weight, logit, softmax ? lse : nullptr, part, rows,
                                             r->experts, r->topk, r->groups, r->top_groups, r->group_best, !softmax,
                                             r->renormalize ? 1 : 0, dtype == RR_BF16, std::max(blocks, 1), r->scale});
    if (blocks > 1)
        l.add(launch_count_sum, CountSumArgs{part, counts, blocks, r->experts});
    return l.finish();
}

rr_status rr_route_bias(const rr_group_router *r, const int32_t *const *counts, int nRanks, float rate,
                        const float *bias, float *out, void *stream)
{
    rr_status st = check_group_router(r);
    if (st != RR_OK)
        return st;
    if (nRanks < 1 || nRanks > RR_MAX_SHARDS)
        return set_error(RR_EINVAL, "nRanks=%d outside [1, RR_MAX_SHARDS]", nRanks);
    if (!counts)
        return set_error(RR_EINVAL, "an array of rank pointers is null");
    if (!isfinite(rate))
        return set_error(RR_EINVAL, "rate is not finite");
    const int64_t e = r->experts;
    RouteBiasArgs a{};
    Buffers b;
    for (int i = 0; i < nRanks; ++i) {
        b.in(counts[i], (e + 1) * 4, 4, "counts");
        a.counts[i] = counts[i];
    }
    b.out(out, e * 4, 4, "out");
    if (bias != out)
        b.in(bias, e * 4, 4, "bias");
    if ((st = b.check()) != RR_OK)
        return st;
    a.bias = bias;
    a.out = out;
    a.ranks = nRanks;
    a.experts = r->experts;
    a.rate = rate;
    Launches l(stream);
    l.add(launch_route_bias, a);
    return l.finish();
}

rr_status rr_group_route_grad(const rr_group_router *r, int dtype, int64_t rows, const void *logits,
                              const int32_t *choice, const float *logit, const float *lse,
                              const float *grad_weight, void *dlogits, void *stream)
{
    rr_status st = check_group_router(r);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_tokens(rows);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), e = r->experts, n = rows * r->topk;
    const bool whole = r->score == RR_SOFTMAX && !r->renormalize;
    Buffers b;
    if (whole)
        b.in(logits, rows * e * es, es, "logits").in(lse, rows * 4, 4, "lse");
    b.in(choice, n * 4, 4, "choice").in(logit, n * 4, 4, "logit").in(grad_weight, n * 4, 4, "grad_weight");
    b.out(dlogits, rows * e * es, es, "dlogits");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_group_grad, GroupGradArgs{whole ? logits : nullptr, choice, logit, whole ? lse : nullptr, grad_weight,
                                           dlogits, rows, r->experts, r->topk, r->score == RR_SIGMOID,
                                           r->renormalize ? 1 : 0, dtype == RR_BF16, r->scale});
    return l.finish();
}

int64_t rr_expert_capacity(const rr_experts *e)
{
    if (check_experts(e) != RR_OK)
        return -1;
    set_ok();
    return capacity_of(e);
}

int64_t rr_expert_workspace(const rr_experts *e)
{
    if (check_experts(e) != RR_OK)
        return -1;
    set_ok();
    return slots_bytes(e);
}

rr_status rr_expert_slots(const rr_experts *e, const int32_t *choice, int32_t *slot, int32_t *source,
                          int32_t *offset, int32_t *count, void *workspace, int64_t workspace_bytes,
                          void *stream)
{
    rr_status st = check_experts(e);
    if (st != RR_OK)
        return st;
    const int64_t n = e->rows * e->topk, need = slots_bytes(e), capacity = capacity_of(e);
    if ((st = check_workspace(workspace_bytes, need)) != RR_OK)
        return st;
    Buffers b;
    b.in(choice, n * 4, 4, "choice").out(slot, n * 4, 4, "slot").out(source, capacity * 4, 4, "source");
    b.out(offset, (int64_t(e->experts) + 1) * 4, 4, "offset").out(count, int64_t(e->experts) * 4, 4, "count");
    b.out(workspace, need, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;
    const int32_t blocks = slots_blocks(n);
    const SlotsArgs a{choice, slot, source, offset, count, blocks > 1 ? static_cast<int32_t *>(workspace) : nullptr,
                      int32_t(n), int32_t(capacity), e->experts, e->first, blocks};
    Launches l(stream);
    if (blocks > 1)
        l.add(launch_slots_count, a);
    l.add(launch_slots, a);
    return l.finish();
}

int64_t rr_quantized_ld(int64_t n) { return quantized_ld(n); }
int64_t rr_quantized_lds(int64_t n) { return quantized_lds(n); }

rr_status rr_quantize_rows(int dtype, int64_t rows, int32_t dim, const void *x, void *values,
                           void *powers, void *stream)
{
    rr_status st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("dim", dim);
    if (st != RR_OK)
        return st;
    if (rows < 0 || rows > INT32_MAX)
        return set_error(RR_EINVAL, "rows=%lld outside [0, 2^31)", (long long)rows);
    const int64_t es = elem_size(dtype);
    Buffers b;
    b.in(x, rows * dim * es, es, "x");
    b.out(values, rows * quantized_ld(dim), 16, "values").out(powers, rows * quantized_lds(dim), 4, "powers");
    if ((st = b.check()) != RR_OK)
        return st;
    if (rows == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_quantize_rows, QuantizeRowsArgs{x, eight(values, powers, dim), rows, dim, dtype == RR_BF16});
    return l.finish();
}

rr_status rr_quantize_slots(const rr_experts *e, int dtype, int32_t dim, const void *x, int gather,
                            const float *weight, const int32_t *source, const int32_t *offset,
                            void *values, void *powers, void *stream)
{
    rr_status st = check_experts(e);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("dim", dim);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), n = e->rows * e->topk, capacity = capacity_of(e);
    Buffers b;
    b.in(x, (gather ? e->rows : capacity) * dim * es, es, "x");
    if (weight)
        b.in(weight, n * 4, 4, "weight");
    b.in(source, capacity * 4, 4, "source").in(offset, (int64_t(e->experts) + 1) * 4, 4, "offset");
    b.out(values, dim * quantized_ld(capacity), 16, "values").out(powers, dim * quantized_lds(capacity), 4, "powers");
    if ((st = b.check()) != RR_OK)
        return st;
    if (n == 0)
        return set_ok();
    uint32_t mul, shift;
    divide_by(e->topk, &mul, &shift);
    Launches l(stream);
    QuantizeSlotsArgs a{x, weight, source, offset, eight(values, powers, capacity), e->rows, int32_t(capacity), e->experts,
                        dim, gather ? 1 : 0, dtype == RR_BF16, mul, shift, 0, 0};
    const int32_t blocks = int32_t(blocks_of(capacity)), most = kSlotBlocks / int32_t(blocks_of(dim));
    for (; a.block0 < blocks; a.block0 += a.blocks) {
        a.blocks = std::min(blocks - a.block0, most);
        l.add(launch_quantize_slots, a);
    }
    return l.finish();
}

rr_status rr_quantize_weight(int dtype, int32_t experts, int32_t n, int32_t k, const void *w, void *values,
                             void *powers, void *tvalues, void *tpowers, void *stream)
{
    rr_status st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("n", n);
    if (st == RR_OK)
        st = check_width("k", k);
    if (st != RR_OK)
        return st;
    if (experts < 1 || experts > RR_MAX_EXPERTS)
        return set_error(RR_EINVAL, "experts=%d outside [1, RR_MAX_EXPERTS]", experts);
    const int64_t es = elem_size(dtype), m = experts;
    Buffers b;
    b.in(w, m * n * k * es, es, "w");
    b.out(values, m * n * quantized_ld(k), 16, "values").out(powers, m * blocks_of(n) * quantized_lds(k), 4, "powers");
    if (tvalues)
        b.out(tvalues, m * k * quantized_ld(n), 16, "tvalues").out(tpowers, m * blocks_of(k) * quantized_lds(n), 4, "tpowers");
    if ((st = b.check()) != RR_OK)
        return st;
    Launches l(stream);
    l.add(launch_quantize_weight, QuantizeWeightArgs{w, eight(values, powers, k), eight(tvalues, tpowers, n), experts, n, k,
                                                     dtype == RR_BF16});
    return l.finish();
}

rr_status rr_expert_product(const rr_experts *e, int dtype, int32_t n, int32_t k, int gather,
                            const void *x, const void *x_powers, const void *w, const void *w_powers,
                            const float *weight, const int32_t *source, const int32_t *offset,
                            const int32_t *count, void *out, void *stream)
{
    rr_status st = check_experts(e);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("n", n);
    if (st == RR_OK)
        st = check_width("k", k);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), m = e->experts, choices = e->rows * e->topk, capacity = capacity_of(e);
    const int64_t rows = gather ? e->rows : capacity;
    if (gather && rows * quantized_ld(k) > kReach)
        return set_error(RR_EINVAL, "rows=%lld, k=%d: gathered values above 2^31 - 2^20 bytes", (long long)rows, k);
    Buffers b;
    b.in(x, rows * quantized_ld(k), 16, "x").in(x_powers, rows * quantized_lds(k), 4, "x_powers");
    b.in(w, m * n * quantized_ld(k), 16, "w").in(w_powers, m * blocks_of(n) * quantized_lds(k), 4, "w_powers");
    if (weight)
        b.in(weight, choices * 4, 4, "weight");
    b.in(source, capacity * 4, 4, "source").in(offset, (m + 1) * 4, 4, "offset").in(count, m * 4, 4, "count");
    b.out(out, capacity * n * es, es, "out");
    if ((st = b.check()) != RR_OK)
        return st;
    if (choices == 0)
        return set_ok();
    uint32_t mul, shift;
    divide_by(e->topk, &mul, &shift);
    Launches l(stream);
    l.add(launch_expert_product, ExpertProductArgs{eight(w, w_powers, k), eight(x, x_powers, k), weight, source, offset,
                                                   count, out, rows, n, k, e->experts, e->topk, int32_t(capacity),
                                                   gather ? 1 : 0, dtype == RR_BF16, int32_t(choices), mul, shift});
    return l.finish();
}

rr_status rr_expert_weight_grad(const rr_experts *e, int dtype, int32_t n, int32_t k, const void *dy,
                                const void *dy_powers, const void *x, const void *x_powers,
                                const int32_t *offset, const int32_t *count, void *dw, void *stream)
{
    rr_status st = check_experts(e);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("n", n);
    if (st == RR_OK)
        st = check_width("k", k);
    if (st != RR_OK)
        return st;
    const int64_t es = elem_size(dtype), m = e->experts, capacity = capacity_of(e);
    const int64_t ld = quantized_ld(capacity), lds = quantized_lds(capacity);
    if (ld > kReach / 256)
        return set_error(RR_EINVAL, "rows=%lld, topk=%d: a capacity of %lld positions above 2^23 - 2^12",
                         (long long)e->rows, e->topk, (long long)capacity);
    Buffers b;
    b.in(dy, n * ld, 16, "dy").in(dy_powers, n * lds, 4, "dy_powers");
    b.in(x, k * ld, 16, "x").in(x_powers, k * lds, 4, "x_powers");
    b.in(offset, (m + 1) * 4, 4, "offset").in(count, m * 4, 4, "count");
    b.out(dw, m * n * k * es, es, "dw");
    if ((st = b.check()) != RR_OK)
        return st;
    Launches l(stream);
    l.add(launch_expert_grad, ExpertGradArgs{eight(dy, dy_powers, capacity), eight(x, x_powers, capacity), offset, count,
                                             dw, n, k, e->experts, int32_t(capacity), dtype == RR_BF16});
    return l.finish();
}

rr_status rr_expert_combine(const rr_experts *e, int values_dtype, int dtype, int32_t dim, const void *values,
                            const int32_t *slot, const float *weight, void *y, void *stream)
{
    rr_status st = check_experts(e);
    if (st == RR_OK)
        st = check_dtype(values_dtype);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("dim", dim);
    if (st != RR_OK)
        return st;
    const int64_t vs = elem_size(values_dtype), es = elem_size(dtype), n = e->rows * e->topk, capacity = capacity_of(e);
    Buffers b;
    b.in(values, capacity * dim * vs, vs, "values").in(slot, n * 4, 4, "slot");
    if (weight)
        b.in(weight, n * 4, 4, "weight");
    b.out(y, e->rows * dim * es, es, "y");
    if ((st = b.check()) != RR_OK)
        return st;
    if (n == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_combine_rows, CombineRowsArgs{values, slot, weight, y, e->rows, int32_t(capacity), e->topk, dim,
                                               values_dtype == RR_BF16, dtype == RR_BF16});
    return l.finish();
}

rr_status rr_expert_combine_grad(const rr_experts *e, int values_dtype, int dtype, int32_t dim,
                                 const void *values, const int32_t *slot, const void *dy, float *grad_weight,
                                 void *stream)
{
    rr_status st = check_experts(e);
    if (st == RR_OK)
        st = check_dtype(values_dtype);
    if (st == RR_OK)
        st = check_dtype(dtype);
    if (st == RR_OK)
        st = check_width("dim", dim);
    if (st != RR_OK)
        return st;
    const int64_t vs = elem_size(values_dtype), es = elem_size(dtype), n = e->rows * e->topk, capacity = capacity_of(e);
    Buffers b;
    b.in(values, capacity * dim * vs, vs, "values").in(slot, n * 4, 4, "slot").in(dy, e->rows * dim * es, es, "dy");
    b.out(grad_weight, n * 4, 4, "grad_weight");
    if ((st = b.check()) != RR_OK)
        return st;
    if (n == 0)
        return set_ok();
    Launches l(stream);
    l.add(launch_combine_grad, CombineGradArgs{values, slot, dy, grad_weight, e->rows, int32_t(capacity), e->topk, dim,
                                               values_dtype == RR_BF16, dtype == RR_BF16});
    return l.finish();
}

int64_t rr_grad_workspace(int dtype, int nTensors, const int64_t *count)
{
    int64_t total;
    if (check_tensors(dtype, nTensors, count, &total) != RR_OK)
        return -1;
    set_ok();
    const int64_t parts = square_parts(dtype, nTensors, count);
    return parts > 1 ? parts * 8 : 0;
}

rr_status rr_grad_square_sum(int dtype, int nTensors, const void *const *in, const int64_t *count,
                             double *sum, void *workspace, int64_t workspace_bytes, void *stream)
try {
    int64_t total;
    rr_status st = check_tensors(dtype, nTensors, count, &total);
    if (st != RR_OK)
        return st;
    if (nTensors > 0 && !in)
        return set_error(RR_EINVAL, "in is null");
    const int64_t es = elem_size(dtype), parts = square_parts(dtype, nTensors, count);
    const int64_t need = parts > 1 ? parts * 8 : 0;
    if ((st = check_workspace(workspace_bytes, need)) != RR_OK)
        return st;
    std::vector<Range> r;
    for (int i = 0; i < nTensors && st == RR_OK; ++i)
        st = add_range(r, in[i], count[i] * es, es, "in", i);
    if (st != RR_OK)
        return st;
    join_read(r);
    Buffers b;
    b.out(sum, 8, 8, "sum").out(workspace, need, 256, "workspace");
    if ((st = b.check()) != RR_OK)
        return st;
    if ((st = add_range(r, sum, 8, 8, "sum", -1)) != RR_OK || (st = add_range(r, workspace, need, 256, "workspace", -1)) != RR_OK ||
        (st = check_ranges(r)) != RR_OK)
        return st;
    double *part = parts > 1 ? static_cast<double *>(workspace) : sum;
    Launches l(stream);
    // tensors that the cache holds are read from it when they are scaled; larger ones are
    // summed past the caches, and so is what is scaled (600 million bf16 elements in 300
    // tensors: 596 us, with all loads kept 635 us; 50 million fp32 elements 97 us, summed past
    // the caches 102 us)
    const int32_t stream_it = total * es > kCacheBytes;
    if (small(dtype, nTensors, count)) {
        each_launch(kSmallVectors, dtype, nTensors, in, nullptr, count,
                    [&](const ClipTable &t, bool) { l.add(launch_square_small, SquareSumArgs{sum, 0, 0, t}); });
        return l.finish();
    }
    int64_t done = 0;
    each_launch(kSquareVectors, dtype, nTensors, in, nullptr, count, [&](const ClipTable &t, bool) {
        l.add(launch_square_sum, SquareSumArgs{part + done, stream_it, 0, t});
        done += t.blocks();
    });
    if (parts > 1)
        l.add(launch_sum_parts, SumPartsArgs{part, sum, int32_t(parts)});
    return l.finish();
} catch (const std::bad_alloc &) {
    return set_error(RR_EINVAL, "no host memory for the checks of %d tensors", nTensors);
}

rr_status rr_grad_clip(int dtype, const double *const *sums, int nSums, double max_norm, int nTensors,
                       const void *const *in, void *const *out, const int64_t *count, float *norm,
                       void *stream)
try {
    int64_t total;
    rr_status st = check_tensors(dtype, nTensors, count, &total);
    if (st != RR_OK)
        return st;
    if (nSums < 1 || nSums > RR_MAX_SHARDS)
        return set_error(RR_EINVAL, "nSums=%d outside [1, RR_MAX_SHARDS]", nSums);
    if (!sums || (nTensors > 0 && (!in || !out)))
        return set_error(RR_EINVAL, "an array of pointers is null");
    if (!(max_norm >= 0.0) || !isfinite(max_norm))
        return set_error(RR_EINVAL, "max_norm is below 0 or not finite");
    const int64_t es = elem_size(dtype);
    Buffers b;
    for (int i = 0; i < nSums; ++i)
        b.in(sums[i], 8, 8, "sums");
    b.out(norm, 4, 4, "norm");
    if ((st = b.check()) != RR_OK)
        return st;
    // what is read: the sums, and the tensors that are not scaled in place
    std::vector<Range> r, written;
    for (int i = 0; i < nSums && st == RR_OK; ++i)
        st = add_range(r, sums[i], 8, 8, "sums", -1);
    for (int i = 0; i < nTensors && st == RR_OK; ++i) {
        if (count[i] > 0 && in[i] != out[i])
            st = add_range(r, in[i], count[i] * es, es, "in", i);
        if (st == RR_OK)
            st = add_range(written, out[i], count[i] * es, es, "out", i);
    }
    if (st == RR_OK)
        st = add_range(written, norm, 4, 4, "norm", -1);
    if (st != RR_OK)
        return st;
    join_read(r);
    r.insert(r.end(), written.begin(), written.end());
    if ((st = check_ranges(r)) != RR_OK)
        return st;
    Launches l(stream);
    each_launch(kClipVectors, dtype, nTensors, in, out, count, [&](const ClipTable &t, bool first) {
        ClipArgs a{};
        for (int n = 0; n < nSums; ++n)
            a.sums[n] = sums[n];
        a.max_norm = max_norm;
        a.norm = first ? norm : nullptr;
        a.n_sums = nSums;
        a.t = t;
        l.add(launch_clip, a);
    });
    return l.finish();
} catch (const std::bad_alloc &) {
    return set_error(RR_EINVAL, "no host memory for the checks of %d tensors", nTensors);
}

}  // extern "C"
