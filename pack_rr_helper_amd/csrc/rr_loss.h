// rr_loss.h -- what the host layer of the sharded losses (rr_loss.cpp) shares
// with their kernels (rr_vocab.hip, rr_route.hip) and with the plans of
// rr_api.cpp.  Not part of the public ABI.
#pragma once

#include <stdint.h>
#include <string.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "rr.h"

namespace rr {

// One launch of a loss operator: the function that enqueues it and its
// arguments by value.  A plan records it as it is.
struct Op {
    hipError_t (*launch)(const Op &, hipStream_t);
    alignas(16) char args[496];

    template <typename A>
    static Op make(hipError_t (*launch)(const Op &, hipStream_t), const A &a)
    {
        static_assert(sizeof(A) <= sizeof(Op::args) && std::is_trivially_copyable<A>::value, "");
        Op op{};
        op.launch = launch;
        memcpy(op.args, &a, sizeof a);
        return op;
    }
    template <typename A>
    A get() const
    {
        A a;
        memcpy(&a, args, sizeof a);
        return a;
    }
};

// In rr_api.cpp: enqueue an op, or append it to the plan that this thread
// records; the error state of the calling thread.
hipError_t emit_op(const Op &op, hipStream_t stream);
rr_status op_failed(hipError_t e);
rr_status set_error(rr_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
rr_status set_ok();

// ---------------------------------------------------------------------------
// Vocabulary head.  Every product is C[j][i] = sum_k A[i][k] * B[j][k], an
// operand lying as [i or j][k], or tall as [k][i or j]: "i" (the fast axis of
// C) runs over the vocabulary for the logits and over dim for dw and dx.
// ---------------------------------------------------------------------------

struct Product {
    const void *a, *b;   // [ni][lda], [nj][ldb]; tall [nk][lda], [nk][ldb]
    int64_t lda, ldb;    // elements
    int32_t ni, nj, nk;
    int32_t bf16;        // element type of a and b
};

// Rows that start at, and are a multiple of, 16 bytes.
inline bool in_chunks(const void *p, int64_t ld, int64_t es)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0;
}

// The logits' softmax statistics per part of the vocabulary.
struct StatsArgs {
    Product p;           // a = w, b = x
    float scale;
    float2 *part;        // [parts][nj]
};
// Partial statistics of one row.
int64_t stats_parts(const Product &p);
hipError_t launch_stats(const Op &, hipStream_t);

// stats[row] from its parts, and the logits of the entries of this shard.
struct StatsDoneArgs {
    const float2 *part;
    const void *x, *w;
    const int64_t *index;
    float2 *stats;
    float *picked;
    int64_t first;
    int32_t parts, rows, topk, vocab, dim, bf16;
    float scale;
};
hipError_t launch_stats_done(const Op &, hipStream_t);

struct CombineArgs {
    const float2 *stats[RR_MAX_SHARDS];
    const float *picked[RR_MAX_SHARDS];
    int32_t shards, rows, topk, bf16;
    int64_t total;
    float scale;
    const int64_t *index;
    const void *teacher;
    float *lse, *logit, *prob, *loss;
};
hipError_t launch_cross_entropy(const Op &, hipStream_t);
hipError_t launch_distill(const Op &, hipStream_t);

// What makes a row's (lse in units of ln 2, grad * scale), both 0 for a row
// without a gradient (no target, or grad * scale = 0); of distillation, row is
// filled with them first.
struct RowsArgs {
    const int64_t *index;
    const float *lse, *prob, *grad;  // prob: null for cross entropy
    int32_t rows, topk;
    int64_t total;
    float scale;
    float2 *row;
};
// A matrix copied to rows that start at multiples of 16 bytes and end in zeros.
struct AlignArgs {
    const void *in;      // [rows][cols]
    void *out;           // [rows][ldo]
    int64_t rows, ldo;
    int32_t cols;
};

// dz of one piece of the vocabulary; of distillation without its targets.
// Operands in 16-byte chunks.
struct DzArgs {
    Product p;           // a = the piece of w, b = x
    RowsArgs rows;
    const float *logit;
    int64_t first;       // the piece's first entry of the vocabulary
    void *dz;            // [nj][ldz]
    int64_t ldz;
    AlignArgs x;         // in not null: x copied beside, rows without a gradient as zeros
};
hipError_t launch_dz(const Op &, hipStream_t);

// dz at the targets of one piece, for distillation.
struct TargetArgs {
    const int64_t *index;
    const float *logit, *prob;
    const float2 *row;
    int32_t rows, topk, count, bf16;  // entries [first, first + count) of the vocabulary
    int64_t first;
    void *dz;
    int64_t ldz;
};
hipError_t launch_targets(const Op &, hipStream_t);

// factors: fill rows.row; x.in, w.in: null where there is nothing to copy.  Rows
// of x without a gradient become zeros.
struct PrepareArgs {
    RowsArgs rows;
    AlignArgs x, w;
    int32_t factors, bf16;
};
hipError_t launch_prepare(const Op &, hipStream_t);

// A product, A tall, stored as the element type, or in fp32 as one sum for each
// of the `splits` parts of k.  Operands in 16-byte chunks.
struct StoreArgs {
    Product p;
    void *out;           // [nj][ldo]
    int64_t ldo;
    float *acc;          // not null: [splits][nj][lda] instead of out
    int64_t lda;         // a multiple of 4
    int32_t splits, add; // add: to what acc holds
};
// dx = (w, dz), dw = (x, dz), the second with a tall B too.
struct StoresArgs {
    StoreArgs x, w;
};
int32_t product_splits(const Product &p, bool tall_b);
hipError_t launch_stores(const Op &, hipStream_t);

// out = the sum of the partial sums (none: zero).
struct GatherArgs {
    const float *acc;    // [splits][rows][lda]
    void *out;           // [rows][dim]
    int64_t rows, lda;
    int32_t dim, splits;
};
// out: null where there is nothing to do, not for both.
struct GathersArgs {
    GatherArgs x, w;
    int32_t bf16;
};
hipError_t launch_gather(const Op &, hipStream_t);

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

struct RouteArgs {
    const void *logits;
    const uint8_t *keep;
    int32_t *choice;
    float *weight, *lse;
    int32_t *counts;     // of one workgroup: the results; else [blocks][experts + 1]
    float *prob_sum;     //                             else [blocks][experts]
    int64_t rows;
    int32_t experts, topk, renormalize, bf16, blocks;
};
int32_t route_blocks(int64_t rows, int32_t experts);
hipError_t launch_route(const Op &, hipStream_t);

struct RouteSumArgs {
    const int32_t *part_counts;
    const float *part_sum;
    int32_t *counts;
    float *prob_sum;
    int32_t blocks, experts;
};
hipError_t launch_route_sum(const Op &, hipStream_t);

struct BalanceArgs {
    const int32_t *counts[RR_MAX_SHARDS];
    const float *prob_sum[RR_MAX_SHARDS];
    int32_t ranks, experts, topk;
    float *loss, *slope;
};
hipError_t launch_balance(const Op &, hipStream_t);

struct RouteGradArgs {
    const void *logits;
    const uint8_t *keep;
    const int32_t *choice;
    const float *weight, *lse, *slope, *grad_loss, *grad_weight;
    void *dlogits;
    int64_t rows;
    int32_t experts, topk, renormalize, bf16;
};
hipError_t launch_route_grad(const Op &, hipStream_t);

}  // namespace rr
