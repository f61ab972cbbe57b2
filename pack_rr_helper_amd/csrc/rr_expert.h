// rr_expert.h -- what the host layer of the expert layer and the clipping
// (rr_expert.cpp) shares with their kernels (rr_group_route.hip, rr_slots.hip,
// rr_expert_product.hip, rr_clip.hip).  Not part of the public ABI.
#pragma once

#include "rr_loss.h"

namespace rr {

// Bytes of the last level cache.
constexpr int64_t kCacheBytes = INT64_C(256) << 20;

// ---------------------------------------------------------------------------
// Routing in groups
// ---------------------------------------------------------------------------

struct GroupRouteArgs {
    const void *logits;
    const float *bias;
    const uint8_t *keep;
    int32_t *choice;
    float *weight, *logit, *lse;
    int32_t *counts;     // of one workgroup: the result; else [blocks][experts + 1]
    int64_t rows;
    int32_t experts, topk, groups, top_groups, group_best, sigmoid, renormalize, bf16, blocks;
    float scale;
};
int32_t group_route_blocks(int64_t rows, int32_t experts, int32_t groups);
hipError_t launch_group_route(const Op &, hipStream_t);

struct CountSumArgs {
    const int32_t *part;
    int32_t *counts;
    int32_t blocks, experts;
};
hipError_t launch_count_sum(const Op &, hipStream_t);

struct RouteBiasArgs {
    const int32_t *counts[RR_MAX_SHARDS];
    const float *bias;
    float *out;
    int32_t ranks, experts;
    float rate;
};
hipError_t launch_route_bias(const Op &, hipStream_t);

struct GroupGradArgs {
    const void *logits;
    const int32_t *choice;
    const float *logit, *lse, *grad_weight;
    void *dlogits;
    int64_t rows;
    int32_t experts, topk, sigmoid, renormalize, bf16;
    float scale;
};
hipError_t launch_group_grad(const Op &, hipStream_t);

// ---------------------------------------------------------------------------
// Slots of an expert layer, and what moves rows to and from them
// ---------------------------------------------------------------------------

struct SlotsArgs {
    const int32_t *choice;
    int32_t *slot, *source, *offset, *count;
    int32_t *part;       // [blocks][experts], more than one workgroup only
    int32_t choices, capacity, experts, first, blocks;
};
int32_t slots_blocks(int64_t choices);
hipError_t launch_slots_count(const Op &, hipStream_t);
hipError_t launch_slots(const Op &, hipStream_t);

// One operand in 8 bits.
struct Eight {
    unsigned char *values, *powers;
    int64_t ld, lds;
};

struct QuantizeRowsArgs {
    const void *x;
    Eight to;
    int64_t rows;
    int32_t dim, bf16;
};
hipError_t launch_quantize_rows(const Op &, hipStream_t);

struct QuantizeSlotsArgs {
    const void *x;
    const float *weight;
    const int32_t *source, *offset;
    Eight to;
    int64_t rows;
    int32_t capacity, experts, dim, gather, bf16;
    uint32_t topk_mul, topk_shift;  // n / topk = (high word of topk_mul * n + n) >> topk_shift, n < 2^31
    int32_t block0, blocks;  // this launch's blocks of positions
};
// Blocks of 128 x 128 in a launch: one has less than 2^32 threads.
constexpr int32_t kSlotBlocks = 1 << 20;
hipError_t launch_quantize_slots(const Op &, hipStream_t);

struct QuantizeWeightArgs {
    const void *w;
    Eight to, turned;    // turned.values may be null
    int32_t experts, n, k, bf16;
};
hipError_t launch_quantize_weight(const Op &, hipStream_t);

struct CombineRowsArgs {
    const void *values;
    const int32_t *slot;
    const float *weight;
    void *y;
    int64_t rows;
    int32_t capacity, topk, dim, from_bf16, bf16;
};
hipError_t launch_combine_rows(const Op &, hipStream_t);

struct CombineGradArgs {
    const void *values;
    const int32_t *slot;
    const void *dy;
    float *grad_weight;
    int64_t rows;
    int32_t capacity, topk, dim, from_bf16, bf16;
};
hipError_t launch_combine_grad(const Op &, hipStream_t);

// ---------------------------------------------------------------------------
// Products in 8 bits
// ---------------------------------------------------------------------------

struct ExpertProductArgs {
    Eight w, x;
    const float *weight;
    const int32_t *source, *offset, *count;
    void *out;
    int64_t rows;        // of x
    int32_t n, k, experts, topk, capacity, gather, bf16, choices;
    uint32_t topk_mul, topk_shift;  // as above
};
hipError_t launch_expert_product(const Op &, hipStream_t);

struct ExpertGradArgs {
    Eight dy, x;
    const int32_t *offset, *count;
    void *dw;
    int32_t n, k, experts, capacity, bf16;
};
hipError_t launch_expert_grad(const Op &, hipStream_t);

// ---------------------------------------------------------------------------
// Gradient norm
// ---------------------------------------------------------------------------

// Tensors of one launch; those without elements are left out.  And its tiles: a launch
// has less than 2^32 threads.
constexpr int32_t kClipTensors = 90, kClipTiles = 1 << 23;

struct ClipTable {
    int32_t tile0[kClipTensors];  // tiles of the tensors before
    int32_t tensors, tiles, bf16, vectors;  // vectors: of 16 bytes, of a thread in a tile
    const void *in[kClipTensors];
    void *out[kClipTensors];
    int64_t count[kClipTensors];

    // Adds a tensor, or as much of its start as there is room for; the elements added.
    int64_t add(const void *in, void *out, int64_t count);
    // The launch's workgroups, one for each tile.
    int32_t blocks() const { return tiles > 0 ? tiles : 1; }
};
// Tiles of 32 KiB to sum, of 8 KiB to scale, of 4 KiB where one workgroup sums them.
constexpr int32_t kSquareVectors = 8, kClipVectors = 2, kSmallVectors = 1;

struct SquareSumArgs {
    double *part;        // one per workgroup of this launch
    int32_t stream, reserved;  // more than the last level cache holds
    ClipTable t;
};
hipError_t launch_square_sum(const Op &, hipStream_t);
// All by one workgroup; part: the sum.
hipError_t launch_square_small(const Op &, hipStream_t);

struct SumPartsArgs {
    const double *part;
    double *sum;
    int32_t parts;
};
hipError_t launch_sum_parts(const Op &, hipStream_t);

struct ClipArgs {
    const double *sums[RR_MAX_SHARDS];
    double max_norm;
    float *norm;         // null: another launch's
    int32_t n_sums, reserved;
    ClipTable t;
};
hipError_t launch_clip(const Op &, hipStream_t);

}  // namespace rr
