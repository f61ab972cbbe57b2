// rr_vocab.hip -- gfx950 kernels of the sharded vocabulary head: the logits'
// softmax statistics and their gradient, without keeping the logits.
//
// The four products of a training step (logits for the statistics, logits
// again for dz, dw = dz^T x, dx = dz w) are tiles on the matrix cores
// (rr_product.h) with different ends.  The vocabulary runs along the registers
// of a tile, so a row's maximum and sum over the tile are taken within a lane
// and over the four lane groups of a wave.
#include "rr_lanes.h"
#include "rr_product.h"

#include <math.h>

namespace rr {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;

template <bool BF16>
__device__ __forceinline__ float load(const void *p, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float((unsigned)static_cast<const unsigned short *>(p)[i] << 16);
    else
        return static_cast<const float *>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store(void *p, int64_t i, float v)
{
    if constexpr (BF16)
        static_cast<__bf16 *>(p)[i] = (__bf16)v;
    else
        static_cast<float *>(p)[i] = v;
}

// exp(x - top) where top may be infinite: -inf - -inf counts as nothing.
__device__ __forceinline__ float exp_below(float x, float top)
{
    return x == -INFINITY ? 0.0f : expf(x - top);
}

// One wave's rows of a tile: part = the logits' maximum and sum of exponentials,
// max z and sum exp(z - max).  Bound by the product, and by the weights' bytes
// for few rows (48 x 2048 x 50001 in bf16: 33 us, 6.2 TB/s from the last level
// cache); the exponentials take a tenth of a tile's time at dim 2048.
template <typename T>
__global__ __launch_bounds__(T::kThreads) void stats_kernel(StatsArgs a, int tiles_i, int tiles_j)
{
    __shared__ __attribute__((aligned(1024))) char lds[T::kLdsBytes];
    int ti, tj;
    tile_at(blockIdx.x, gridDim.x, tiles_i, tiles_j, ti, tj);
    const int i0 = ti * T::TI, j0 = tj * T::TJ, part = ti * (T::TI / (T::FI * 16)) + T::wave_i() / (T::FI * 16);
    typename T::Pipe pipe;
    pipe.start(a.p, i0, j0, 0, (a.p.nk + T::kStep - 1) / T::kStep, lds);
    typename T::Acc acc;
    acc.clear();
    pipe.finish(acc);
    // z = scale * acc; the largest is at the largest of acc once scale is
    // positive.  A scale of 0 goes into acc: -inf past the vocabulary stays what
    // it is.
    const float scale = a.scale == 0.0f ? 1.0f : fabsf(a.scale), c = scale * kLog2e;
    if (a.scale <= 0.0f) {
        const float by = a.scale == 0.0f ? 0.0f : -1.0f;
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int j = 0; j < T::FJ; ++j)
                acc.c[i][j] *= by;
    }
    if (i0 + T::TI > a.p.ni) {
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + T::lane_i(i) + e >= a.p.ni) {
#pragma unroll
                    for (int j = 0; j < T::FJ; ++j)
                        acc.c[i][j][e] = -INFINITY;
                }
    }
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fmaxf(top, acc.c[i][j][e]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : -(top * c);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc.c[i][j][e], c, base));
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        // Every term has the rounding of base in its exponent, which the
        // largest's own exponent shows; the largest counts 1.  At huge logits
        // that rounding is past a float's range, and there only the largest counts.
        const float off = __builtin_fmaf(top, c, base);
        const bool far = !(fabsf(off) < 64.0f);
        sum = far ? sum : sum * __builtin_amdgcn_exp2f(-off);
        if (top != -INFINITY && (sum < 1.0f || (far && sum == sum)))
            sum = 1.0f;
        const int row = j0 + T::lane_j(j);
        if (threadIdx.x % 64 < 16 && row < a.p.nj)
            a.part[int64_t(part) * a.p.nj + row] = float2{top == -INFINITY ? top : top * scale, sum};
    }
}

// (top, sum) of the union of two sets of logits.
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float top = fmaxf(a.x, b.x);
    const float fa = a.x == top ? 1.0f : exp_below(a.x, top), fb = b.x == top ? 1.0f : exp_below(b.x, top);
    return float2{top, a.y * fa + b.y * fb};
}

// x . w over G lanes, x and w in the element type; the sum in every lane.
template <bool BF16, int G>
__device__ __forceinline__ float dot(const char *x, const char *w, int dim)
{
    constexpr int kEs = BF16 ? 2 : 4, kPer = 16 / kEs;
    float z = 0.0f;
#pragma unroll 4
    for (int k = threadIdx.x % G * kPer; k < dim; k += G * kPer) {
        const u32x4 u = load_chunk<kEs>(x + k * kEs, (dim - k) * kEs), v = load_chunk<kEs>(w + k * kEs, (dim - k) * kEs);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {
                z = __builtin_fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), z);
                z = __builtin_fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(v[e] & 0xffff0000u), z);
            } else {
                z = __builtin_fmaf(__uint_as_float(u[e]), __uint_as_float(v[e]), z);
            }
        }
    }
    return lanes_sum<G>(z);
}

// picked[n] by G lanes, x being n's row.
template <bool BF16, int G>
__device__ __forceinline__ void pick(const StatsDoneArgs &a, int64_t n, const char *x)
{
    const int64_t i = a.index[n] - a.first;
    float z = 0.0f;
    if (i >= 0 && i < a.vocab)
        z = dot<BF16, G>(x, static_cast<const char *>(a.w) + i * a.dim * (BF16 ? 2 : 4), a.dim) * a.scale;
    if (threadIdx.x % G == 0)
        a.picked[n] = z;
}

constexpr int kRowEntries = 64;  // of a row that one workgroup takes

// The first `joins` workgroups join the parts of `wide` rows each (a power of
// two up to 64), the others compute the logits of one entry per G lanes.  Of
// many entries a row, a workgroup takes up to 64 and keeps the row's x in LDS
// (SHARED), which leaves the first-level cache to w.  Bound by the entries' rows
// of w: 4096 x 64 of 4 KiB in 118-134 us, 8 TB/s from the last level cache.
template <bool BF16, int G, bool SHARED>
__global__ __launch_bounds__(kThreads) void stats_done_kernel(StatsDoneArgs a, int joins, int wide)
{
    __shared__ float2 sums[kThreads];
    if (int(blockIdx.x) < joins) {
        const int r = threadIdx.x % wide, t0 = threadIdx.x / wide, step = kThreads / wide;
        const int64_t row = int64_t(blockIdx.x) * wide + r;
        float2 s{-INFINITY, 0.0f};
        if (row < a.rows) {
            int t = t0;
            for (; t + 3 * step < a.parts; t += 4 * step) {
                float2 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = a.part[int64_t(t + u * step) * a.rows + row];
                s = join(s, join(join(v[0], v[1]), join(v[2], v[3])));
            }
            for (; t < a.parts; t += step)
                s = join(s, a.part[int64_t(t) * a.rows + row]);
        }
        sums[threadIdx.x] = s;
        for (int n = kThreads / 2; n >= wide; n /= 2) {
            __syncthreads();
            if (int(threadIdx.x) < n)
                sums[threadIdx.x] = join(sums[threadIdx.x], sums[threadIdx.x + n]);
        }
        if (t0 == 0 && row < a.rows)
            a.stats[row] = sums[threadIdx.x];
        return;
    }
    constexpr int kEs = BF16 ? 2 : 4, kGroups = kThreads / G;
    const int64_t first = int64_t(blockIdx.x) - joins, step = int64_t(gridDim.x) - joins;
    const int group = threadIdx.x / G;
    const char *x = static_cast<const char *>(a.x);
    if constexpr (SHARED) {
        extern __shared__ __attribute__((aligned(16))) char row[];
        const int per = (a.topk + kRowEntries - 1) / kRowEntries, bytes = a.dim * kEs;
        for (int64_t b = first; b < int64_t(a.rows) * per; b += step) {
            const int64_t r = b / per;
            const int e0 = int(b - r * per) * kRowEntries, e1 = a.topk - e0 < kRowEntries ? a.topk : e0 + kRowEntries;
            for (int c = threadIdx.x * 16; c < bytes; c += kThreads * 16)
                *reinterpret_cast<u32x4 *>(row + c) = load_chunk<kEs>(x + r * bytes + c, bytes - c);
            __syncthreads();
            for (int e = e0 + group; e < e1; e += kGroups)
                pick<BF16, G>(a, r * a.topk + e, row);
            __syncthreads();
        }
    } else {
        const int64_t entries = int64_t(a.rows) * a.topk;
        for (int64_t n = first * kGroups + group; n < entries; n += step * kGroups)
            pick<BF16, G>(a, n, x + n / a.topk * a.dim * kEs);
    }
}

__device__ __forceinline__ bool counts(int64_t index, int64_t total)
{
    return index >= 0 && index < total;
}

__device__ __forceinline__ float joined_lse(const CombineArgs &a, int64_t j)
{
    float2 s = a.stats[0][j];
    for (int i = 1; i < a.shards; ++i)
        s = join(s, a.stats[i][j]);
    return s.x + logf(s.y);
}

__device__ __forceinline__ float joined_logit(const CombineArgs &a, int64_t n)
{
    float z = a.picked[0][n];
    for (int i = 1; i < a.shards; ++i)
        z += a.picked[i][n];
    return z;
}

__global__ __launch_bounds__(kThreads) void cross_entropy_kernel(CombineArgs a)
{
    const int64_t j = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (j >= a.rows)
        return;
    const float lse = joined_lse(a, j), z = joined_logit(a, j);
    a.lse[j] = lse;
    a.logit[j] = z;
    a.loss[j] = counts(a.index[j], a.total) ? lse - z : 0.0f;
}

// A teacher's logit at its scale; one of -inf leaves its entry out at a scale of 0
// too.
template <bool BF16>
__device__ __forceinline__ float teacher_logit(const CombineArgs &a, int64_t n)
{
    const float t = load<BF16>(a.teacher, n);
    return a.scale == 0.0f && t == -INFINITY ? t : a.scale * t;
}

// One wave per row.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void distill_kernel(CombineArgs a)
{
    const int64_t j = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    const int lane = threadIdx.x % 64;
    if (j >= a.rows)
        return;
    const float lse = joined_lse(a, j);
    float top = -INFINITY, sum = 0.0f;
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t n = j * a.topk + e;
        if (counts(a.index[n], a.total))
            top = fmaxf(top, teacher_logit<BF16>(a, n));
    }
    top = lanes_max<64>(top);
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t n = j * a.topk + e;
        if (counts(a.index[n], a.total))
            sum += exp_below(teacher_logit<BF16>(a, n), top);
    }
    sum = lanes_sum<64>(sum);
    const float log_sum = logf(sum);
    float loss = 0.0f;
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t n = j * a.topk + e;
        const float z = joined_logit(a, n), t = teacher_logit<BF16>(a, n);
        const bool live = counts(a.index[n], a.total) && t != -INFINITY;
        const float p = live ? exp_below(t, top) / sum : 0.0f;
        a.logit[n] = z;
        a.prob[n] = p;
        if (live && p != 0.0f)
            loss += p * ((t - top) - log_sum - z + lse);
    }
    loss = lanes_sum<64>(loss);
    if (lane == 0) {
        a.lse[j] = lse;
        a.loss[j] = loss;
    }
}

// Whether row j has a gradient: a target, and a loss of some weight.  By a whole
// wave.
__device__ __forceinline__ bool has_gradient(const RowsArgs &a, int64_t j)
{
    if (a.grad[j] * a.scale == 0.0f)
        return false;
    bool used = false;
    if (a.prob) {
        for (int e = threadIdx.x % 64; e < a.topk; e += 64)
            used |= a.prob[j * a.topk + e] != 0.0f;
    } else {
        used = counts(a.index[j], a.total);
    }
    return __ballot(used) != 0;
}

// One wave per row at a time, from row `first` in steps of `waves`: 174 MB in
// 56 us, 6.2 TB/s both ways.  Where `of` is given, rows without a gradient become
// zeros: dw is then free of whatever they hold.
template <int ES>
__device__ __forceinline__ void align_rows(const AlignArgs &a, const RowsArgs *of, int64_t first, int64_t waves)
{
    const int lane = threadIdx.x % 64, bytes = a.cols * ES;
    for (int64_t r = first; r < a.rows; r += waves) {
        const char *from = static_cast<const char *>(a.in) + r * bytes;
        char *to = static_cast<char *>(a.out) + r * a.ldo * ES;
        const int have = !of || has_gradient(*of, r) ? bytes : 0;
        for (int c = lane * 16; c < bytes; c += 64 * 16)
            *reinterpret_cast<u32x4 *>(to + c) = load_chunk<ES>(from + c, have - c);
    }
}

__device__ __forceinline__ int round64(int n) { return (n + 63) / 64 * 64; }

// dz = coefficient * exp(z - lse), zero past the piece up to the next multiple
// of 64; the first `copies` workgroups copy x for dw meanwhile.  4096 x 2048 x
// 32000 in bf16: 464-480 us, 1.1 PFLOP/s, of which the statistics' kernel takes
// 415 us.  bf16 keeps dz at 8 bits for the products, whose operand it is on the
// matrix units.  These roundings average out where a gradient sums many of
// them; where it sums few they add to its own (1023 x 1024 x 32000: 0.0019 off
// in all, 0.0017 with dz in fp32; 64 entries a row: 0.0024).
template <typename T>
__global__ __launch_bounds__(T::kThreads) void dz_kernel(DzArgs a, int tiles_i, int tiles_j, int copies)
{
    // a row's factors, its target within the piece (-1: none) and dz there
    struct Row {
        float2 r;
        int target;
        float d;
    };
    __shared__ __attribute__((aligned(1024))) char lds[T::kLdsBytes];
    __shared__ Row rows[T::TJ];
    constexpr int kWaves = T::kThreads / 64;
    if (int(blockIdx.x) < copies) {
        align_rows<T::kEs>(a.x, &a.rows, int64_t(blockIdx.x) * kWaves + threadIdx.x / 64, int64_t(copies) * kWaves);
        return;
    }
    int ti, tj;
    tile_at(blockIdx.x - copies, gridDim.x - copies, tiles_i, tiles_j, ti, tj);
    const int i0 = ti * T::TI, j0 = tj * T::TJ;
    // this thread's row, at a clamped place; its loads fly together with the tile's first
    const int mine = j0 + int(threadIdx.x), in = mine < a.p.nj ? mine : 0;
    float lse = 0.0f, grad = 0.0f, logit = 0.0f;
    int64_t at = -1;
    Row row{float2{0.0f, 0.0f}, -1, 0.0f};
    if (a.rows.prob) {
        row.r = a.rows.row[in];
    } else {
        at = a.rows.index[in];
        lse = a.rows.lse[in];
        grad = a.rows.grad[in];
        logit = a.logit[in];
    }
    typename T::Pipe pipe;
    pipe.start(a.p, i0, j0, 0, (a.p.nk + T::kStep - 1) / T::kStep, lds);
    // a row of no weight is left as one without a target: exp(z - lse) of the
    // zeros that take the place of its logits may overflow
    if (counts(at, a.rows.total) && grad * a.rows.scale != 0.0f) {
        row.r = float2{lse * kLog2e, grad * a.rows.scale};
        if (at >= a.first && at < a.first + a.p.ni) {
            row.target = int(at - a.first);
            row.d = row.r.y * (__builtin_amdgcn_exp2f(__builtin_fmaf(logit, kLog2e, -row.r.x)) - 1.0f);
        }
    }
    if (mine >= a.p.nj)
        row = Row{float2{0.0f, 0.0f}, -1, 0.0f};
    if (int(threadIdx.x) < T::TJ)
        rows[threadIdx.x] = row;
    typename T::Acc acc;
    acc.clear();
    pipe.finish(acc);
    const bool full = i0 + T::TI <= a.p.ni;
    const float c = a.rows.scale * kLog2e;
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
        const Row of = rows[T::lane_j(j)];
        f32x4 d[T::FI];
        // no dz in a row without a gradient, whatever its logits
        if (of.r.y == 0.0f) {
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
                acc.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[i][e] = of.r.y * __builtin_amdgcn_exp2f(__builtin_fmaf(acc.c[i][j][e], c, -of.r.x));
                if (!full && i0 + T::lane_i(i) + e >= a.p.ni)
                    d[i][e] = 0.0f;
            }
        const int64_t to = j0 + T::lane_j(j);
        char *out = static_cast<char *>(a.dz) + (to * a.ldz + i0) * T::kEs;
        T::store_row(out, d, to < a.p.nj ? round64(a.p.ni) - i0 : 0);
        // by the lane that has just written there
        if (of.target >= 0 && T::stores(of.target - i0 - T::wave_i()))
            store<T::kEs == 2>(out, of.target - i0, of.d);
    }
}

// One wave per row.  Equal entries of a row write the same value.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void targets_kernel(TargetArgs a)
{
    struct Entry {
        int i;      // within the piece, or -1
        float p;
    };
    __shared__ Entry of_row[kThreads / 64][RR_MAX_TOPK];
    const int64_t j = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    const int lane = threadIdx.x % 64;
    Entry *entry = of_row[threadIdx.x / 64];
    if (j >= a.rows)
        return;
    bool any = false;
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t i = a.index[j * a.topk + e] - a.first;
        const bool in = i >= 0 && i < a.count;
        entry[e] = Entry{in ? int(i) : -1, a.prob[j * a.topk + e]};
        any |= in;
    }
    if (!__ballot(any))
        return;
    // one wave's LDS operations keep their order; so has the compiler to
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float2 row = a.row[j];
    for (int e = lane; e < a.topk; e += 64) {
        const int i = entry[e].i;
        float p = 0.0f;
#pragma unroll 8
        for (int o = 0; o < a.topk; ++o)
            p += entry[o].i == i ? entry[o].p : 0.0f;
        if (i >= 0) {
            const float z = a.logit[j * a.topk + e];
            store<BF16>(a.dz, j * a.ldz + i,
                        row.y == 0.0f ? 0.0f : row.y * (__builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -row.x)) - p));
        }
    }
}

// What a gradient needs first: the rows' factors, and copies of x and w in
// 16-byte chunks, each by its own workgroups of one launch.
template <int ES>
__global__ __launch_bounds__(kThreads) void prepare_kernel(PrepareArgs a, int rows_blocks, int x_blocks)
{
    constexpr int kWaves = kThreads / 64;
    int b = blockIdx.x;
    const int wave = threadIdx.x / 64;
    if (b < rows_blocks) {
        const int64_t j = int64_t(b) * kWaves + wave;
        if (j >= a.rows.rows)
            return;
        const bool used = has_gradient(a.rows, j);
        if (threadIdx.x % 64 == 0)
            a.rows.row[j] = used ? float2{a.rows.lse[j] * kLog2e, a.rows.grad[j] * a.rows.scale} : float2{0.0f, 0.0f};
        return;
    }
    b -= rows_blocks;
    if (b < x_blocks)
        align_rows<ES>(a.x, &a.rows, int64_t(b) * kWaves + wave, int64_t(x_blocks) * kWaves);
    else
        align_rows<ES>(a.w, nullptr, int64_t(b - x_blocks) * kWaves + wave,
                       int64_t(int(gridDim.x) - rows_blocks - x_blocks) * kWaves);
}

// Tile `block` of dw or dx.
template <typename T>
__device__ __forceinline__ void store_tile(const StoreArgs &a, int block, char *lds)
{
    const int tiles_i = (a.p.ni - 1) / T::TI + 1, tiles_j = (a.p.nj - 1) / T::TJ + 1;
    const int tiles = tiles_i * tiles_j, split = block / tiles;
    int ti, tj;
    tile_at(block - split * tiles, tiles, tiles_i, tiles_j, ti, tj);
    const int i0 = ti * T::TI, j0 = tj * T::TJ;
    const int steps = (a.p.nk + T::kStep - 1) / T::kStep, per = (steps + a.splits - 1) / a.splits;
    const int s0 = split * per < steps ? split * per : steps, s1 = s0 + per < steps ? s0 + per : steps;
    typename T::Pipe pipe;
    pipe.start(a.p, i0, j0, s0, s1, lds);
    typename T::Acc acc;
    acc.clear();
    const auto part = [&](int j, int i) {
        const int row = j0 + T::lane_j(j), col = i0 + T::lane_i(i);
        float *to = a.acc + (int64_t(split) * a.p.nj + row) * a.lda + col;
        return row < a.p.nj && col < a.lda ? reinterpret_cast<f32x4 *>(to) : nullptr;
    };
    if (a.add) {
#pragma unroll
        for (int j = 0; j < T::FJ; ++j)
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
                if (const f32x4 *from = part(j, i))
                    acc.c[i][j] = *from;
    }
    pipe.finish(acc);
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
        if (a.acc) {
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
                if (f32x4 *to = part(j, i))
                    *to = acc.c[i][j];
        } else {
            f32x4 v[T::FI];
#pragma unroll
            for (int i = 0; i < T::FI; ++i)
                v[i] = acc.c[i][j];
            const int64_t row = j0 + T::lane_j(j);
            T::store_row(static_cast<char *>(a.out) + (row * a.ldo + i0) * T::kEs, v, row < a.p.nj ? a.p.ni - i0 : 0);
        }
    }
}

// 4096 x 2048 x 32000 in bf16 in 455-470 us, 1.15 PFLOP/s.
template <typename T>
__global__ __launch_bounds__(T::kThreads) void store_kernel(StoreArgs a)
{
    __shared__ __attribute__((aligned(1024))) char lds[T::kLdsBytes];
    store_tile<T>(a, blockIdx.x, lds);
}

// dx and dw in one launch, where neither fills the compute units for long.
template <typename TX, typename TW>
__global__ __launch_bounds__(TX::kThreads) void stores_kernel(StoresArgs a, int x_blocks)
{
    static_assert(TX::kThreads == TW::kThreads, "");
    __shared__ __attribute__((aligned(1024))) char lds[TX::kLdsBytes > TW::kLdsBytes ? TX::kLdsBytes : TW::kLdsBytes];
    if (int(blockIdx.x) < x_blocks)
        store_tile<TX>(a.x, blockIdx.x, lds);
    else
        store_tile<TW>(a.w, blockIdx.x - x_blocks, lds);
}

// Four columns of a row per PARTS threads, each of which takes its share of the
// sums: with 256 parts of 35 x 192 in 14 us by one thread each, in 4 us by eight.
template <bool BF16, int PARTS>
__device__ __forceinline__ void gather(const GatherArgs &a, int block, int blocks)
{
    constexpr int kWide = kThreads / PARTS;
    __shared__ f32x4 sums[kThreads];
    const int part = threadIdx.x / kWide;
    const int64_t wide = a.lda / 4, n = a.rows * wide, stride = a.rows * a.lda;
    for (int64_t t0 = int64_t(block) * kWide; t0 < n; t0 += int64_t(blocks) * kWide) {
        const int64_t t = t0 + threadIdx.x % kWide, row = t / wide;
        const int col = int(t - row * wide) * 4;
        f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
        if (t < n) {
#pragma unroll 8
            for (int i = part; i < a.splits; i += PARTS)
                s += *reinterpret_cast<const f32x4 *>(a.acc + i * stride + row * a.lda + col);
        }
        if constexpr (PARTS > 1) {
            sums[threadIdx.x] = s;
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int o = 1; o < PARTS; ++o)
                    s += sums[o * kWide + threadIdx.x];
            __syncthreads();
        }
        if (part == 0 && t < n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.dim)
                    store<BF16>(a.out, row * a.dim + col + e, s[e]);
    }
}

// The first x_blocks workgroups join dx, the others dw.
template <bool BF16, int PARTS>
__global__ __launch_bounds__(kThreads) void gather_kernel(GathersArgs a, int x_blocks)
{
    if (int(blockIdx.x) < x_blocks)
        gather<BF16, PARTS>(a.x, blockIdx.x, x_blocks);
    else
        gather<BF16, PARTS>(a.w, blockIdx.x - x_blocks, gridDim.x - x_blocks);
}

unsigned blocks(int64_t n, int64_t per) { return unsigned((n + per - 1) / per); }

}  // namespace

#define RR_LAUNCH(kernel, grid, a)                                   \
    do {                                                             \
        (void)hipGetLastError();                                     \
        kernel<<<(grid), dim3(kThreads), 0, stream>>>(a);            \
        return hipGetLastError();                                    \
    } while (0)

namespace {

enum Shape { kRows16, kRows32, kRows64, kMid, kBig };

int tiles(int n, int per) { return n / per + (n % per != 0); }

struct Form {
    Shape shape;
    int32_t splits;  // parts of k
};

// Tiles and parts of a product by the time that they would take: the busiest of
// 256 compute units has so many tiles, at the rate that a tile's shape reached
// against the largest (4096 x 2048 x 32768 in bf16: 1010 TFLOP/s, 0.75 and 0.64
// of it at 128 x 128 and 128 x 64; 2048 x 1024 x 16384 in fp32: 116 TFLOP/s at
// 128 x 128, 0.93 and 0.83 of it at 128 x 64 and 128 x 32).  A workgroup of the
// smaller ones alone on its unit does not fill it.  In units of a
// multiplication of a compute unit at that rate; a part of k costs the writing
// and reading of its sums, about 5 (bf16) or 0.5 (fp32) for each, and their
// joining a launch, 4 us.  Up to 64 rows the narrowest tile that holds them
// streams the vocabulary past them.
Form form_of(const Product &p, bool may_split, bool tall_b)
{
    static const struct {
        Shape shape;
        int ti, tj;
        double bf16, fp32;
    } all[] = {{kRows16, 128, 16, 0.3, 0.6}, {kRows32, 128, 32, 0.46, 0.83}, {kRows64, 128, 64, 0.64, 0.93},
               {kMid, 128, 128, 0.75, 1.0}, {kBig, 256, 256, 1.0, 0.0}};
    Form best{kMid, 1};
    double least = INFINITY;
    const int steps = tiles(p.nk, p.bf16 ? 64 : 32), most = may_split ? (steps / 4 < 256 ? steps / 4 : 256) : 1;
    for (const auto &f : all) {
        const double rate = p.bf16 ? f.bf16 : f.fp32;
        if (rate == 0.0 || (tall_b && f.tj < (p.bf16 ? 128 : 64)))
            continue;
        // rows that fit a narrow tile
        if (!tall_b && p.nj <= 64 && (f.tj < p.nj || f.tj > 64 || f.tj >= 2 * p.nj + 16))
            continue;
        const double n = double(tiles(p.ni, f.ti)) * tiles(p.nj, f.tj);
        for (int s = 1; s <= (most < 1 ? 1 : most); ++s) {
            const double busy = ceil(n * s / 256);
            const double time = (busy == 1 && f.shape != kBig ? 1.6 : busy) * f.ti * f.tj / rate * (double(p.nk) / s + 256) +
                                (s > 1 ? (p.bf16 ? 5.0 : 0.5) * s * p.ni * p.nj + (p.bf16 ? 1e7 : 1e6) : 0.0);
            if (time < least) {
                least = time;
                best = Form{f.shape, s};
            }
        }
    }
    return best;
}

// Both operands in 16-byte chunks.
bool direct(const Product &p)
{
    const int es = p.bf16 ? 2 : 4;
    return in_chunks(p.a, p.lda, es) && in_chunks(p.b, p.ldb, es) && p.nk * int64_t(es) % 16 == 0;
}

template <bool BF16, int TJ, int STAGES, bool DIRECT, bool TA, bool TB>
using Rows = Tile<BF16, 128, TJ, 4, 1, DIRECT ? STAGES : 2, DIRECT, TA, TB>;
template <bool BF16, bool DIRECT, bool TA, bool TB> using Mid = Tile<BF16, 128, 128, 2, 2, 2, DIRECT, TA, TB>;
template <bool BF16, bool DIRECT, bool TA, bool TB> using Big = Tile<BF16, 256, 256, 2, 4, 2, DIRECT, TA, TB>;

// f(tile type).  For few rows a third step in LDS covers the latency of the
// streamed weights (20 x 4096 x 32000 in bf16: 47 us against 49 us); in fp32,
// which the matrix units bound, a third workgroup on a compute unit is worth
// more (777 x 1000 x 5004 training: 360 us against 390 us).
template <bool BF16, bool DIRECT, bool TA, bool TB, typename F>
hipError_t with_shape(Shape s, F f)
{
    if constexpr (!TB) {
        if (s == kRows16)
            return f(Rows<BF16, 16, 3, DIRECT, TA, TB>{});
        if (s == kRows32)
            return f(Rows<BF16, 32, BF16 ? 3 : 2, DIRECT, TA, TB>{});
    }
    if constexpr (!(TB && BF16))
        if (s == kRows64)
            return f(Rows<BF16, 64, BF16 ? 3 : 2, DIRECT, TA, TB>{});
    if constexpr (BF16)
        if (s == kBig)
            return f(Big<BF16, DIRECT, TA, TB>{});
    return f(Mid<BF16, DIRECT, TA, TB>{});
}

// The logits' tile; operands at any element alignment, or (ALIGNED) in 16-byte chunks.
template <bool ALIGNED, typename F>
hipError_t with_logits_tile(const Product &p, F f)
{
    const Shape s = form_of(p, false, false).shape;
    if (ALIGNED || direct(p))
        return p.bf16 ? with_shape<true, true, false, false>(s, f) : with_shape<false, true, false, false>(s, f);
    if constexpr (!ALIGNED)
        return p.bf16 ? with_shape<true, false, false, false>(s, f) : with_shape<false, false, false, false>(s, f);
    return hipErrorInvalidValue;
}

}  // namespace

int64_t stats_parts(const Product &p)
{
    switch (form_of(p, false, false).shape) {
    case kRows16: case kRows32: case kRows64: return int64_t(tiles(p.ni, 128)) * 4;
    case kMid: return int64_t(tiles(p.ni, 128)) * 2;
    default: return int64_t(tiles(p.ni, 256)) * 2;
    }
}

hipError_t launch_stats(const Op &op, hipStream_t stream)
{
    const StatsArgs a = op.get<StatsArgs>();
    (void)hipGetLastError();
    return with_logits_tile<false>(a.p, [&](auto t) {
        using T = decltype(t);
        const int ti = tiles(a.p.ni, T::TI), tj = tiles(a.p.nj, T::TJ);
        stats_kernel<T><<<dim3(unsigned(ti) * unsigned(tj)), dim3(T::kThreads), 0, stream>>>(a, ti, tj);
        return hipGetLastError();
    });
}

hipError_t launch_stats_done(const Op &op, hipStream_t stream)
{
    const StatsDoneArgs a = op.get<StatsDoneArgs>();
    // rows per workgroup: few, so that there are workgroups for all compute units
    int wide = 1;
    while (wide < 64 && a.rows / wide > 512)
        wide *= 2;
    // 16 lanes an entry once that fills the compute units; x shared where
    // workgroups of a row fill them too and it is long (bf16 with its joins:
    // 3596 x 2112 x 1292 with 64 entries 100 us against 115 us for scoring, but
    // 310 x 3328 x 1228 with 100 entries 52 us against 41 us and 7722 x 128 x
    // 4690 78 us against 75 us)
    const int64_t all = int64_t(a.rows) * a.topk, bytes = int64_t(a.dim) * (a.bf16 ? 2 : 4);
    const int64_t of_rows = int64_t(a.rows) * ((a.topk + kRowEntries - 1) / kRowEntries);
    const bool shared = a.topk >= 8 && of_rows >= 2048 && bytes >= 1024 && bytes <= 32768;
    const int lanes = all < 8192 ? 64 : 16;
    const unsigned joins = blocks(a.rows, wide), entries = shared ? blocks(of_rows, 1) : blocks(all, kThreads / lanes),
                   grid = joins + (entries < 65536u ? entries : 65536u);
    (void)hipGetLastError();
    const auto go = [&](auto bf16) {
        if (shared)
            stats_done_kernel<decltype(bf16)::value, 16, true>
                <<<dim3(grid), dim3(kThreads), size_t(bytes + 15) / 16 * 16, stream>>>(a, joins, wide);
        else if (lanes == 64)
            stats_done_kernel<decltype(bf16)::value, 64, false><<<dim3(grid), dim3(kThreads), 0, stream>>>(a, joins, wide);
        else
            stats_done_kernel<decltype(bf16)::value, 16, false><<<dim3(grid), dim3(kThreads), 0, stream>>>(a, joins, wide);
        return hipGetLastError();
    };
    return a.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

hipError_t launch_cross_entropy(const Op &op, hipStream_t stream)
{
    const CombineArgs a = op.get<CombineArgs>();
    RR_LAUNCH(cross_entropy_kernel, dim3(blocks(a.rows, kThreads)), a);
}

hipError_t launch_distill(const Op &op, hipStream_t stream)
{
    const CombineArgs a = op.get<CombineArgs>();
    const dim3 grid(blocks(a.rows, kThreads / 64));
    if (a.bf16)
        RR_LAUNCH(distill_kernel<true>, grid, a);
    RR_LAUNCH(distill_kernel<false>, grid, a);
}

hipError_t launch_dz(const Op &op, hipStream_t stream)
{
    const DzArgs a = op.get<DzArgs>();
    (void)hipGetLastError();
    return with_logits_tile<true>(a.p, [&](auto t) {
        using T = decltype(t);
        const int ti = tiles(a.p.ni, T::TI), tj = tiles(a.p.nj, T::TJ);
        // x's copy by the first workgroups, a multiple of the eight dies
        const unsigned waves = T::kThreads / 64, rows = a.x.in ? blocks(a.x.rows, 8 * waves) * 8 : 0, copies = rows < 256u ? rows : 256u;
        dz_kernel<T><<<dim3(unsigned(ti) * unsigned(tj) + copies), dim3(T::kThreads), 0, stream>>>(a, ti, tj, int(copies));
        return hipGetLastError();
    });
}

hipError_t launch_targets(const Op &op, hipStream_t stream)
{
    const TargetArgs a = op.get<TargetArgs>();
    const dim3 grid(blocks(a.rows, kThreads / 64));
    if (a.bf16)
        RR_LAUNCH(targets_kernel<true>, grid, a);
    RR_LAUNCH(targets_kernel<false>, grid, a);
}

hipError_t launch_prepare(const Op &op, hipStream_t stream)
{
    const PrepareArgs a = op.get<PrepareArgs>();
    const auto some = [](const AlignArgs &m) {
        const unsigned n = m.in ? blocks(m.rows, kThreads / 64) : 0;
        return n < 8192u ? n : 8192u;
    };
    const unsigned r = a.factors ? blocks(a.rows.rows, kThreads / 64) : 0, x = some(a.x), w = some(a.w);
    (void)hipGetLastError();
    if (a.bf16)
        prepare_kernel<2><<<dim3(r + x + w), dim3(kThreads), 0, stream>>>(a, r, x);
    else
        prepare_kernel<4><<<dim3(r + x + w), dim3(kThreads), 0, stream>>>(a, r, x);
    return hipGetLastError();
}

int32_t product_splits(const Product &p, bool tall_b) { return form_of(p, true, tall_b).splits; }

namespace {

template <typename T>
unsigned store_blocks(const StoreArgs &a)
{
    return unsigned(tiles(a.p.ni, T::TI)) * unsigned(tiles(a.p.nj, T::TJ)) * unsigned(a.splits);
}

template <bool BF16>
hipError_t stores(const StoresArgs &a, hipStream_t stream)
{
    const Shape sx = form_of(a.x.p, true, false).shape, sw = form_of(a.w.p, true, true).shape;
    if (sx == kBig || sw == kBig) {
        const auto go = [&](const StoreArgs &s) {
            return [&s, stream](auto t) {
                using T = decltype(t);
                store_kernel<T><<<dim3(store_blocks<T>(s)), dim3(T::kThreads), 0, stream>>>(s);
                return hipGetLastError();
            };
        };
        const hipError_t e = with_shape<BF16, true, true, false>(sx, go(a.x));
        return e == hipSuccess ? with_shape<BF16, true, true, true>(sw, go(a.w)) : e;
    }
    return with_shape<BF16, true, true, false>(sx, [&](auto tx) {
        return with_shape<BF16, true, true, true>(sw, [&](auto tw) {
            using TX = decltype(tx);
            using TW = decltype(tw);
            if constexpr (TX::kThreads == TW::kThreads && TX::kThreads == 256) {
                const unsigned x = store_blocks<TX>(a.x);
                stores_kernel<TX, TW><<<dim3(x + store_blocks<TW>(a.w)), dim3(TX::kThreads), 0, stream>>>(a, x);
                return hipGetLastError();
            } else {
                return hipErrorInvalidValue;
            }
        });
    });
}

}  // namespace

hipError_t launch_stores(const Op &op, hipStream_t stream)
{
    const StoresArgs a = op.get<StoresArgs>();
    (void)hipGetLastError();
    return a.x.p.bf16 ? stores<true>(a, stream) : stores<false>(a, stream);
}

hipError_t launch_gather(const Op &op, hipStream_t stream)
{
    const GathersArgs a = op.get<GathersArgs>();
    const bool many = a.x.splits >= 16 || a.w.splits >= 16;
    const auto some = [&](const GatherArgs &g) {
        const unsigned n = g.out ? blocks(g.rows * (g.lda / 4), many ? kThreads / 8 : kThreads) : 0;
        return n < 4096u ? n : 4096u;
    };
    const unsigned x = some(a.x), w = some(a.w);
    (void)hipGetLastError();
    const auto go = [&](auto bf16) {
        if (many)
            gather_kernel<decltype(bf16)::value, 8><<<dim3(x + w), dim3(kThreads), 0, stream>>>(a, x);
        else
            gather_kernel<decltype(bf16)::value, 1><<<dim3(x + w), dim3(kThreads), 0, stream>>>(a, x);
        return hipGetLastError();
    };
    return a.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace rr
