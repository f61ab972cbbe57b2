// rr_vocab.hip -- gfx950 kernels of the sharded vocabulary head: the logits'
// softmax statistics and their gradient, without keeping the logits.
//
// Simplest form: every product is computed in 64 x 64 tiles staged through
// LDS, each thread accumulating 4 x 4 results in fp32.
#include "rr_loss.h"

namespace rr {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

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

// c[y][x] = sum over k of A[i0 + 4 tx + x][k] B[j0 + 4 ty + y][k].
template <bool BF16>
__device__ void product_tile(const Product &p, int64_t i0, int64_t j0, float (&c)[4][4])
{
    __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int y = 0; y < 4; ++y)
        for (int x = 0; x < 4; ++x)
            c[y][x] = 0.0f;
    for (int k0 = 0; k0 < p.nk; k0 += kStep) {
        for (int t = threadIdx.x; t < kTile * kStep; t += kThreads) {
            const int k = t % kStep, r = t / kStep;
            const bool in = k0 + k < p.nk;
            sa[k][r] = in && i0 + r < p.ni ? load<BF16>(p.a, (i0 + r) * p.lda + k0 + k) : 0.0f;
            sb[k][r] = in && j0 + r < p.nj ? load<BF16>(p.b, (j0 + r) * p.ldb + k0 + k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int y = 0; y < 4; ++y)
                for (int x = 0; x < 4; ++x)
                    c[y][x] = __builtin_fmaf(sa[k][4 * tx + x], sb[k][4 * ty + y], c[y][x]);
        __syncthreads();
    }
}

// exp(x - top) where top may be infinite: -inf - -inf counts as nothing.
__device__ __forceinline__ float exp_below(float x, float top)
{
    return x == -INFINITY ? 0.0f : expf(x - top);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void stats_kernel(StatsArgs a)
{
    const int64_t i0 = int64_t(blockIdx.x) * kTile, j0 = int64_t(blockIdx.y) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4];
    product_tile<BF16>(a.p, i0, j0, c);
    for (int y = 0; y < 4; ++y) {
        const int64_t j = j0 + 4 * ty + y;
        float top = -INFINITY, sum = 0.0f;
        bool nan = false;
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + 4 * tx + x;
            c[y][x] *= a.scale;
            if (i < a.p.ni) {
                top = fmaxf(top, c[y][x]);
                nan |= c[y][x] != c[y][x];
            }
        }
        for (int d = 1; d < 16; d *= 2)
            top = fmaxf(top, __shfl_xor(top, d));
        for (int x = 0; x < 4; ++x)
            if (i0 + 4 * tx + x < a.p.ni)
                sum += exp_below(c[y][x], top);
        if (nan)
            sum = NAN;
        for (int d = 1; d < 16; d *= 2)
            sum += __shfl_xor(sum, d);
        if (j >= a.p.nj)
            continue;
        if (tx == 0)
            a.part[int64_t(blockIdx.x) * a.p.nj + j] = float2{top, sum};
        for (int e = 0; e < a.topk; ++e) {
            const int64_t i = a.index[j * a.topk + e] - a.first;
            for (int x = 0; x < 4; ++x)
                if (i == i0 + 4 * tx + x && i < a.p.ni)
                    a.picked[j * a.topk + e] = c[y][x];
        }
    }
}

// (top, sum) of the union of two sets of logits.
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float top = fmaxf(a.x, b.x);
    const float fa = a.x == top ? 1.0f : exp_below(a.x, top), fb = b.x == top ? 1.0f : exp_below(b.x, top);
    return float2{top, a.y * fa + b.y * fb};
}

__global__ __launch_bounds__(kThreads) void stats_done_kernel(StatsDoneArgs a)
{
    const int64_t j = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (j >= a.rows)
        return;
    float2 s{-INFINITY, 0.0f};
    for (int t = 0; t < a.tiles; ++t)
        s = join(s, a.part[int64_t(t) * a.rows + j]);
    a.stats[j] = s;
    for (int e = 0; e < a.topk; ++e) {
        const int64_t i = a.index[j * a.topk + e] - a.first;
        if (i < 0 || i >= a.vocab)
            a.picked[j * a.topk + e] = 0.0f;
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

__device__ __forceinline__ float wave_max(float v)
{
    for (int d = 1; d < 64; d *= 2)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
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
            top = fmaxf(top, a.scale * load<BF16>(a.teacher, n));
    }
    top = wave_max(top);
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t n = j * a.topk + e;
        if (counts(a.index[n], a.total))
            sum += exp_below(a.scale * load<BF16>(a.teacher, n), top);
    }
    sum = wave_sum(sum);
    const float log_sum = logf(sum);
    float loss = 0.0f;
    for (int e = lane; e < a.topk; e += 64) {
        const int64_t n = j * a.topk + e;
        const float z = joined_logit(a, n), t = a.scale * load<BF16>(a.teacher, n);
        const bool live = counts(a.index[n], a.total) && t != -INFINITY;
        const float p = live ? exp_below(t, top) / sum : 0.0f;
        a.logit[n] = z;
        a.prob[n] = p;
        if (live && p != 0.0f)
            loss += p * ((t - top) - log_sum - z + lse);
    }
    loss = wave_sum(loss);
    if (lane == 0) {
        a.lse[j] = lse;
        a.loss[j] = loss;
    }
}

__global__ __launch_bounds__(kThreads) void rows_kernel(RowsArgs a)
{
    const int64_t j = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (j >= a.rows)
        return;
    bool used = false;
    for (int e = 0; e < a.topk; ++e)
        used |= a.prob ? a.prob[j * a.topk + e] != 0.0f : counts(a.index[j * a.topk + e], a.total);
    a.row[j] = used ? float2{a.lse[j], a.grad[j] * a.scale} : float2{0.0f, 0.0f};
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void dz_kernel(DzArgs a)
{
    const int64_t i0 = int64_t(blockIdx.x) * kTile, j0 = int64_t(blockIdx.y) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4];
    product_tile<BF16>(a.p, i0, j0, c);
    for (int y = 0; y < 4; ++y) {
        const int64_t j = j0 + 4 * ty + y;
        if (j >= a.p.nj)
            continue;
        const float2 row = a.row[j];
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + 4 * tx + x;
            if (i >= a.p.ni)
                continue;
            const float d = row.y == 0.0f ? 0.0f : row.y * expf(a.scale * c[y][x] - row.x);
            store<BF16>(a.dz, j * a.ldz + i, d);
            store<BF16>(a.dzt, i * a.ldt + j, d);
        }
    }
}

// One thread per entry.  Equal entries of a row write the same value.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void targets_kernel(TargetArgs a)
{
    const int64_t n = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (n >= int64_t(a.rows) * a.topk)
        return;
    const int64_t at = a.index[n], i = at - a.first, j = n / a.topk;
    if (i < 0 || i >= a.count)
        return;
    const float2 row = a.row[j];
    float p = 1.0f;
    if (a.prob) {
        p = 0.0f;
        for (int e = 0; e < a.topk; ++e)
            if (a.index[j * a.topk + e] == at)
                p += a.prob[j * a.topk + e];
    }
    const float d = row.y == 0.0f ? 0.0f : row.y * (expf(a.logit[n] - row.x) - p);
    store<BF16>(a.dz, j * a.ldz + i, d);
    store<BF16>(a.dzt, i * a.ldt + j, d);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void transpose_kernel(TransposeArgs a)
{
    __shared__ T tile[64][65];
    const int64_t r0 = int64_t(blockIdx.x) * 64, c0 = int64_t(blockIdx.y) * 64;
    for (int t = threadIdx.x; t < 64 * 64; t += kThreads) {
        const int r = t / 64, c = t % 64;
        tile[r][c] = r0 + r < a.rows && c0 + c < a.cols ? static_cast<const T *>(a.in)[(r0 + r) * a.ldi + c0 + c] : T(0);
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 64 * 64; t += kThreads) {
        const int c = t / 64, r = t % 64;
        if (c0 + c < a.cols)
            static_cast<T *>(a.out)[(c0 + c) * a.ldo + r0 + r] = tile[r][c];
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void store_kernel(StoreArgs a)
{
    const int64_t i0 = int64_t(blockIdx.x) * kTile, j0 = int64_t(blockIdx.y) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4];
    product_tile<BF16>(a.p, i0, j0, c);
    for (int y = 0; y < 4; ++y)
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + 4 * tx + x, j = j0 + 4 * ty + y;
            if (i >= a.p.ni || j >= a.p.nj)
                continue;
            if (a.acc) {
                float *s = a.acc + j * a.p.ni + i;
                *s = a.add ? *s + c[y][x] : c[y][x];
            } else {
                store<BF16>(a.out, j * a.ldo + i, c[y][x]);
            }
        }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void gather_kernel(GatherArgs a)
{
    for (int64_t n = int64_t(blockIdx.x) * kThreads + threadIdx.x; n < a.n; n += int64_t(gridDim.x) * kThreads) {
        float s = 0.0f;
        for (int i = 0; i < a.splits; ++i)
            s += a.acc[i * a.n + n];
        store<BF16>(a.out, n, s);
    }
}

unsigned blocks(int64_t n, int64_t per) { return unsigned((n + per - 1) / per); }

}  // namespace

#define RR_LAUNCH(kernel, grid, a)                                   \
    do {                                                             \
        (void)hipGetLastError();                                     \
        kernel<<<(grid), dim3(kThreads), 0, stream>>>(a);            \
        return hipGetLastError();                                    \
    } while (0)

int32_t stats_tile(const Product &) { return kTile; }

hipError_t launch_stats(const Op &op, hipStream_t stream)
{
    const StatsArgs a = op.get<StatsArgs>();
    const dim3 grid(blocks(a.p.ni, kTile), blocks(a.p.nj, kTile));
    if (a.p.bf16)
        RR_LAUNCH(stats_kernel<true>, grid, a);
    RR_LAUNCH(stats_kernel<false>, grid, a);
}

hipError_t launch_stats_done(const Op &op, hipStream_t stream)
{
    const StatsDoneArgs a = op.get<StatsDoneArgs>();
    RR_LAUNCH(stats_done_kernel, dim3(blocks(a.rows, kThreads)), a);
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

hipError_t launch_rows(const Op &op, hipStream_t stream)
{
    const RowsArgs a = op.get<RowsArgs>();
    RR_LAUNCH(rows_kernel, dim3(blocks(a.rows, kThreads)), a);
}

hipError_t launch_dz(const Op &op, hipStream_t stream)
{
    const DzArgs a = op.get<DzArgs>();
    const dim3 grid(blocks(a.p.ni, kTile), blocks(a.p.nj, kTile));
    if (a.p.bf16)
        RR_LAUNCH(dz_kernel<true>, grid, a);
    RR_LAUNCH(dz_kernel<false>, grid, a);
}

hipError_t launch_targets(const Op &op, hipStream_t stream)
{
    const TargetArgs a = op.get<TargetArgs>();
    const dim3 grid(blocks(int64_t(a.rows) * a.topk, kThreads));
    if (a.bf16)
        RR_LAUNCH(targets_kernel<true>, grid, a);
    RR_LAUNCH(targets_kernel<false>, grid, a);
}

hipError_t launch_transpose(const Op &op, hipStream_t stream)
{
    const TransposeArgs a = op.get<TransposeArgs>();
    const dim3 grid(blocks(a.rows, 64), blocks(a.cols, 64));
    if (a.bf16)
        RR_LAUNCH(transpose_kernel<unsigned short>, grid, a);
    RR_LAUNCH(transpose_kernel<unsigned>, grid, a);
}

hipError_t launch_store(const Op &op, hipStream_t stream)
{
    const StoreArgs a = op.get<StoreArgs>();
    const dim3 grid(blocks(a.p.ni, kTile), blocks(a.p.nj, kTile));
    if (a.p.bf16)
        RR_LAUNCH(store_kernel<true>, grid, a);
    RR_LAUNCH(store_kernel<false>, grid, a);
}

hipError_t launch_gather(const Op &op, hipStream_t stream)
{
    const GatherArgs a = op.get<GatherArgs>();
    const dim3 grid(blocks(a.n, kThreads) < 4096u ? blocks(a.n, kThreads) : 4096u);
    if (a.bf16)
        RR_LAUNCH(gather_kernel<true>, grid, a);
    RR_LAUNCH(gather_kernel<false>, grid, a);
}

}  // namespace rr
