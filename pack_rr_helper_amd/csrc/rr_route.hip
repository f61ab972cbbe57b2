// rr_route.hip -- gfx950 kernels of the router: the topk choice, the weights,
// the experts' counts and probability sums, the balance loss and its gradient.
//
// Simplest form: one wave per row, the row's experts spread over its lanes.
#include "rr_loss.h"

namespace rr {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPerLane = RR_MAX_EXPERTS / 64;

template <bool BF16>
__device__ __forceinline__ float load(const void *p, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float((unsigned)static_cast<const unsigned short *>(p)[i] << 16);
    else
        return static_cast<const float *>(p)[i];
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

// Unsigned keys in the order of the floats, NaN on top.
__device__ __forceinline__ unsigned order_key(float v)
{
    if (v != v)
        return 0xffffffffu;
    const unsigned u = __float_as_uint(v + 0.0f);  // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float exp_below(float x, float top)
{
    return x == -INFINITY ? 0.0f : expf(x - top);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a)
{
    __shared__ int count[RR_MAX_EXPERTS + 1];
    __shared__ float sums[kWaves][RR_MAX_EXPERTS];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    for (int i = threadIdx.x; i <= a.experts; i += kThreads)
        count[i] = 0;
    __syncthreads();
    float sum[kPerLane];
    for (int s = 0; s < kPerLane; ++s)
        sum[s] = 0.0f;
    for (int64_t r = int64_t(blockIdx.x) * kWaves + wave; r < a.rows; r += int64_t(gridDim.x) * kWaves) {
        if (a.keep && !a.keep[r]) {
            if (lane < a.topk) {
                a.choice[r * a.topk + lane] = -1;
                a.weight[r * a.topk + lane] = 0.0f;
            }
            if (lane == 0)
                a.lse[r] = 0.0f;
            continue;
        }
        float z[kPerLane], top = -INFINITY, total = 0.0f;
        unsigned long long key[kPerLane];
        for (int s = 0; s < kPerLane; ++s) {
            const int e = s * 64 + lane;
            z[s] = -INFINITY;
            key[s] = 0;
            if (e < a.experts) {
                z[s] = load<BF16>(a.logits, r * a.experts + e);
                key[s] = (unsigned long long)order_key(z[s]) << 32 | unsigned(~e);
                top = fmaxf(top, z[s]);
            }
        }
        top = wave_max(top);
        for (int s = 0; s < kPerLane; ++s)
            total += exp_below(z[s], top);
        total = wave_sum(total);
        const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
        for (int s = 0; s < kPerLane; ++s)
            sum[s] += exp_below(z[s], top) * inv;
        // the topk largest keys, one at a time
        float w = 0.0f;
        int mine = -1;
        for (int k = 0; k < a.topk; ++k) {
            unsigned long long best = 0;
            for (int s = 0; s < kPerLane; ++s)
                best = key[s] > best ? key[s] : best;
            for (int d = 1; d < 64; d *= 2) {
                const unsigned long long o = __shfl_xor(best, d);
                best = o > best ? o : best;
            }
            const int e = int(~unsigned(best));
            for (int s = 0; s < kPerLane; ++s)
                if (s * 64 + lane == e)
                    key[s] = 0;
            float ez = 0.0f;
            for (int s = 0; s < kPerLane; ++s)
                ez = s == e / 64 ? z[s] : ez;
            ez = __shfl(ez, e % 64);
            if (lane == k) {
                mine = e;
                w = exp_below(ez, top);
            }
        }
        if (a.renormalize) {
            const float chosen = wave_sum(w);
            w = chosen == 0.0f ? 0.0f : w / chosen;
        } else {
            w *= inv;
        }
        if (lane < a.topk) {
            a.choice[r * a.topk + lane] = mine;
            a.weight[r * a.topk + lane] = w;
            atomicAdd(&count[mine], 1);
        }
        if (lane == 0) {
            a.lse[r] = top + logf(total);
            atomicAdd(&count[a.experts], 1);
        }
    }
    for (int s = 0; s < kPerLane; ++s)
        sums[wave][s * 64 + lane] = sum[s];
    __syncthreads();
    for (int i = threadIdx.x; i < a.experts; i += kThreads) {
        float t = 0.0f;
        for (int w = 0; w < kWaves; ++w)
            t += sums[w][i];
        a.prob_sum[int64_t(blockIdx.x) * a.experts + i] = t;
    }
    for (int i = threadIdx.x; i <= a.experts; i += kThreads)
        a.counts[int64_t(blockIdx.x) * (a.experts + 1) + i] = count[i];
}

__global__ __launch_bounds__(kThreads) void route_sum_kernel(RouteSumArgs a)
{
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i > a.experts)
        return;
    int n = 0;
    float s = 0.0f;
    for (int b = 0; b < a.blocks; ++b) {
        n += a.part_counts[int64_t(b) * (a.experts + 1) + i];
        if (i < a.experts)
            s += a.part_sum[int64_t(b) * a.experts + i];
    }
    a.counts[i] = n;
    if (i < a.experts)
        a.prob_sum[i] = s;
}

__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a)
{
    __shared__ float sums[kWaves];
    int64_t n = 0;
    for (int r = 0; r < a.ranks; ++r)
        n += a.counts[r][a.experts];
    const float tokens = float(n), inv = n > 0 ? 1.0f / tokens : 0.0f;
    float s = 0.0f;
    for (int i = threadIdx.x; i < a.experts; i += kThreads) {
        int64_t c = 0;
        float p = 0.0f;
        for (int r = 0; r < a.ranks; ++r) {
            c += a.counts[r][i];
            p += a.prob_sum[r][i];
        }
        const float f = float(c) * inv / float(a.topk);
        a.slope[i] = float(a.experts) * f * inv;
        s += f * (p * inv);
    }
    s = wave_sum(s);
    if (threadIdx.x % 64 == 0)
        sums[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int w = 0; w < kWaves; ++w)
            t += sums[w];
        a.loss[0] = n > 0 ? float(a.experts) * t : 0.0f;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a)
{
    const int lane = threadIdx.x % 64;
    const int64_t r = int64_t(blockIdx.x) * kWaves + threadIdx.x / 64;
    if (r >= a.rows)
        return;
    const bool kept = !a.keep || a.keep[r];
    const float lse = a.lse[r], gl = a.grad_loss[0];
    float p[kPerLane], g[kPerLane], dot = 0.0f, chosen = 0.0f;
    if (kept && a.renormalize) {
        if (lane < a.topk)
            chosen = a.weight[r * a.topk + lane] * a.grad_weight[r * a.topk + lane];
        chosen = wave_sum(chosen);
    }
    for (int s = 0; s < kPerLane; ++s) {
        const int e = s * 64 + lane;
        p[s] = g[s] = 0.0f;
        if (kept && e < a.experts) {
            p[s] = exp_below(load<BF16>(a.logits, r * a.experts + e), lse);
            g[s] = gl * a.slope[e];
            if (!a.renormalize)
                for (int k = 0; k < a.topk; ++k)
                    if (a.choice[r * a.topk + k] == e)
                        g[s] += a.grad_weight[r * a.topk + k];
            dot += p[s] * g[s];
        }
    }
    dot = wave_sum(dot);
    for (int s = 0; s < kPerLane; ++s) {
        const int e = s * 64 + lane;
        if (e >= a.experts)
            continue;
        float d = p[s] * (g[s] - dot);
        if (kept && a.renormalize)
            for (int k = 0; k < a.topk; ++k)
                if (a.choice[r * a.topk + k] == e)
                    d += a.weight[r * a.topk + k] * (a.grad_weight[r * a.topk + k] - chosen);
        if constexpr (BF16)
            static_cast<__bf16 *>(a.dlogits)[r * a.experts + e] = (__bf16)d;
        else
            static_cast<float *>(a.dlogits)[r * a.experts + e] = d;
    }
}

}  // namespace

#define RR_LAUNCH(kernel, grid, a)                                   \
    do {                                                             \
        (void)hipGetLastError();                                     \
        kernel<<<(grid), dim3(kThreads), 0, stream>>>(a);            \
        return hipGetLastError();                                    \
    } while (0)

int32_t route_blocks(int64_t rows, int32_t)
{
    const int64_t n = (rows + kWaves - 1) / kWaves;
    return rows <= 16 ? 1 : int32_t(n < 1024 ? n : 1024);
}

hipError_t launch_route(const Op &op, hipStream_t stream)
{
    const RouteArgs a = op.get<RouteArgs>();
    if (a.bf16)
        RR_LAUNCH(route_kernel<true>, dim3(a.blocks), a);
    RR_LAUNCH(route_kernel<false>, dim3(a.blocks), a);
}

hipError_t launch_route_sum(const Op &op, hipStream_t stream)
{
    const RouteSumArgs a = op.get<RouteSumArgs>();
    RR_LAUNCH(route_sum_kernel, dim3(a.experts / kThreads + 1), a);
}

hipError_t launch_balance(const Op &op, hipStream_t stream)
{
    const BalanceArgs a = op.get<BalanceArgs>();
    RR_LAUNCH(balance_kernel, dim3(1), a);
}

hipError_t launch_route_grad(const Op &op, hipStream_t stream)
{
    const RouteGradArgs a = op.get<RouteGradArgs>();
    const dim3 grid(unsigned((a.rows + kWaves - 1) / kWaves));
    if (a.bf16)
        RR_LAUNCH(route_grad_kernel<true>, grid, a);
    RR_LAUNCH(route_grad_kernel<false>, grid, a);
}

}  // namespace rr
