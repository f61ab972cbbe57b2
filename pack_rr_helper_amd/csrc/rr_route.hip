// rr_route.hip -- gfx950 kernels of the router: the topk choice, the weights,
// the experts' counts and probability sums, the balance loss and its gradient.
//
// A row is held by G lanes in registers, PER experts each, so that one wave
// works on 64 / G rows and up to 256 experts every exchange stays within a DPP
// row.  Up to 8 choices, each lane sorts its own experts' keys and sorted lists
// are merged across the lanes; more choices are taken one largest key at a
// time.  rr_route is bound by these vector instructions, rr_route_grad by its
// bytes.  Loads are unconditional, at clamped places: a load under a condition
// is waited for where the condition ends.
#include "rr_loss.h"
#include "rr_rows.h"

namespace rr {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kRouteThreads = 512, kRouteWaves = kRouteThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// Unsigned keys above 0 in the order of the floats: a positive number's bits
// above all others, a negative one's negated, which makes both zeros equal.
__device__ __forceinline__ unsigned order_key(float v)
{
    const unsigned u = __float_as_uint(v), m = unsigned(int(u) >> 31);
    return (u ^ (m | 0x80000000u)) - m;
}
// of every NaN
constexpr unsigned kNanKey = 0xffff0000u;

__device__ __forceinline__ float key_value(unsigned key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : 0u - key);
}

// A logit and its expert as one number, larger for the larger logit and for
// the lower index among equals.  bf16 leaves 16 bits of a word for the index;
// fp32 takes a double in [1, 2), whose order is that of its bits and whose
// minimum and maximum are single instructions.
template <bool BF16>
struct Key;

template <>
struct Key<true> {
    typedef unsigned T;
    __device__ static T make(unsigned k, int e) { return (k & 0xffff0000u) | unsigned(0xffff - e); }
    __device__ static int expert(T k) { return 0xffff - int(k & 0xffffu); }
    __device__ static float value(T k) { return key_value(k & 0xffff0000u); }
    __device__ static T larger(T a, T b) { return a > b ? a : b; }
    __device__ static T smaller(T a, T b) { return a < b ? a : b; }
};

template <>
struct Key<false> {
    typedef double T;
    static_assert(RR_MAX_EXPERTS <= 1024, "the index has ten bits");
    __device__ static T make(unsigned k, int e)
    {
        return __builtin_bit_cast(double, (unsigned long long)(0x3ff00000u | k >> 22) << 32 | (k << 10 | unsigned(1023 - e)));
    }
    __device__ static unsigned long long bits(T k) { return __builtin_bit_cast(unsigned long long, k); }
    __device__ static int expert(T k) { return 1023 - int(bits(k) & 1023u); }
    __device__ static float value(T k) { return key_value(unsigned(bits(k) >> 10)); }
    __device__ static T larger(T a, T b) { return fmax(a, b); }
    __device__ static T smaller(T a, T b) { return fmin(a, b); }
};

// exp(x - base).  The product's rounding is |x - base| 2^-24 of the result.
__device__ __forceinline__ float exp_from(float x, float base)
{
    return __builtin_amdgcn_exp2f((x - base) * kLog2e);
}

// -inf - -inf is to count as nothing.
__device__ __forceinline__ float finite_base(float top) { return top == -INFINITY ? 0.0f : top; }

// L: at least topk and merged as lists, or 0.  65536 x 256, top 8, in bf16 in
// 21 us (30 us by taking the largest eight times), 100003 x 60, top 4, in fp32 in
// 13 us; bound by vector instructions, about 500 for the four rows of a wave.
template <bool BF16, typename R, int L>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a)
{
    using K = Key<BF16>;
    using T = typename K::T;
    constexpr int G = R::G, PER = R::PER, kGroups = kRouteThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;  // choices per lane
    __shared__ int count[G * PER + 1];
    __shared__ float sums[kRouteWaves][G * PER];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const int64_t step = int64_t(gridDim.x) * kGroups, bytes = step * a.experts * R::kEs;
    for (int i = threadIdx.x; i <= a.experts; i += kRouteThreads)
        count[i] = 0;
    __syncthreads();
    float sum[PER];
#pragma unroll
    for (int s = 0; s < PER; ++s)
        sum[s] = 0.0f;
    int kept = 0;
    int64_t r = int64_t(blockIdx.x) * kGroups + group;
    const char *from = static_cast<const char *>(a.logits) + r * a.experts * R::kEs;
    R row;
    unsigned char keep = 1;
    if (r < a.rows) {
        row.load(from, lane, a.experts);
        if (a.keep)
            keep = a.keep[r];
    }
    for (; r < a.rows; r += step) {
        // the next row is on its way meanwhile
        R next = row;
        unsigned char next_keep = 1;
        from += bytes;
        if (r + step < a.rows) {
            next.load(from, lane, a.experts);
            if (a.keep)
                next_keep = a.keep[r + step];
        }
        int mine[kKeep];
        float w[kKeep], lse = 0.0f;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            mine[i] = -1, w[i] = 0.0f;
        if (keep) {
            row.pad(lane, a.experts);
            float z[PER], total, base;
            T top_key;
            T key[PER];
            bool nan = false;
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                key[s] = K::make(order_key(row.get(s)), R::expert(lane, s));
                if (s % 2)
                    nan |= __builtin_isunordered(row.get(s - 1), row.get(s));
            }
            if (nan) {
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    if (row.get(s) != row.get(s))
                        key[s] = K::make(kNanKey, R::expert(lane, s));
            }
            if constexpr (L > 0) {
                T best[L];
                sort_top<K, PER, L>(key, best);
                merge_lanes<K, G, (PER < L ? PER : L), L>(best);
                top_key = best[0];
                constexpr int kHave = PER * G < L ? PER * G : L;
#pragma unroll
                for (int i = 0; i < kKeep; ++i) {
                    T k = best[0];
#pragma unroll
                    for (int n = 1; n < kHave; ++n)
                        k = i * G + lane == n ? best[n] : k;
                    mine[i] = K::expert(k);
                    w[i] = K::value(k);
                }
            } else {
                top_key = key[0];
                for (int k = 0; k < a.topk; ++k) {
                    T best = key[0];
#pragma unroll
                    for (int s = 1; s < PER; ++s)
                        best = K::larger(best, key[s]);
                    best = across<G>(best, [](T x, T y) { return K::larger(x, y); });
                    top_key = k == 0 ? best : top_key;
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        key[s] = key[s] == best ? T(0) : key[s];
#pragma unroll
                    for (int i = 0; i < kKeep; ++i)
                        if (k == i * G + lane) {
                            mine[i] = K::expert(best);
                            w[i] = K::value(best);
                        }
                }
            }
            base = finite_base(K::value(top_key));
            total = 0.0f;
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                z[s] = exp_from(row.get(s), base);
                total += z[s];
            }
            total = lanes_sum<G>(total);
            float chosen = 0.0f;
            const float inv = total == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(total);
#pragma unroll
            for (int s = 0; s < PER; ++s)
                sum[s] = __builtin_fmaf(z[s], inv, sum[s]);
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                w[i] = i * G + lane < a.topk ? exp_from(w[i], base) : 0.0f;
                chosen += w[i];
            }
            float by = inv;
            if (a.renormalize) {
                chosen = lanes_sum<G>(chosen);
                by = chosen == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(chosen);
            }
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                w[i] *= by;
                if (i * G + lane < a.topk)
                    atomicAdd(&count[mine[i]], 1);
            }
            lse = __builtin_fmaf(__builtin_amdgcn_logf(total), kLn2, K::value(top_key));
            ++kept;
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (i * G + lane < a.topk) {
                a.choice[r * a.topk + i * G + lane] = mine[i];
                a.weight[r * a.topk + i * G + lane] = w[i];
            }
        if (lane == 0)
            a.lse[r] = lse;
        row = next;
        keep = next_keep;
    }
    if (lane == 0 && kept)
        atomicAdd(&count[a.experts], kept);
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        for (int d = G; d < 64; d *= 2)
            sum[s] += __shfl_xor(sum[s], d);
        if (threadIdx.x % 64 < G)
            sums[threadIdx.x / 64][R::expert(lane, s)] = sum[s];
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= a.experts; i += kRouteThreads) {
        if (i < a.experts) {
            float t = 0.0f;
            for (int w = 0; w < kRouteWaves; ++w)
                t += sums[w][i];
            a.prob_sum[int64_t(blockIdx.x) * a.experts + i] = t;
        }
        a.counts[int64_t(blockIdx.x) * (a.experts + 1) + i] = count[i];
    }
}

// Sixteen experts per workgroup, 64 threads for each: 512 parts of 256 in 4 us.
constexpr int kSumThreads = 1024, kSumWide = 16;

__global__ __launch_bounds__(kSumThreads) void route_sum_kernel(RouteSumArgs a)
{
    __shared__ int ns[kSumThreads];
    __shared__ float ss[kSumThreads];
    const int i = blockIdx.x * kSumWide + threadIdx.x % kSumWide, first = threadIdx.x / kSumWide;
    const int in = i < a.experts ? i : a.experts, is = i < a.experts ? i : 0;
    constexpr int kStep = kSumThreads / kSumWide;
    int n = 0;
    float s = 0.0f;
#pragma unroll 8
    for (int b = first; b < a.blocks; b += kStep) {
        n += a.part_counts[int64_t(b) * (a.experts + 1) + in];
        s += a.part_sum[int64_t(b) * a.experts + is];
    }
    ns[threadIdx.x] = n;
    ss[threadIdx.x] = s;
    for (int half = kSumThreads / 2; half >= kSumWide; half /= 2) {
        __syncthreads();
        if (int(threadIdx.x) < half) {
            ns[threadIdx.x] += ns[threadIdx.x + half];
            ss[threadIdx.x] += ss[threadIdx.x + half];
        }
    }
    if (first == 0 && i <= a.experts) {
        a.counts[i] = ns[threadIdx.x];
        if (i < a.experts)
            a.prob_sum[i] = ss[threadIdx.x];
    }
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
    s = lanes_sum<64>(s);
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

// What one row's gradient needs beside its logits, of the choices that a lane
// holds.
template <int KEEP>
struct Chosen {
    int c[KEEP];
    float w[KEEP], g[KEEP], lse;
    int keep;

    template <int G>
    __device__ void load(const RouteGradArgs &a, int64_t r, int lane)
    {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t n = r * a.topk + (i * G + lane < a.topk ? i * G + lane : 0);
            c[i] = a.choice[n];
            w[i] = a.weight[n];
            g[i] = a.grad_weight[n];
        }
        lse = a.lse[r];
        keep = a.keep ? a.keep[r] : 1;
    }
};

// The chosen experts' own terms lie in LDS, zero at every other expert, and
// are zeroed again once read.  65536 x 256 in bf16 in 12.4 us, 5.9 TB/s.
template <bool BF16, typename R, int L, bool RENORM>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a)
{
    constexpr int G = R::G, PER = R::PER, V = R::V, kGroups = kThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;
    __shared__ __attribute__((aligned(16))) float chosen_terms[kGroups][G * PER];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    float *own = chosen_terms[group];
    const int64_t step = int64_t(gridDim.x) * kGroups;
    int64_t r = int64_t(blockIdx.x) * kGroups + group;
    if (r >= a.rows)
        return;
    R row;
    Chosen<kKeep> of;
    row.load(static_cast<const char *>(a.logits) + r * a.experts * R::kEs, lane, a.experts);
    of.template load<G>(a, r, lane);
    const float gl = a.grad_loss[0];
    float slope[PER];
#pragma unroll
    for (int s = 0; s < PER; s += V) {
        const int e = R::expert(lane, s);
        __builtin_memcpy(&slope[s], a.slope + (e < a.experts ? e : 0), 4 * V);
        for (int n = 0; n < V; ++n)
            own[e + n] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < PER; ++s)
        slope[s] *= gl;
    for (; r < a.rows; r += step) {
        R next = row;
        Chosen<kKeep> next_of = of;
        if (r + step < a.rows) {
            next.load(static_cast<const char *>(a.logits) + (r + step) * a.experts * R::kEs, lane, a.experts);
            next_of.template load<G>(a, r + step, lane);
        }
        float d[PER];
        if (of.keep) {
            row.pad(lane, a.experts);
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                if (i * G + lane >= a.topk || unsigned(of.c[i]) >= unsigned(a.experts))
                    of.c[i] = -1;
                mean += i * G + lane < a.topk ? of.w[i] * of.g[i] : 0.0f;
            }
            if constexpr (RENORM)
                mean = lanes_sum<G>(mean);
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (of.c[i] >= 0)
                    own[of.c[i]] = RENORM ? of.w[i] * (of.g[i] - mean) : of.g[i];
            // one wave's LDS operations keep their order; so has the compiler to
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const float base = finite_base(of.lse);
            float p[PER], term[PER], dot = 0.0f;
#pragma unroll
            for (int s = 0; s < PER; s += V)
                __builtin_memcpy(&term[s], __builtin_assume_aligned(own + R::expert(lane, s), V % 4 ? 4 * V : 16), 4 * V);
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                p[s] = exp_from(row.get(s), base);
                d[s] = RENORM ? slope[s] : slope[s] + term[s];
                dot = __builtin_fmaf(p[s], d[s], dot);
            }
            dot = lanes_sum<G>(dot);
#pragma unroll
            for (int s = 0; s < PER; ++s)
                d[s] = RENORM ? __builtin_fmaf(p[s], d[s] - dot, term[s]) : p[s] * (d[s] - dot);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (of.c[i] >= 0)
                    own[of.c[i]] = 0.0f;
        } else {
#pragma unroll
            for (int s = 0; s < PER; ++s)
                d[s] = 0.0f;
        }
        row.set(d);
        row.store(static_cast<char *>(a.dlogits) + r * a.experts * R::kEs, lane, a.experts);
        row = next;
        of = next_of;
    }
}

}  // namespace

int32_t route_blocks(int64_t rows, int32_t experts)
{
    const int64_t groups = kRouteThreads / lanes_of(experts), n = (rows + groups - 1) / groups;
    // up to four rows per group a second launch costs more than it saves; 512
    // workgroups fill the compute units, more only make the sums longer
    return n <= 4 ? 1 : int32_t(n < 512 ? n : 512);
}

namespace {

template <bool BF16>
hipError_t route(const RouteArgs &a, hipStream_t stream)
{
    return with_row<BF16>(a.experts, [&](auto row) {
        return with_list(a.topk, [&](auto list) {
            route_kernel<BF16, decltype(row), decltype(list)::value>
                <<<dim3(unsigned(a.blocks)), dim3(kRouteThreads), 0, stream>>>(a);
            return hipGetLastError();
        });
    });
}

template <bool BF16>
hipError_t route_grad(const RouteGradArgs &a, hipStream_t stream)
{
    const int64_t groups = kThreads / lanes_of(a.experts), n = (a.rows + groups - 1) / groups;
    const dim3 grid(unsigned(n < 2048 ? n : 2048)), threads(kThreads);
    return with_row<BF16>(a.experts, [&](auto row) {
        using R = decltype(row);
        if (a.topk <= 8 && a.renormalize)
            route_grad_kernel<BF16, R, 8, true><<<grid, threads, 0, stream>>>(a);
        else if (a.topk <= 8)
            route_grad_kernel<BF16, R, 8, false><<<grid, threads, 0, stream>>>(a);
        else if (a.renormalize)
            route_grad_kernel<BF16, R, 0, true><<<grid, threads, 0, stream>>>(a);
        else
            route_grad_kernel<BF16, R, 0, false><<<grid, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_route(const Op &op, hipStream_t stream)
{
    const RouteArgs a = op.get<RouteArgs>();
    (void)hipGetLastError();
    return a.bf16 ? route<true>(a, stream) : route<false>(a, stream);
}

hipError_t launch_route_sum(const Op &op, hipStream_t stream)
{
    const RouteSumArgs a = op.get<RouteSumArgs>();
    (void)hipGetLastError();
    route_sum_kernel<<<dim3(unsigned(a.experts / kSumWide + 1)), dim3(kSumThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance(const Op &op, hipStream_t stream)
{
    const BalanceArgs a = op.get<BalanceArgs>();
    (void)hipGetLastError();
    balance_kernel<<<dim3(1), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_grad(const Op &op, hipStream_t stream)
{
    const RouteGradArgs a = op.get<RouteGradArgs>();
    (void)hipGetLastError();
    return a.bf16 ? route_grad<true>(a, stream) : route_grad<false>(a, stream);
}

}  // namespace rr
