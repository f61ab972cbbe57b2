// rr_group_route.hip -- gfx950 kernels of the router in groups: the groups and
// experts of a token by their choice scores s + bias, the weights, the counts,
// the bias's next step and the gradient.
//
// A row is held by G lanes, each of its groups by as many of them as fit (a power
// of two), PER experts each.  The choice scores are doubles, whose vector
// instructions run at the rate of floats here: a choice that 32-bit roundings
// decide would differ from any other implementation's.  Ten low bits of a score
// give way to the expert's index, so that one maximum orders scores and indices.
#include "rr_expert.h"
#include "rr_rows.h"

namespace rr {
namespace {

constexpr int kThreads = 256;
constexpr int kRouteThreads = 512;

// What stands for NaN, the infinities and places without an expert among the keys.
constexpr double kNan = 0x1p1000, kInf = 0x1p900, kDead = -0x1p1000;

// A choice score and its expert as one number, larger for the larger score and for
// the lower index among equals.
struct Key {
    typedef double T;
    static_assert(RR_MAX_EXPERTS <= 1024, "the index has ten bits");
    __device__ static T make(double c, int e)
    {
        c = c != c ? kNan : fmin(fmax(c, -kInf), kInf);
        const unsigned long long u = __builtin_bit_cast(unsigned long long, c);
        const unsigned at = (u >> 63) ? unsigned(e) : unsigned(1023 - e);
        return __builtin_bit_cast(double, (u & ~1023ull) | at);
    }
    __device__ static int expert(T k)
    {
        const unsigned long long u = __builtin_bit_cast(unsigned long long, k);
        const int at = int(u & 1023u);
        return (u >> 63) ? at : 1023 - at;
    }
    __device__ static double score(T k)
    {
        return __builtin_bit_cast(double, __builtin_bit_cast(unsigned long long, k) & ~1023ull);
    }
    __device__ static bool none(T k) { return k < -0x1p800; }
    __device__ static T larger(T a, T b) { return fmax(a, b); }
    __device__ static T smaller(T a, T b) { return fmin(a, b); }
};

template <int G>
__device__ __forceinline__ double lanes_sum64(double v)
{
    return across<G>(v, [](double a, double b) { return a + b; });
}

__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

// The two largest of the lanes of a group (LANES of them, a power of two).
template <int G, int STEP = 0>
__device__ __forceinline__ void best_two(double &a, double &b, int lanes)
{
    if constexpr (1 << STEP < G) {
        if (1 << STEP < lanes) {
            const double oa = other<STEP>(a), ob = other<STEP>(b);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
            best_two<G, STEP + 1>(a, b, lanes);
        }
    }
}

// lanes: of a group.  L: at least topk and merged as lists, or 0.
template <bool BF16, int G, int PER, int V, int L>
__global__ __launch_bounds__(kRouteThreads) void group_route_kernel(GroupRouteArgs a, int lanes)
{
    using T = Key::T;
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    constexpr int kGroups = kRouteThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;  // choices per lane
    __shared__ int count[RR_MAX_EXPERTS + 1];
    const int lane = threadIdx.x % G, of_row = threadIdx.x / G, size = a.experts / a.groups;
    const int group = lane / lanes, first = lane % lanes * PER;  // the lane's experts: first.. of its group
    for (int i = threadIdx.x; i <= a.experts; i += kRouteThreads)
        count[i] = 0;
    __syncthreads();
    int kept = 0;
    for (int64_t r = int64_t(blockIdx.x) * kGroups + of_row; r < a.rows; r += int64_t(gridDim.x) * kGroups) {
        const Raw *from = static_cast<const Raw *>(a.logits) + r * a.experts;
        int mine[kKeep];
        float w[kKeep], z_of[kKeep], lse = 0.0f;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            mine[i] = -1, w[i] = 0.0f, z_of[i] = -INFINITY;
        if (!a.keep || a.keep[r]) {
            float z[PER], bias[PER];
#pragma unroll
            for (int s = 0; s < PER; s += V) {
                const int at = group < a.groups && first + s < size ? group * size + first + s : 0;
                Raw v[V];
                __builtin_memcpy(v, from + at, sizeof v);
#pragma unroll
                for (int n = 0; n < V; ++n)
                    z[s + n] = __uint_as_float(BF16 ? unsigned(v[n]) << 16 : unsigned(v[n]));
                if (a.bias)
                    __builtin_memcpy(&bias[s], a.bias + at, 4 * V);
            }
            T key[PER];
            double total = 1.0, inv = 1.0;
            float top = -INFINITY, base = 0.0f;
            if (!a.sigmoid) {
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    top = group < a.groups && first + s < size ? fmaxf(top, z[s]) : top;
                top = lanes_max<G>(top);
                base = top == -INFINITY ? 0.0f : top;
                total = 0.0;
            }
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                const bool in = group < a.groups && first + s < size;
                double c;
                if (a.sigmoid) {
                    c = sigmoid64(double(z[s]));
                } else {
                    c = exp(double(z[s]) - double(base));
                    total += in ? c : 0.0;
                }
                key[s] = c;
            }
            if (!a.sigmoid) {
                total = lanes_sum64<G>(total);
                inv = total == 0.0 ? 0.0 : 1.0 / total;
                lse = total == 0.0 ? -INFINITY : float(double(base) + log(total));
            }
            double one = kDead, two = kDead;
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                const bool in = group < a.groups && first + s < size;
                double c = a.sigmoid ? key[s] : key[s] * inv;
                c = a.bias ? c + double(bias[s]) : c;
                key[s] = in ? Key::make(c, group * size + first + s) : kDead;
                const double v = in ? Key::score(key[s]) : kDead;
                two = fmax(two, fmin(one, v));
                one = fmax(one, v);
            }
            if (a.top_groups < a.groups) {
                best_two<G>(one, two, lanes);
                const double mark = a.group_best == 2 ? one + two : one;
                int before = 0;
                for (int g = 0; g < a.groups; ++g) {
                    const double m = __shfl(mark, int(threadIdx.x % 64) / G * G + g * lanes);
                    before += m > mark || (m == mark && g < group);
                }
                if (before >= a.top_groups) {
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        key[s] = kDead;
                }
            }
            T pick[kKeep];
            if constexpr (L > 0) {
                T best[L];
                sort_top<Key, PER, L>(key, best);
                merge_lanes<Key, G, (PER < L ? PER : L), L>(best);
                constexpr int kHave = PER * G < L ? PER * G : L;
#pragma unroll
                for (int i = 0; i < kKeep; ++i) {
                    pick[i] = best[0];
#pragma unroll
                    for (int n = 1; n < kHave; ++n)
                        pick[i] = i * G + lane == n ? best[n] : pick[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < kKeep; ++i)
                    pick[i] = kDead;
                for (int k = 0; k < a.topk; ++k) {
                    T best = key[0];
#pragma unroll
                    for (int s = 1; s < PER; ++s)
                        best = fmax(best, key[s]);
                    best = across<G>(best, [](T x, T y) { return fmax(x, y); });
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        key[s] = key[s] == best ? kDead : key[s];
#pragma unroll
                    for (int i = 0; i < kKeep; ++i)
                        pick[i] = k == i * G + lane ? best : pick[i];
                }
            }
            double s_of[kKeep], sum = 0.0;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                s_of[i] = 0.0;
                if (i * G + lane < a.topk && !Key::none(pick[i])) {
                    mine[i] = Key::expert(pick[i]);
                    const Raw v = from[mine[i]];
                    z_of[i] = __uint_as_float(BF16 ? unsigned(v) << 16 : unsigned(v));
                    s_of[i] = a.sigmoid ? sigmoid64(double(z_of[i])) : exp(double(z_of[i]) - double(base)) * inv;
                    sum += s_of[i];
                    atomicAdd(&count[mine[i]], 1);
                }
            }
            double by = double(a.scale);
            if (a.renormalize) {
                sum = lanes_sum64<G>(sum);
                by = sum == 0.0 ? 0.0 : by / sum;
            }
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                w[i] = mine[i] >= 0 ? float(s_of[i] * by) : 0.0f;
            ++kept;
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (i * G + lane < a.topk) {
                const int64_t at = r * a.topk + i * G + lane;
                a.choice[at] = mine[i];
                a.weight[at] = w[i];
                a.logit[at] = z_of[i];
            }
        if (lane == 0 && !a.sigmoid && a.lse)
            a.lse[r] = lse;
    }
    if (lane == 0 && kept)
        atomicAdd(&count[a.experts], kept);
    __syncthreads();
    for (int i = threadIdx.x; i <= a.experts; i += kRouteThreads)
        a.counts[int64_t(blockIdx.x) * (a.experts + 1) + i] = count[i];
}

// Sixteen experts per workgroup, 64 threads for each.
constexpr int kSumThreads = 1024, kSumWide = 16;

__global__ __launch_bounds__(kSumThreads) void count_sum_kernel(CountSumArgs a)
{
    __shared__ int ns[kSumThreads];
    const int i = blockIdx.x * kSumWide + threadIdx.x % kSumWide, first = threadIdx.x / kSumWide;
    const int in = i <= a.experts ? i : a.experts;
    int n = 0;
#pragma unroll 8
    for (int b = first; b < a.blocks; b += kSumThreads / kSumWide)
        n += a.part[int64_t(b) * (a.experts + 1) + in];
    ns[threadIdx.x] = n;
    for (int half = kSumThreads / 2; half >= kSumWide; half /= 2) {
        __syncthreads();
        if (int(threadIdx.x) < half)
            ns[threadIdx.x] += ns[threadIdx.x + half];
    }
    if (first == 0 && i <= a.experts)
        a.counts[i] = ns[threadIdx.x];
}

// One workgroup: sign(sum n - experts * n_e), in whole numbers.
__global__ __launch_bounds__(kThreads) void route_bias_kernel(RouteBiasArgs a)
{
    __shared__ long long sums[kThreads];
    long long all = 0;
    for (int i = threadIdx.x; i < a.experts; i += kThreads)
        for (int r = 0; r < a.ranks; ++r)
            all += a.counts[r][i];
    sums[threadIdx.x] = all;
    for (int half = kThreads / 2; half > 0; half /= 2) {
        __syncthreads();
        if (int(threadIdx.x) < half)
            sums[threadIdx.x] += sums[threadIdx.x + half];
    }
    __syncthreads();
    all = sums[0];
    for (int i = threadIdx.x; i < a.experts; i += kThreads) {
        long long n = 0;
        for (int r = 0; r < a.ranks; ++r)
            n += a.counts[r][i];
        n *= a.experts;
        a.out[i] = a.bias[i] + (all > n ? a.rate : all < n ? -a.rate : 0.0f);
    }
}

// What one row's gradient needs, of the choices that a lane holds.
template <int KEEP>
struct Chosen {
    int c[KEEP];
    float z[KEEP], g[KEEP], lse;

    template <int G>
    __device__ void load(const GroupGradArgs &a, int64_t r, int lane, bool whole)
    {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int64_t n = r * a.topk + (i * G + lane < a.topk ? i * G + lane : 0);
            c[i] = a.choice[n];
            z[i] = a.logit[n];
            g[i] = a.grad_weight[n];
        }
        lse = whole ? a.lse[r] : 0.0f;
    }
};

// The chosen experts' terms lie in LDS, zero at every other expert, and are zeroed
// again once read.  Only softmax that is not renormalized (WHOLE) reads the logits.
//   sigmoid: ds/dz = s (1 - s) with 1 - s = sigmoid(-z); softmax: dz_e = p_e (d_e - sum p d).
template <bool BF16, typename R, int L, bool WHOLE>
__global__ __launch_bounds__(kThreads) void group_grad_kernel(GroupGradArgs a)
{
    constexpr int G = R::G, PER = R::PER, V = R::V, kGroups = kThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;
    __shared__ __attribute__((aligned(16))) float chosen_terms[kGroups][G * PER];
    const int lane = threadIdx.x % G, of_row = threadIdx.x / G;
    float *own = chosen_terms[of_row];
    const int64_t step = int64_t(gridDim.x) * kGroups;
    int64_t r = int64_t(blockIdx.x) * kGroups + of_row;
    if (r >= a.rows)
        return;
#pragma unroll
    for (int s = 0; s < PER; ++s)
        own[R::expert(lane, s)] = 0.0f;
    Chosen<kKeep> of;
    of.template load<G>(a, r, lane, WHOLE);
    for (; r < a.rows; r += step) {
        R row;
        if constexpr (WHOLE)
            row.load(static_cast<const char *>(a.logits) + r * a.experts * R::kEs, lane, a.experts);
        Chosen<kKeep> next = of;
        if (r + step < a.rows)
            next.template load<G>(a, r + step, lane, WHOLE);
        float term[kKeep], dot = 0.0f;
        int live = 0;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (i * G + lane >= a.topk || unsigned(of.c[i]) >= unsigned(a.experts))
                of.c[i] = -1;
            live |= of.c[i] >= 0;
        }
        if (WHOLE) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                term[i] = of.c[i] >= 0 ? a.scale * of.g[i] : 0.0f;
                dot += of.c[i] >= 0 ? expf(of.z[i] - (of.lse == -INFINITY ? 0.0f : of.lse)) * term[i] : 0.0f;
            }
            dot = lanes_sum<G>(dot);
            live = lanes_max<G>(live ? 1.0f : 0.0f) > 0.0f;
        } else {
            // in 64 bits: s of logits far below 0 are small, their quotients are not
            double s[kKeep], t[kKeep], sum = 0.0, mean = 0.0;
            float top = -INFINITY;
            if (!a.sigmoid) {
#pragma unroll
                for (int i = 0; i < kKeep; ++i)
                    top = of.c[i] >= 0 ? fmaxf(top, of.z[i]) : top;
                top = lanes_max<G>(top);
                top = top == -INFINITY ? 0.0f : top;
            }
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const double z = double(of.z[i]);
                s[i] = of.c[i] < 0 ? 0.0 : a.sigmoid ? sigmoid64(z) : exp(z - double(top));
                t[i] = a.sigmoid ? sigmoid64(-z) : 1.0;
                sum += s[i];
                mean += of.c[i] < 0 ? 0.0 : s[i] * double(of.g[i]);
            }
            double by = double(a.scale);
            if (a.renormalize) {
                sum = lanes_sum64<G>(sum);
                mean = lanes_sum64<G>(mean);
                by = sum == 0.0 ? 0.0 : by / sum;
                mean = sum == 0.0 ? 0.0 : mean / sum;
            } else {
                mean = 0.0;
            }
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                term[i] = of.c[i] < 0 ? 0.0f : float(s[i] * t[i] * by * (double(of.g[i]) - mean));
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (of.c[i] >= 0)
                own[of.c[i]] = term[i];
        // one wave's LDS operations keep their order; so has the compiler to
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float d[PER];
#pragma unroll
        for (int s = 0; s < PER; s += V)
            __builtin_memcpy(&d[s], __builtin_assume_aligned(own + R::expert(lane, s), V % 4 ? 4 * V : 16), 4 * V);
        if constexpr (WHOLE) {
            const float base = of.lse == -INFINITY ? 0.0f : of.lse;
#pragma unroll
            for (int s = 0; s < PER; ++s)
                d[s] = live ? expf(row.get(s) - base) * (d[s] - dot) : 0.0f;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (of.c[i] >= 0)
                own[of.c[i]] = 0.0f;
        row.set(d);
        row.store(static_cast<char *>(a.dlogits) + r * a.experts * R::kEs, lane, a.experts);
        of = next;
    }
}

// A row's layout: `lanes` of G hold a group, `per` experts each.
struct Layout {
    int g, lanes, per;
};

Layout layout_of(int experts, int groups)
{
    int padded = 1;
    while (padded < groups)
        padded *= 2;
    const int size = experts / groups;
    // sixteen lanes where they hold a row in sixteen registers each
    for (const int g : {16, 64})
        if (padded <= g && (g == 64 || (size + g / padded - 1) / (g / padded) <= 16)) {
            const int lanes = g / padded;
            return Layout{g, lanes, (size + lanes - 1) / lanes};
        }
    return Layout{0, 0, 0};
}

template <bool BF16, int G, int PER>
hipError_t route(const GroupRouteArgs &a, int lanes, hipStream_t stream)
{
    const dim3 grid(unsigned(a.blocks)), threads(kRouteThreads);
    const bool four = a.experts / a.groups % 4 == 0;
    if (a.topk <= 8 && four)
        group_route_kernel<BF16, G, PER, 4, 8><<<grid, threads, 0, stream>>>(a, lanes);
    else if (a.topk <= 8)
        group_route_kernel<BF16, G, PER, 1, 8><<<grid, threads, 0, stream>>>(a, lanes);
    else if (four)
        group_route_kernel<BF16, G, PER, 4, 0><<<grid, threads, 0, stream>>>(a, lanes);
    else
        group_route_kernel<BF16, G, PER, 1, 0><<<grid, threads, 0, stream>>>(a, lanes);
    return hipGetLastError();
}

template <bool BF16>
hipError_t route(const GroupRouteArgs &a, hipStream_t stream)
{
    const Layout l = layout_of(a.experts, a.groups);
    if (l.g == 16)
        return l.per <= 4 ? route<BF16, 16, 4>(a, l.lanes, stream) : l.per <= 8 ? route<BF16, 16, 8>(a, l.lanes, stream)
                                                                              : route<BF16, 16, 16>(a, l.lanes, stream);
    return l.per <= 8 ? route<BF16, 64, 8>(a, l.lanes, stream) : l.per <= 16 ? route<BF16, 64, 16>(a, l.lanes, stream)
                                                                           : route<BF16, 64, 32>(a, l.lanes, stream);
}

template <bool BF16>
hipError_t grad(const GroupGradArgs &a, hipStream_t stream)
{
    const int64_t groups = kThreads / lanes_of(a.experts), n = (a.rows + groups - 1) / groups;
    const dim3 grid(unsigned(n < 2048 ? n : 2048)), threads(kThreads);
    const bool whole = !a.sigmoid && !a.renormalize;
    return with_row<BF16>(a.experts, [&](auto row) {
        using R = decltype(row);
        if (a.topk <= 8 && whole)
            group_grad_kernel<BF16, R, 8, true><<<grid, threads, 0, stream>>>(a);
        else if (a.topk <= 8)
            group_grad_kernel<BF16, R, 8, false><<<grid, threads, 0, stream>>>(a);
        else if (whole)
            group_grad_kernel<BF16, R, 0, true><<<grid, threads, 0, stream>>>(a);
        else
            group_grad_kernel<BF16, R, 0, false><<<grid, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace

int32_t group_route_blocks(int64_t rows, int32_t experts, int32_t groups)
{
    const int64_t per = kRouteThreads / layout_of(experts, groups).g, n = (rows + per - 1) / per;
    // up to four rows per group of lanes a second launch costs more than it saves
    return n <= 4 ? 1 : int32_t(n < 512 ? n : 512);
}

hipError_t launch_group_route(const Op &op, hipStream_t stream)
{
    const GroupRouteArgs a = op.get<GroupRouteArgs>();
    (void)hipGetLastError();
    return a.bf16 ? route<true>(a, stream) : route<false>(a, stream);
}

hipError_t launch_count_sum(const Op &op, hipStream_t stream)
{
    const CountSumArgs a = op.get<CountSumArgs>();
    (void)hipGetLastError();
    count_sum_kernel<<<dim3(unsigned(a.experts / kSumWide + 1)), dim3(kSumThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_bias(const Op &op, hipStream_t stream)
{
    const RouteBiasArgs a = op.get<RouteBiasArgs>();
    (void)hipGetLastError();
    route_bias_kernel<<<dim3(1), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_group_grad(const Op &op, hipStream_t stream)
{
    const GroupGradArgs a = op.get<GroupGradArgs>();
    (void)hipGetLastError();
    return a.bf16 ? grad<true>(a, stream) : grad<false>(a, stream);
}

}  // namespace rr
