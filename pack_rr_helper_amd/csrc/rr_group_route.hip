// rr_group_route.hip -- gfx950 kernels of the router in groups: the groups and
// experts of a token by their choice scores s + bias, the weights, the counts,
// the bias's next step and the gradient.
//
// A row is held by G lanes, each of its groups by as many of them as fit (a power
// of two), PER experts each.  A choice that 32-bit roundings decide would differ from any
// other implementation's, so that it is made in 64 bits wherever that can matter:
// scores are ordered in 32 bits first, and if no decision of the wave's rows was closer
// than their roundings, those decisions stand.  Else the wave starts again in 64 bits.
// How often depends on the logits and the bias, as an exact tie is always too close: 65536 x
// 256, top 8 of 4 of 8 groups, in bf16, with the counts' launch, take 47-51 us with a bias of
// random numbers or of multiples of 0.001 up to 0.1, 54 us of such up to 0.02, and without a
// bias, where most waves meet two equal logits, 90 us (in fp32, where they are rare, 47 us with
// any).
// Either way a score's low bits give way to the expert's index, so that one maximum
// orders both.
#include "rr_expert.h"
#include "rr_rows.h"

namespace rr {
namespace {

constexpr int kThreads = 256;
constexpr int kRouteThreads = 256;

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
};

template <int G>
__device__ __forceinline__ double lanes_sum64(double v)
{
    return across<G>(v, [](double a, double b) { return a + b; });
}

// exp(x) for |x| <= 700, to 2^-45: 2^n 2^f with f in [-1/2, 1/2], and 2^f = exp(f ln 2) by
// its series up to the eleventh power, (ln 2 / 2)^12 / 12! = 2^-47 being left.
__device__ __forceinline__ double exp64(double x)
{
    const double t = x * 1.4426950408889634074, n = __builtin_rint(t);
    // ln 2 is off by 2^-55, n is at most 1010
    const double f = __builtin_fma(n, -0.69314718055994530942, x);
    double p = 1.0 / 39916800;
    constexpr double kOver[] = {1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 11; ++i)
        p = __builtin_fma(p, f, kOver[i]);
    return __builtin_amdgcn_ldexp(p, int(n));
}

// 1 / d for 1 <= d < 2^1011, to 2^-45: an approximation and one step of Newton's.
__device__ __forceinline__ double inverse64(double d)
{
    const double y = __builtin_amdgcn_rcp(d);
    return __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
}

// The range of logits that exp64 takes; others, and NaN, go by definition.
constexpr float kReach = 700.0f;

__device__ __forceinline__ bool in_reach(float z) { return fabsf(z) <= kReach; }

// sigmoid(z), to 2^-44 in reach.
__device__ __forceinline__ double sigmoid64(float z)
{
    const double s = inverse64(1.0 + exp64(-double(__builtin_amdgcn_fmed3f(z, -kReach, kReach))));
    return in_reach(z) ? s : z != z ? __builtin_nan("") : z > 0.0f ? 1.0 : 0.0;
}

// exp(z - base), z <= base; 0 for a z further away than doubles hold.
__device__ __forceinline__ double exp_from64(float z, float base)
{
    const double d = double(z) - double(base);
    const double e = exp64(fmax(d, -double(kReach)));
    return d >= -double(kReach) ? e : d != d ? __builtin_nan("") : 0.0;
}

// The same in either width.
template <typename T>
__device__ __forceinline__ T exp_from(float z, float base)
{
    if constexpr (std::is_same_v<T, double>)
        return exp_from64(z, base);
    else
        return expf(z - base);
}

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

// The logits of the experts that a lane holds, V side by side; two of bf16 to a word.
template <bool BF16, int PER, int V>
struct Held {
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    static constexpr bool kPairs = BF16 && V > 1;
    static constexpr int kWords = kPairs ? PER / 2 : PER;
    unsigned w[kWords];

    // Experts past the row are anything: the row's first.
    __device__ void load(const Raw *row, int at, int end)
    {
#pragma unroll
        for (int s = 0; s < PER; s += V) {
            const Raw *p = row + (at + s < end ? at + s : 0);
            if constexpr (V == 1)
                w[s] = *p;
            else
                __builtin_memcpy(&w[kPairs ? s / 2 : s], p, V * sizeof(Raw));
        }
    }
    __device__ float get(int s) const
    {
        if constexpr (kPairs)
            return __uint_as_float(s % 2 ? w[s / 2] & 0xffff0000u : w[s / 2] << 16);
        else
            return __uint_as_float(BF16 ? w[s] << 16 : w[s]);
    }
};

// What the scores of a workgroup's rows lie between, and how they become keys in 32 bits:
// steps of 1 / scale from `low` on, above the expert's index.
struct Scale {
    float low, scale;
    // Scores closer than that may be in another order: their exponentials, quotients and
    // sums round by less than 2^-22 (1 + |c|), and to steps.
    float margin;
    unsigned steps;
    bool use;          // no bias is so large that the steps' start would be off by more than 8
};

template <int BITS>
__device__ __forceinline__ Scale scale_of(const float *bias, int experts)
{
    float low = INFINITY, high = -INFINITY;
    bool fine = true;
    for (int i = threadIdx.x % 64; i < experts; i += 64) {
        fine &= fabsf(bias[i]) < 16.0f;
        low = fminf(low, bias[i]);
        high = fmaxf(high, bias[i]);
    }
    low = -lanes_max<64>(-low);
    high = lanes_max<64>(high);
    Scale s;
    s.low = low;
    s.scale = (float(1u << (32 - BITS)) - 64.0f) / (high - low + 1.0f);
    s.margin = 0x1p-20f * (2.0f + fmaxf(fabsf(low), fabsf(high)));
    s.steps = unsigned(s.margin * s.scale) + 3;
    s.use = !__any(!fine);
    return s;
}

// Keys in 32 bits; 0: none.
template <int BITS>
struct Short {
    typedef unsigned T;
    __device__ static T make(float c, const Scale &s, int e)
    {
        // above none, and below 2^(32 - BITS)
        return unsigned(__builtin_fmaf(c, s.scale, __builtin_fmaf(-s.low, s.scale, 16.5f))) << BITS | unsigned((1 << BITS) - 1 - e);
    }
    __device__ static int expert(T k) { return (1 << BITS) - 1 - int(k & ((1u << BITS) - 1)); }
    __device__ static T larger(T a, T b) { return a > b ? a : b; }
    __device__ static T smaller(T a, T b) { return a < b ? a : b; }
};

// The experts that a lane is to store (choice i * G + lane) by keys in 32 bits; false
// if a decision was closer than those tell.  p[s]: scores in 32 bits.
template <int BITS, int G, int PER, int L, int KEEP>
__device__ __forceinline__ bool choose_short(const GroupRouteArgs &a, const float *p, const float *bias, const Scale &scale,
                                             int lanes, int group, int at, int end, int *pick)
{
    using K = Short<BITS>;
    const int lane = threadIdx.x % G;
    unsigned key[PER];
    float one = -INFINITY, two = -INFINITY;
    bool sure = scale.use;
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        const bool in = at + s < end;
        const float c = p[s] + bias[s];
        sure &= c == c || !in;
        key[s] = in ? K::make(c, scale, at + s) : 0;
        const float v = in ? c : -INFINITY;
        two = fmaxf(two, fminf(one, v));
        one = fmaxf(one, v);
    }
    if (a.top_groups < a.groups) {
#pragma unroll
        for (int d = 1; d < G; d *= 2)
            if (d < lanes) {
                const float oa = __shfl_xor(one, d), ob = __shfl_xor(two, d);
                two = fmaxf(fminf(one, oa), fmaxf(two, ob));
                one = fmaxf(one, oa);
            }
        const float mark = a.group_best == 2 ? one + two : one;
        int before = 0;
#pragma unroll 8
        for (int g = 0; g < a.groups; ++g) {
            const float m = __shfl(mark, (int(threadIdx.x % 64) / G * G + g * lanes) & 63);
            before += m > mark;
            sure &= g == group || group >= a.groups || fabsf(m - mark) > 4.0f * scale.margin;
        }
        if (before >= a.top_groups) {
#pragma unroll
            for (int s = 0; s < PER; ++s)
                key[s] = 0;
        }
    }
    unsigned last = 0;
    if constexpr (L > 0) {
        unsigned best[L];
        sort_top<K, PER, L>(key, best);
        merge_lanes<K, G, (PER < L ? PER : L), L>(best);
        constexpr int kHave = PER * G < L ? PER * G : L;
        last = best[0];
#pragma unroll
        for (int n = 1; n < kHave; ++n)
            if (n < a.topk) {
                sure &= (best[n - 1] >> BITS) - (best[n] >> BITS) > scale.steps;
                last = best[n];
            }
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            unsigned k = best[0];
#pragma unroll
            for (int n = 1; n < kHave; ++n)
                k = i * G + lane == n ? best[n] : k;
            pick[i] = K::expert(k);
        }
    } else {
        unsigned mine[KEEP] = {};
        for (int k = 0; k < a.topk; ++k) {
            // the largest below the last
            unsigned best = 0;
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                const unsigned v = k == 0 || key[s] < last ? key[s] : 0;
                best = best > v ? best : v;
            }
            best = across<G>(best, [](unsigned x, unsigned y) { return x > y ? x : y; });
            sure &= k == 0 || (last >> BITS) - (best >> BITS) > scale.steps;
            last = best;
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                mine[i] = k == i * G + lane ? best : mine[i];
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            pick[i] = K::expert(mine[i]);
    }
    // the last one from all that were not chosen
    const unsigned least = last >> BITS > scale.steps ? (last >> BITS) - scale.steps : 0;
    unsigned above = 0;
#pragma unroll
    for (int s = 0; s < PER; ++s)
        above += (key[s] >> BITS) >= least;
    return sure && least > 0 && across<G>(above, [](unsigned x, unsigned y) { return x + y; }) == unsigned(a.topk);
}

// The same in 64 bits, -1 for places that no expert is left for.  Softmax: `base` and
// `inv`, the factor of exp(z - base).
template <bool SIGMOID, int G, int PER, int KEEP, typename H>
__device__ __forceinline__ void choose(const GroupRouteArgs &a, const H &z, const float *bias, int lanes, int group, int at,
                                       int end, float base, double inv, int *pick)
{
    const int lane = threadIdx.x % G;
    double key[PER], one = kDead, two = kDead;
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        const double c = (SIGMOID ? sigmoid64(z.get(s)) : exp_from64(z.get(s), base) * inv) + double(bias[s]);
        const bool in = at + s < end;
        key[s] = in ? Key::make(c, at + s) : kDead;
        const double v = in ? Key::score(key[s]) : kDead;
        two = fmax(two, fmin(one, v));
        one = fmax(one, v);
        // a few at a time: side by side they would not fit the registers
        if (s % 2)
            __builtin_amdgcn_sched_barrier(0);
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
    double mine[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        mine[i] = kDead;
    for (int k = 0; k < a.topk; ++k) {
        double best = key[0];
#pragma unroll
        for (int s = 1; s < PER; ++s)
            best = fmax(best, key[s]);
        best = across<G>(best, [](double x, double y) { return fmax(x, y); });
#pragma unroll
        for (int s = 0; s < PER; ++s)
            key[s] = key[s] == best ? kDead : key[s];
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            mine[i] = k == i * G + lane ? best : mine[i];
    }
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        pick[i] = Key::none(mine[i]) ? -1 : Key::expert(mine[i]);
}

// lanes: of a group.  L: at least topk and merged as lists, or 0.
template <bool SIGMOID, bool BF16, int G, int PER, int V, int L>
__global__ __launch_bounds__(kRouteThreads, PER <= 8 ? 4 : PER <= 16 ? 3 : 2) void group_route_kernel(GroupRouteArgs a, int lanes)
{
    using Raw = typename Held<BF16, PER, V>::Raw;
    constexpr int kGroups = kRouteThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;  // choices per lane
    __shared__ int count[RR_MAX_EXPERTS + 1];
    __shared__ float bias[RR_MAX_EXPERTS + 64 * PER];   // and what lanes read past the row
    const int lane = threadIdx.x % G, of_row = threadIdx.x / G, size = a.experts / a.groups;
    // the lane's experts: from `at` on, below `end`
    const int group = lane / lanes, at = group * size + lane % lanes * PER, end = group < a.groups ? group * size + size : 0;
    const int64_t step = int64_t(gridDim.x) * kGroups;
    int64_t r = int64_t(blockIdx.x) * kGroups + of_row;
    const Raw *from = static_cast<const Raw *>(a.logits) + r * a.experts;
    Held<BF16, PER, V> next{};
    unsigned char next_keep = 0;
    if (r < a.rows) {
        next.load(from, at, end);
        next_keep = a.keep ? a.keep[r] : 1;
    }
    for (int i = threadIdx.x; i <= a.experts; i += kRouteThreads)
        count[i] = 0;
    for (int i = threadIdx.x; i < RR_MAX_EXPERTS + 64 * PER; i += kRouteThreads)
        bias[i] = a.bias && i < a.experts ? a.bias[i] : 0.0f;
    __syncthreads();
    constexpr int kBits = G * PER <= 256 ? 8 : 10;
    const Scale scale = scale_of<kBits>(bias, a.experts);
    int kept = 0;
    for (; r < a.rows; r += step, from += step * a.experts) {
        const Held<BF16, PER, V> z = next;
        const bool keep = next_keep;
        // the next row is on its way meanwhile
        if (r + step < a.rows) {
            next.load(from + step * a.experts, at, end);
            next_keep = a.keep ? a.keep[r + step] : 1;
        }
        int mine[kKeep];
        float w[kKeep], z_of[kKeep], lse = 0.0f;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            mine[i] = -1, w[i] = 0.0f, z_of[i] = -INFINITY;
        if (keep) {
            float base = 0.0f, p[PER];
            double inv = 1.0;
            int pick[kKeep];
            if constexpr (!SIGMOID) {
                float top = -INFINITY;
                double total = 0.0;
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    top = at + s < end ? fmaxf(top, z.get(s)) : top;
                top = lanes_max<G>(top);
                base = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int s = 0; s < PER; ++s) {
                    const double e = at + s < end ? exp_from64(z.get(s), base) : 0.0;
                    p[s] = float(e);
                    total += e;
                    if (s % 2)
                        __builtin_amdgcn_sched_barrier(0);
                }
                total = lanes_sum64<G>(total);
                inv = total == 0.0 ? 0.0 : 1.0 / total;
                lse = total == 0.0 ? -INFINITY : float(double(base) + log(total));
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    p[s] *= float(inv);
            } else {
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    p[s] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z.get(s)));
            }
            if (__any(!choose_short<kBits, G, PER, L, kKeep>(a, p, bias + at, scale, lanes, group, at, end, pick)))
                choose<SIGMOID, G, PER, kKeep>(a, z, bias + at, lanes, group, at, end, base, inv, pick);
            double s_of[kKeep], sum = 0.0;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                s_of[i] = 0.0;
                if (i * G + lane < a.topk && pick[i] >= 0) {
                    mine[i] = pick[i];
                    const Raw v = from[mine[i]];
                    z_of[i] = __uint_as_float(BF16 ? unsigned(v) << 16 : unsigned(v));
                    s_of[i] = SIGMOID ? sigmoid64(z_of[i]) : exp_from64(z_of[i], base) * inv;
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
                const int64_t to = r * a.topk + i * G + lane;
                a.choice[to] = mine[i];
                a.weight[to] = w[i];
                a.logit[to] = z_of[i];
            }
        if (lane == 0 && !SIGMOID && a.lse)
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
//   sigmoid: ds/dz = s (1 - s) with 1 - s = sigmoid(-z); softmax: dz_e = scale p_e (g_e - sum p g),
//   g of the chosen, else 0.
// In 64 bits, rounded once; of WHOLE only fp32 results are (65536 x 256, top 8: 27 us, in 32 bits
// 22 us), as bf16's own rounding is 2^16 times those of 32 bits.  Softmax's p are divided by
// their sum over the row, so that what lse lost as a float (2^-24 of it, for every p of the row)
// is not theirs.
template <bool BF16, typename R, int L, bool WHOLE>
__global__ __launch_bounds__(kThreads) void group_grad_kernel(GroupGradArgs a)
{
    constexpr int G = R::G, PER = R::PER, V = R::V, kGroups = kThreads / G;
    constexpr int kKeep = ((L ? L : RR_MAX_ROUTE_TOPK) + G - 1) / G;
    using Real = std::conditional_t<BF16, float, double>;
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
        float term[kKeep];
        int live = 0;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (i * G + lane >= a.topk || unsigned(of.c[i]) >= unsigned(a.experts))
                of.c[i] = -1;
            live |= of.c[i] >= 0;
        }
        // WHOLE: exp(z - lse), and what makes them sum to 1
        Real whole[WHOLE ? PER : 1], dot = 0, inv = 0;
        if constexpr (WHOLE) {
            const float base = of.lse == -INFINITY ? 0.0f : of.lse;
            row.pad(lane, a.experts);
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                whole[s] = exp_from<Real>(row.get(s), base);
                inv += whole[s];
                // a few at a time: side by side they would not fit the registers
                if (!BF16 && s % 2)
                    __builtin_amdgcn_sched_barrier(0);
            }
            const auto add = [](Real x, Real y) { return x + y; };
            inv = across<G>(inv, add);
            inv = inv == 0 ? Real(0) : Real(1) / inv;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                term[i] = of.g[i];
                dot += of.c[i] >= 0 ? exp_from<Real>(of.z[i], base) * Real(of.g[i]) : Real(0);
            }
            dot = across<G>(dot, add) * inv;
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
                const float z = of.z[i];
                s[i] = of.c[i] < 0 ? 0.0 : a.sigmoid ? sigmoid64(z) : exp_from64(z, top);
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
#pragma unroll
            for (int s = 0; s < PER; ++s)
                d[s] = live ? float(Real(a.scale) * (whole[s] * inv) * (Real(d[s]) - dot)) : 0.0f;
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

template <bool SIGMOID, bool BF16, int G, int PER>
hipError_t route(const GroupRouteArgs &a, int lanes, hipStream_t stream)
{
    const dim3 grid(unsigned(a.blocks)), threads(kRouteThreads);
    const bool four = a.experts / a.groups % 4 == 0;
    if (a.topk <= 8 && four)
        group_route_kernel<SIGMOID, BF16, G, PER, 4, 8><<<grid, threads, 0, stream>>>(a, lanes);
    else if (a.topk <= 8)
        group_route_kernel<SIGMOID, BF16, G, PER, 1, 8><<<grid, threads, 0, stream>>>(a, lanes);
    else if (four)
        group_route_kernel<SIGMOID, BF16, G, PER, 4, 0><<<grid, threads, 0, stream>>>(a, lanes);
    else
        group_route_kernel<SIGMOID, BF16, G, PER, 1, 0><<<grid, threads, 0, stream>>>(a, lanes);
    return hipGetLastError();
}

template <bool SIGMOID, bool BF16>
hipError_t route(const GroupRouteArgs &a, hipStream_t stream)
{
    const Layout l = layout_of(a.experts, a.groups);
    if (l.g == 16)
        return l.per <= 4   ? route<SIGMOID, BF16, 16, 4>(a, l.lanes, stream)
               : l.per <= 8 ? route<SIGMOID, BF16, 16, 8>(a, l.lanes, stream)
                            : route<SIGMOID, BF16, 16, 16>(a, l.lanes, stream);
    return l.per <= 8    ? route<SIGMOID, BF16, 64, 8>(a, l.lanes, stream)
           : l.per <= 16 ? route<SIGMOID, BF16, 64, 16>(a, l.lanes, stream)
                         : route<SIGMOID, BF16, 64, 32>(a, l.lanes, stream);
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
    return n <= 4 ? 1 : int32_t(n < 768 ? n : 768);
}

hipError_t launch_group_route(const Op &op, hipStream_t stream)
{
    const GroupRouteArgs a = op.get<GroupRouteArgs>();
    (void)hipGetLastError();
    if (a.sigmoid)
        return a.bf16 ? route<true, true>(a, stream) : route<true, false>(a, stream);
    return a.bf16 ? route<false, true>(a, stream) : route<false, false>(a, stream);
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
