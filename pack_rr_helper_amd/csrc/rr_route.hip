// rr_route.hip -- gfx950 kernels of the router: the topk choice, the weights,
// the experts' counts and probability sums, the balance loss and its gradient.
//
// A row is held by G lanes in registers, PER experts each: 16 lanes up to 256
// experts, so that a wave works on four rows at once and every exchange stays
// within a DPP row, a whole wave above.  The choice takes the largest key topk
// times; a key orders as its logit does and is taken out once chosen.  Per row
// that is about topk * (3 * PER + 12) vector instructions, which is what bounds
// rr_route; rr_route_grad is bound by its bytes.
#include "rr_loss.h"

namespace rr {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;

// Lane exchange within rows of 16: rotation by N.
template <int N>
__device__ __forceinline__ unsigned rotate(unsigned v)
{
    return unsigned(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + N, 0xf, 0xf, false));
}

// f over the G lanes of a row, the result in every lane.  f commutes, and both
// sides of each exchange combine the same two values, so all lanes get the
// same bits.
template <int G, typename F>
__device__ __forceinline__ unsigned across(unsigned v, F f)
{
    v = f(v, rotate<8>(v));
    v = f(v, rotate<4>(v));
    v = f(v, rotate<2>(v));
    v = f(v, rotate<1>(v));
    if constexpr (G == 64) {
        v = f(v, unsigned(__shfl_xor(int(v), 16)));
        v = f(v, unsigned(__shfl_xor(int(v), 32)));
    }
    return v;
}

template <int G>
__device__ __forceinline__ float row_sum(float v)
{
    return __uint_as_float(across<G>(__float_as_uint(v), [](unsigned a, unsigned b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

template <int G>
__device__ __forceinline__ float row_max(float v)
{
    return __uint_as_float(across<G>(__float_as_uint(v), [](unsigned a, unsigned b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

__device__ __forceinline__ float wave_sum(float v)
{
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// Unsigned keys in the order of the floats, NaN on top, above 0.
__device__ __forceinline__ unsigned order_key(float v)
{
    const unsigned u = __float_as_uint(v + 0.0f);  // -0 is 0
    return v != v ? 0xffffffffu : u ^ (unsigned(int(u) >> 31) | 0x80000000u);
}

template <bool BF16>
__device__ __forceinline__ float key_value(unsigned key)
{
    const unsigned u = key & 0x80000000u ? key ^ 0x80000000u : ~key;
    return __uint_as_float(BF16 ? u & 0xffff0000u : u);
}

// exp(x - base).  The product's rounding is |x - base| 2^-24 of the result.
__device__ __forceinline__ float exp_from(float x, float base)
{
    return __builtin_amdgcn_exp2f((x - base) * kLog2e);
}

// -inf - -inf is to count as nothing.
__device__ __forceinline__ float finite_base(float top) { return top == -INFINITY ? 0.0f : top; }

// The part of a row of `experts` elements that one lane holds: PER of them in
// chunks of V, chunk c of lane l at element (c * G + l) * V.  V divides
// `experts`, so a chunk lies in the row or past it.
template <bool BF16, int G_, int PER_, int V_>
struct Row {
    static constexpr int G = G_, PER = PER_, V = V_, kGroups = kThreads / G, kChunks = PER / V;
    static constexpr int kKeep = (RR_MAX_ROUTE_TOPK + G - 1) / G;  // choices of a row per lane
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    struct Chunk {
        Raw v[V];
    };
    Chunk c[kChunks];

    __device__ static int expert(int lane, int s) { return (s / V * G + lane) * V + s % V; }

    __device__ void load(const void *p, int lane, int experts, Raw pad)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                c[i].v[e] = pad;
            const int at = (i * G + lane) * V;
            if (at < experts)
                __builtin_memcpy(&c[i], static_cast<const Raw *>(p) + at, sizeof(Chunk));
        }
    }
    __device__ void store(void *p, int lane, int experts) const
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = (i * G + lane) * V;
            if (at < experts)
                __builtin_memcpy(static_cast<Raw *>(p) + at, &c[i], sizeof(Chunk));
        }
    }
    __device__ float get(int s) const
    {
        if constexpr (BF16)
            return __uint_as_float(unsigned(c[s / V].v[s % V]) << 16);
        else
            return __uint_as_float(c[s / V].v[s % V]);
    }
    __device__ void set(int s, float f)
    {
        if constexpr (BF16)
            c[s / V].v[s % V] = __builtin_bit_cast(unsigned short, (__bf16)f);
        else
            c[s / V].v[s % V] = __float_as_uint(f);
    }
    static constexpr Raw kNothing = BF16 ? Raw(0xff80) : Raw(0xff800000u);  // -inf
};

template <bool BF16, typename R>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a)
{
    constexpr int G = R::G, PER = R::PER;
    __shared__ int count[G * PER + 1];
    __shared__ float sums[kWaves][G * PER];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const int64_t es = BF16 ? 2 : 4, step = int64_t(gridDim.x) * R::kGroups;
    for (int i = threadIdx.x; i <= a.experts; i += kThreads)
        count[i] = 0;
    __syncthreads();
    float sum[PER];
#pragma unroll
    for (int s = 0; s < PER; ++s)
        sum[s] = 0.0f;
    int kept = 0;
    int64_t r = int64_t(blockIdx.x) * R::kGroups + group;
    const char *from = static_cast<const char *>(a.logits) + r * a.experts * es;
    R row;
    bool keep = true;
    if (r < a.rows) {
        row.load(from, lane, a.experts, R::kNothing);
        keep = !a.keep || a.keep[r];
    }
    for (; r < a.rows; r += step) {
        // the next row is on its way while this one is worked on
        R next = row;
        bool next_keep = true;
        from += step * a.experts * es;
        if (r + step < a.rows) {
            next.load(from, lane, a.experts, R::kNothing);
            next_keep = !a.keep || a.keep[r + step];
        }
        int mine[R::kKeep];
        float w[R::kKeep], top = -INFINITY, lse = 0.0f;
#pragma unroll
        for (int i = 0; i < R::kKeep; ++i)
            mine[i] = -1, w[i] = 0.0f;
        if (keep) {
            float z[PER], total = 0.0f;
            unsigned key[PER];
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                z[s] = row.get(s);
                key[s] = order_key(z[s]);
                // bf16 leaves 16 bits free for the index, the lowest on top
                if constexpr (BF16)
                    key[s] = (key[s] & 0xffff0000u) | unsigned(0xffff - R::expert(lane, s));
                if (R::expert(lane, s) >= a.experts)
                    key[s] = 0;
                top = fmaxf(top, z[s]);
            }
            top = row_max<G>(top);
            const float base = finite_base(top);
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                z[s] = exp_from(z[s], base);
                total += z[s];
            }
            total = row_sum<G>(total);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int s = 0; s < PER; ++s)
                sum[s] = __builtin_fmaf(z[s], inv, sum[s]);
            for (int k = 0; k < a.topk; ++k) {
                unsigned best = 0;
                int e = 0;
                if constexpr (BF16) {
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        best = key[s] > best ? key[s] : best;
                    best = across<G>(best, [](unsigned x, unsigned y) { return x > y ? x : y; });
                    e = 0xffff - int(best & 0xffffu);
                } else {
                    // a lane's experts ascend with s: the first of equals is the lowest
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        if (key[s] > best) {
                            best = key[s];
                            e = R::expert(lane, s);
                        }
                    const unsigned own = best;
                    best = across<G>(best, [](unsigned x, unsigned y) { return x > y ? x : y; });
                    e = int(across<G>(own == best ? unsigned(e) : 0xffffu,
                                      [](unsigned x, unsigned y) { return x < y ? x : y; }));
                }
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    key[s] = e == R::expert(lane, s) ? 0 : key[s];
#pragma unroll
                for (int i = 0; i < R::kKeep; ++i)
                    if (k == i * G + lane) {
                        mine[i] = e;
                        w[i] = key_value<BF16>(best);
                    }
            }
            float chosen = 0.0f;
#pragma unroll
            for (int i = 0; i < R::kKeep; ++i) {
                w[i] = i * G + lane < a.topk ? exp_from(w[i], base) : 0.0f;
                chosen += w[i];
            }
            float by = inv;
            if (a.renormalize) {
                chosen = row_sum<G>(chosen);
                by = chosen == 0.0f ? 0.0f : 1.0f / chosen;
            }
#pragma unroll
            for (int i = 0; i < R::kKeep; ++i) {
                w[i] *= by;
                if (mine[i] >= 0)
                    atomicAdd(&count[mine[i]], 1);
            }
            lse = top + logf(total);
            ++kept;
        }
#pragma unroll
        for (int i = 0; i < R::kKeep; ++i)
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
    for (int i = threadIdx.x; i <= a.experts; i += kThreads) {
        if (i < a.experts) {
            float t = 0.0f;
            for (int w = 0; w < kWaves; ++w)
                t += sums[w][i];
            a.prob_sum[int64_t(blockIdx.x) * a.experts + i] = t;
        }
        a.counts[int64_t(blockIdx.x) * (a.experts + 1) + i] = count[i];
    }
}

// Sixteen experts per workgroup, 64 threads for each.
constexpr int kSumThreads = 1024, kSumWide = 16;

__global__ __launch_bounds__(kSumThreads) void route_sum_kernel(RouteSumArgs a)
{
    __shared__ int ns[kSumThreads];
    __shared__ float ss[kSumThreads];
    const int i = blockIdx.x * kSumWide + threadIdx.x % kSumWide, first = threadIdx.x / kSumWide;
    constexpr int kStep = kSumThreads / kSumWide;
    int n = 0;
    float s = 0.0f;
    if (i <= a.experts) {
#pragma unroll 8
        for (int b = first; b < a.blocks; b += kStep) {
            n += a.part_counts[int64_t(b) * (a.experts + 1) + i];
            if (i < a.experts)
                s += a.part_sum[int64_t(b) * a.experts + i];
        }
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

// The chosen experts' own terms lie in LDS, zero at every other expert, and
// are zeroed again once read.
template <bool BF16, typename R>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a)
{
    constexpr int G = R::G, PER = R::PER, V = R::V;
    __shared__ __attribute__((aligned(16))) float chosen_terms[R::kGroups][G * PER];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    float *own = chosen_terms[group];
    const int64_t es = BF16 ? 2 : 4, step = int64_t(gridDim.x) * R::kGroups;
    const float gl = a.grad_loss[0];
    float slope[PER];
#pragma unroll
    for (int s = 0; s < PER; ++s) {
        const int e = R::expert(lane, s);
        slope[s] = e < a.experts ? gl * a.slope[e] : 0.0f;
        own[e] = 0.0f;
    }
    for (int64_t r = int64_t(blockIdx.x) * R::kGroups + group; r < a.rows; r += step) {
        const int64_t at = r * a.experts * es;
        R row;
        row.load(static_cast<const char *>(a.logits) + at, lane, a.experts, R::kNothing);
        const float base = finite_base(a.lse[r]);
        float w[R::kKeep], g[R::kKeep], mean = 0.0f;
        int c[R::kKeep];
#pragma unroll
        for (int i = 0; i < R::kKeep; ++i) {
            const int64_t n = r * a.topk + i * G + lane;
            const bool in = i * G + lane < a.topk;
            c[i] = in ? a.choice[n] : -1;
            w[i] = in && a.renormalize ? a.weight[n] : 0.0f;
            g[i] = in ? a.grad_weight[n] : 0.0f;
            if (c[i] >= a.experts)
                c[i] = -1;
            mean += w[i] * g[i];
        }
        if (!a.keep || a.keep[r]) {
            if (a.renormalize)
                mean = row_sum<G>(mean);
#pragma unroll
            for (int i = 0; i < R::kKeep; ++i)
                if (c[i] >= 0)
                    own[c[i]] = a.renormalize ? w[i] * (g[i] - mean) : g[i];
            // one wave's LDS operations keep their order; so has the compiler to
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            float p[PER], term[PER], dot = 0.0f;
#pragma unroll
            for (int s = 0; s < PER; s += V)
                __builtin_memcpy(&term[s], __builtin_assume_aligned(own + R::expert(lane, s), V % 4 ? 4 * V : 16), 4 * V);
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                p[s] = exp_from(row.get(s), base);
                dot = __builtin_fmaf(p[s], a.renormalize ? slope[s] : slope[s] + term[s], dot);
            }
            dot = row_sum<G>(dot);
#pragma unroll
            for (int s = 0; s < PER; ++s)
                row.set(s, a.renormalize ? __builtin_fmaf(p[s], slope[s] - dot, term[s])
                                         : p[s] * (slope[s] + term[s] - dot));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < R::kKeep; ++i)
                if (c[i] >= 0)
                    own[c[i]] = 0.0f;
        } else {
#pragma unroll
            for (int s = 0; s < PER; ++s)
                row.set(s, 0.0f);
        }
        row.store(static_cast<char *>(a.dlogits) + at, lane, a.experts);
    }
}

// Lanes of a row.
int lanes_of(int experts) { return experts <= 256 ? 16 : 64; }

// f(Row type) for a number of experts: the next power of two per lane, in
// chunks of up to 16 bytes where those divide a row.
template <bool BF16, int G, int PER, typename F>
hipError_t with_chunk(int experts, F f)
{
    constexpr int kMost = BF16 ? 8 : 4, V = PER < kMost ? PER : kMost;
    if (experts % V == 0)
        return f(Row<BF16, G, PER, V>{});
    return f(Row<BF16, G, PER, 1>{});
}

template <bool BF16, typename F>
hipError_t with_row(int experts, F f)
{
    if (lanes_of(experts) == 64)
        return experts <= 512 ? with_chunk<BF16, 64, 8>(experts, f) : with_chunk<BF16, 64, 16>(experts, f);
    if (experts <= 16)
        return with_chunk<BF16, 16, 1>(experts, f);
    if (experts <= 32)
        return with_chunk<BF16, 16, 2>(experts, f);
    if (experts <= 64)
        return with_chunk<BF16, 16, 4>(experts, f);
    if (experts <= 128)
        return with_chunk<BF16, 16, 8>(experts, f);
    return with_chunk<BF16, 16, 16>(experts, f);
}

}  // namespace

int32_t route_blocks(int64_t rows, int32_t experts)
{
    const int64_t groups = kThreads / lanes_of(experts), n = (rows + groups - 1) / groups;
    // up to four rows per group a second launch costs more than it saves
    return n <= 4 ? 1 : int32_t(n < 1024 ? n : 1024);
}

hipError_t launch_route(const Op &op, hipStream_t stream)
{
    const RouteArgs a = op.get<RouteArgs>();
    (void)hipGetLastError();
    const dim3 grid(unsigned(a.blocks)), threads(kThreads);
    if (a.bf16)
        return with_row<true>(a.experts, [&](auto r) {
            route_kernel<true, decltype(r)><<<grid, threads, 0, stream>>>(a);
            return hipGetLastError();
        });
    return with_row<false>(a.experts, [&](auto r) {
        route_kernel<false, decltype(r)><<<grid, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
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
    const int64_t groups = kThreads / lanes_of(a.experts), n = (a.rows + groups - 1) / groups;
    const dim3 grid(unsigned(n < 2048 ? n : 2048)), threads(kThreads);
    (void)hipGetLastError();
    if (a.bf16)
        return with_row<true>(a.experts, [&](auto r) {
            route_grad_kernel<true, decltype(r)><<<grid, threads, 0, stream>>>(a);
            return hipGetLastError();
        });
    return with_row<false>(a.experts, [&](auto r) {
        route_grad_kernel<false, decltype(r)><<<grid, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace rr
