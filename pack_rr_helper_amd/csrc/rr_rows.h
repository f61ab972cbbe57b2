// rr_rows.h -- rows of experts held by the lanes of a wave: loads and stores, and
// the largest keys of a row as lists that are sorted in a lane and merged across
// lanes.  A key type K has T, larger() and smaller().
#pragma once

#include <math.h>

#include <type_traits>

#include "rr_lanes.h"

namespace rr {
namespace {

// Descending order of a sequence that falls and then rises, or the other way.
template <typename K, int N>
__device__ __forceinline__ void sort_bitonic(typename K::T *v)
{
    if constexpr (N > 1) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const auto a = v[i], b = v[i + N / 2];
            v[i] = K::larger(a, b);
            v[i + N / 2] = K::smaller(a, b);
        }
        sort_bitonic<K, N / 2>(v);
        sort_bitonic<K, N / 2>(v + N / 2);
    }
}

// v = the L largest of v (N, falling) and w (N, falling), falling; their count
// is min(2 N, L).
template <typename K, int N, int L>
__device__ __forceinline__ void merge(typename K::T *v, const typename K::T *w)
{
    if constexpr (2 * N <= L) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[N + i] = w[N - 1 - i];
        sort_bitonic<K, 2 * N>(v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = K::larger(v[i], w[N - 1 - i]);
        sort_bitonic<K, N>(v);
    }
}

template <typename K>
__device__ __forceinline__ void order(typename K::T &a, typename K::T &b)
{
    const auto l = K::larger(a, b);
    b = K::smaller(a, b);
    a = l;
}

// Batcher's networks: 1, 5 and 19 exchanges.
template <typename K, int N>
__device__ __forceinline__ void sort(typename K::T *v)
{
    static_assert(N <= 8, "");
    if constexpr (N == 2) {
        order<K>(v[0], v[1]);
    } else if constexpr (N > 2) {
        sort<K, N / 2>(v);
        sort<K, N / 2>(v + N / 2);
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            order<K>(v[i], v[i + N / 2]);
        if constexpr (N == 8) {
            order<K>(v[2], v[4]);
            order<K>(v[3], v[5]);
        }
#pragma unroll
        for (int i = 1; i < N - 1; i += 2)
            order<K>(v[i], v[i + 1]);
    }
}

// The min(N, L) largest of v[N], falling, in out.
template <typename K, int N, int L>
__device__ __forceinline__ void sort_top(const typename K::T *v, typename K::T *out)
{
    if constexpr (N <= L) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            out[i] = v[i];
        sort<K, N>(out);
    } else {
        typename K::T w[L];
        sort_top<K, N / 2, L>(v, out);
        sort_top<K, N / 2, L>(v + N / 2, w);
        merge<K, L, L>(out, w);
    }
}

// The same over the lanes of a row, N values in each.
template <typename K, int G, int N, int L, int STEP = 0>
__device__ __forceinline__ void merge_lanes(typename K::T *v)
{
    if constexpr (1 << STEP < G) {
        typename K::T w[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = other<STEP>(v[i]);
        merge<K, N, L>(v, w);
        merge_lanes<K, G, (2 * N < L ? 2 * N : L), L, STEP + 1>(v);
    }
}

// The part of a row of `experts` elements that one lane holds: PER of them in
// chunks of V, chunk c of lane l at element (c * G + l) * V.  V divides
// `experts`, so a chunk lies in the row or past it and moves as a whole.
template <bool BF16, int G_, int PER_, int V_>
struct Row {
    static constexpr int G = G_, PER = PER_, V = V_, kChunks = PER / V;
    static constexpr int kEs = BF16 ? 2 : 4;
    static constexpr bool kPairs = BF16 && V > 1;    // two elements to a word
    static constexpr int kWords = kPairs ? V / 2 : V;  // of a chunk
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    struct Chunk {
        std::conditional_t<kPairs || !BF16, unsigned, unsigned short> w[kWords];
    };
    unsigned w[kChunks * kWords];

    __device__ static int expert(int lane, int s) { return (s / V * G + lane) * V + s % V; }

    // Elements past the row are anything until pad().
    __device__ void load(const void *p, int lane, int experts)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = (i * G + lane) * V;
            Chunk c;
            __builtin_memcpy(&c, static_cast<const Raw *>(p) + (at < experts ? at : 0), sizeof c);
#pragma unroll
            for (int n = 0; n < kWords; ++n)
                w[i * kWords + n] = c.w[n];
        }
    }
    // -inf past the row
    __device__ void pad(int lane, int experts)
    {
        if (experts < G * PER) {
#pragma unroll
            for (int i = 0; i < kChunks * kWords; ++i)
                w[i] = (i / kWords * G + lane) * V < experts ? w[i] : BF16 ? 0xff80ff80u : 0xff800000u;
        }
    }
    __device__ void store(void *p, int lane, int experts) const
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = (i * G + lane) * V;
            Chunk c;
#pragma unroll
            for (int n = 0; n < kWords; ++n)
                c.w[n] = w[i * kWords + n];
            if (at < experts)
                __builtin_memcpy(static_cast<Raw *>(p) + at, &c, sizeof c);
        }
    }
    __device__ float get(int s) const
    {
        if constexpr (kPairs)
            return __uint_as_float(s % 2 ? w[s / 2] & 0xffff0000u : w[s / 2] << 16);
        else
            return __uint_as_float(BF16 ? w[s] << 16 : w[s]);
    }
    __device__ void set(const float *f)
    {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < kChunks * kWords; ++i)
            if constexpr (kPairs)
                w[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{f[2 * i], f[2 * i + 1]}, bf16x2));
            else if constexpr (BF16)
                w[i] = __builtin_bit_cast(unsigned short, (__bf16)f[i]);
            else
                w[i] = __float_as_uint(f[i]);
    }
};

// Lanes of a row, and f(Row type) for a number of experts.
int lanes_of(int experts) { return experts <= 32 ? 4 : experts <= 64 ? 8 : experts <= 256 ? 16 : 64; }

template <bool BF16, int G, int PER, typename F>
hipError_t with_chunk(int experts, F f)
{
    if constexpr (BF16 && PER >= 8)
        if (experts % 8 == 0)
            return f(Row<BF16, G, PER, 8>{});
    if (experts % 4 == 0)
        return f(Row<BF16, G, PER, 4>{});
    return f(Row<BF16, G, PER, 1>{});
}

template <bool BF16, typename F>
hipError_t with_row(int experts, F f)
{
    if (experts <= 16)
        return with_chunk<BF16, 4, 4>(experts, f);
    if (experts <= 32)
        return with_chunk<BF16, 4, 8>(experts, f);
    if (experts <= 64)
        return with_chunk<BF16, 8, 8>(experts, f);
    if (experts <= 128)
        return with_chunk<BF16, 16, 8>(experts, f);
    if (experts <= 256)
        return with_chunk<BF16, 16, 16>(experts, f);
    if (experts <= 512)
        return with_chunk<BF16, 64, 8>(experts, f);
    return with_chunk<BF16, 64, 16>(experts, f);
}

template <int N> using Int = std::integral_constant<int, N>;

// f(list length) for a number of choices.
template <typename F>
hipError_t with_list(int topk, F f)
{
    return topk <= 2 ? f(Int<2>{}) : topk <= 4 ? f(Int<4>{}) : topk <= 8 ? f(Int<8>{}) : f(Int<0>{});
}

}  // namespace
}  // namespace rr
