// rr_clip.hip -- gfx950 kernels of the global gradient norm: the sum of squares of
// many tensors, and their scaling.  Bound by their bytes.
//
// The tensors of a launch stand in its arguments.  They are cut into tiles, one for
// each workgroup: 2048 workgroups that took their tiles in turn had the sum at 4.6 TB/s
// and the scaling at 4.8 TB/s (600 million elements in bf16).  Squares are summed in 64 bits, which cost what 32 would on this
// card: no finite gradient overflows, and a long sum loses nothing.
#include "rr_expert.h"
#include "rr_lanes.h"

namespace rr {
namespace {

constexpr int kThreads = 256;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// The elements of 16 bytes at any element alignment.
template <bool BF16>
struct Vector {
    static constexpr int N = BF16 ? 8 : 4;
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    u32x4 w;

    typedef u32x4 Free __attribute__((aligned(2)));  // at any element
    // STREAM: not to be kept in the caches
    template <bool STREAM>
    __device__ void load(const Raw *p)
    {
        if constexpr (STREAM)
            w = __builtin_nontemporal_load(reinterpret_cast<const Free *>(p));
        else
            w = *reinterpret_cast<const Free *>(p);
    }
    // what leaves is not read again
    __device__ void store(Raw *p) const { __builtin_nontemporal_store(w, reinterpret_cast<Free *>(p)); }
    // `left` elements of them, zeros past those
    __device__ void load(const Raw *p, int64_t left)
    {
        w = u32x4{0, 0, 0, 0};
        if (left >= N) {
            load<false>(p);
        } else {
#pragma unroll
            for (int i = 0; i < N - 1; ++i)
                if (i < left)
                    w[BF16 ? i / 2 : i] |= unsigned(p[i]) << (BF16 ? i % 2 * 16 : 0);
        }
    }
    __device__ void store(Raw *p, int64_t left) const
    {
        if (left >= N) {
            store(p);
        } else {
#pragma unroll
            for (int i = 0; i < N - 1; ++i)
                if (i < left)
                    p[i] = Raw(w[BF16 ? i / 2 : i] >> (BF16 ? i % 2 * 16 : 0));
        }
    }
    __device__ float get(int i) const
    {
        if constexpr (BF16)
            return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else
            return __uint_as_float(w[i]);
    }
    __device__ void scale(float by)
    {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16)
                w[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{get(2 * i) * by, get(2 * i + 1) * by}, bf16x2));
            else
                w[i] = __float_as_uint(get(i) * by);
        }
    }
};

// A tile's vectors of a thread.  A whole tile is loaded without conditions: a load
// under one is waited for where that ends.
template <int THREADS, int VECTORS, bool STREAM, bool BF16>
__device__ __forceinline__ bool load_tile(const void *from, int64_t count, int64_t first, Vector<BF16> *v)
{
    const int thread = int(threadIdx.x) % THREADS;
    using V = Vector<BF16>;
    const auto *in = static_cast<const typename V::Raw *>(from) + first;
    const bool whole = count - first >= THREADS * VECTORS * V::N;
    if (whole) {
#pragma unroll
        for (int i = 0; i < VECTORS; ++i)
            v[i].template load<STREAM>(in + (i * THREADS + thread) * V::N);
    } else {
#pragma unroll
        for (int i = 0; i < VECTORS; ++i) {
            const int at = (i * THREADS + thread) * V::N;
            v[i].load(in + at, count - first - at);
        }
    }
    return whole;
}

// The tensor of a tile, and the tile's first element there.
template <bool BF16, int VECTORS>
__device__ __forceinline__ int tensor_of(const ClipTable &t, int tile, int64_t &first)
{
    // the last with at most as many tiles before it
    int i = -1;
#pragma unroll
    for (int i0 = 0; i0 < kClipTensors; i0 += 64) {
        const int n = i0 + int(threadIdx.x % 64);
        i += __popcll(__ballot(n < t.tensors && t.tile0[n < kClipTensors ? n : 0] <= tile));
    }
    i = __builtin_amdgcn_readfirstlane(i);
    first = i < 0 ? 0 : int64_t(tile - t.tile0[i]) * (kThreads * VECTORS * (BF16 ? 8 : 4));
    return i;
}

template <bool BF16, int VECTORS>
__device__ __forceinline__ double squares(const Vector<BF16> *v)
{
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < VECTORS; ++n)
#pragma unroll
        for (int e = 0; e < Vector<BF16>::N; ++e)
            sum = __builtin_fma(double(v[n].get(e)), double(v[n].get(e)), sum);
    return sum;
}

// The workgroup's sum, in its first thread.
template <int WAVES>
__device__ __forceinline__ double sum_of_waves(double sum)
{
    __shared__ double sums[WAVES];
    sum = across<64>(sum, [](double x, double y) { return x + y; });
    if (threadIdx.x % 64 == 0)
        sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < WAVES; ++w)
            sum += sums[w];
    return sum;
}

template <bool BF16, bool STREAM>
__global__ __launch_bounds__(kThreads) void square_sum_kernel(SquareSumArgs a)
{
    double sum = 0.0;
    int64_t first;
    const int i = tensor_of<BF16, kSquareVectors>(a.t, int(blockIdx.x), first);
    if (i >= 0) {
        Vector<BF16> v[kSquareVectors];
        load_tile<kThreads, kSquareVectors, STREAM>(a.t.in[i], a.t.count[i], first, v);
        sum = squares<BF16, kSquareVectors>(v);
    }
    sum = sum_of_waves<kThreads / 64>(sum);
    if (threadIdx.x == 0)
        a.part[blockIdx.x] = sum;
}

// One workgroup, a tile a wave at a time.
constexpr int kSmallThreads = 1024;

template <bool BF16>
__global__ __launch_bounds__(kSmallThreads) void square_small_kernel(SquareSumArgs a)
{
    constexpr int kWide = kSmallVectors * kThreads / 64;  // vectors of a lane
    double sum = 0.0;
    for (int tile = threadIdx.x / 64; tile < a.t.tiles; tile += kSmallThreads / 64) {
        int64_t first;
        const int i = tensor_of<BF16, kSmallVectors>(a.t, __builtin_amdgcn_readfirstlane(tile), first);
        Vector<BF16> v[kWide];
        load_tile<64, kWide, false>(a.t.in[i], a.t.count[i], first, v);
        sum += squares<BF16, kWide>(v);
    }
    sum = sum_of_waves<kSmallThreads / 64>(sum);
    if (threadIdx.x == 0)
        a.part[0] = sum;
}

constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void sum_parts_kernel(SumPartsArgs a)
{
    // eight loads at a time under way
    double each[8] = {};
    for (int i0 = 0; i0 < a.parts; i0 += 8 * kSumThreads)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int i = i0 + n * kSumThreads + int(threadIdx.x);
            const double v = a.part[i < a.parts ? i : 0];
            each[n] += i < a.parts ? v : 0.0;
        }
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < 8; ++n)
        sum += each[n];
    sum = sum_of_waves<kSumThreads / 64>(sum);
    if (threadIdx.x == 0)
        a.sum[0] = sum;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void clip_kernel(ClipArgs a)
{
    using V = Vector<BF16>;
    constexpr int VECTORS = kClipVectors;
    double sum = 0.0;
    for (int i = 0; i < a.n_sums; ++i)
        sum += a.sums[i][0];
    const double norm = sqrt(sum);
    const float by = norm > a.max_norm && norm < INFINITY ? float(a.max_norm / norm) : 1.0f;
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0)
        a.norm[0] = float(norm);
    int64_t first;
    const int i = tensor_of<BF16, VECTORS>(a.t, int(blockIdx.x), first);
    if (i < 0 || (by == 1.0f && a.t.in[i] == a.t.out[i]))
        return;
    const int64_t left = a.t.count[i] - first;
    auto *out = static_cast<typename V::Raw *>(a.t.out[i]) + first;
    V v[VECTORS];
    const bool whole = load_tile<kThreads, VECTORS, true>(a.t.in[i], a.t.count[i], first, v);
#pragma unroll
    for (int n = 0; n < VECTORS; ++n)
        v[n].scale(by);
    if (whole) {
#pragma unroll
        for (int n = 0; n < VECTORS; ++n)
            v[n].store(out + (n * kThreads + int(threadIdx.x)) * V::N);
    } else {
#pragma unroll
        for (int n = 0; n < VECTORS; ++n) {
            const int at = (n * kThreads + int(threadIdx.x)) * V::N;
            v[n].store(out + at, left - at);
        }
    }
}

}  // namespace

int64_t ClipTable::add(const void *from, void *to, int64_t n)
{
    const int64_t per = int64_t(kThreads) * vectors * (bf16 ? 8 : 4), room = (kClipTiles - tiles) * per;
    n = n < room ? n : room;
    if (n == 0 || tensors == kClipTensors)
        return 0;
    tile0[tensors] = tiles;
    in[tensors] = from;
    out[tensors] = to;
    count[tensors++] = n;
    tiles += int32_t((n + per - 1) / per);
    return n;
}

hipError_t launch_square_sum(const Op &op, hipStream_t stream)
{
    const SquareSumArgs a = op.get<SquareSumArgs>();
    const dim3 grid(unsigned(a.t.blocks())), threads(kThreads);
    (void)hipGetLastError();
    if (a.t.bf16 && a.stream)
        square_sum_kernel<true, true><<<grid, threads, 0, stream>>>(a);
    else if (a.t.bf16)
        square_sum_kernel<true, false><<<grid, threads, 0, stream>>>(a);
    else if (a.stream)
        square_sum_kernel<false, true><<<grid, threads, 0, stream>>>(a);
    else
        square_sum_kernel<false, false><<<grid, threads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_square_small(const Op &op, hipStream_t stream)
{
    const SquareSumArgs a = op.get<SquareSumArgs>();
    (void)hipGetLastError();
    if (a.t.bf16)
        square_small_kernel<true><<<dim3(1), dim3(kSmallThreads), 0, stream>>>(a);
    else
        square_small_kernel<false><<<dim3(1), dim3(kSmallThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_sum_parts(const Op &op, hipStream_t stream)
{
    const SumPartsArgs a = op.get<SumPartsArgs>();
    (void)hipGetLastError();
    sum_parts_kernel<<<dim3(1), dim3(kSumThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_clip(const Op &op, hipStream_t stream)
{
    const ClipArgs a = op.get<ClipArgs>();
    (void)hipGetLastError();
    if (a.t.bf16)
        clip_kernel<true><<<dim3(unsigned(a.t.blocks())), dim3(kThreads), 0, stream>>>(a);
    else
        clip_kernel<false><<<dim3(unsigned(a.t.blocks())), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace rr
