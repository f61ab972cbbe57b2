// rr_clip.hip -- gfx950 kernels of the global gradient norm: the sum of squares of
// many tensors, and their scaling.  Bound by their bytes.
//
// The tensors of a launch stand in its arguments.  They are cut into tiles, and a
// workgroup takes a contiguous range of all tiles, so that it looks for its first
// tensor once.  Squares are summed in 64 bits, which cost what 32 would on this
// card: no finite gradient overflows, and a long sum loses nothing.
#include "rr_expert.h"
#include "rr_lanes.h"

namespace rr {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 8;                                // of a thread in a tile
constexpr int kTileBytes = kThreads * kVectors * 16;

__host__ __device__ inline int64_t tiles_of(int64_t count, int64_t es) { return (count * es + kTileBytes - 1) / kTileBytes; }

// The elements of 16 bytes at any element alignment, `left` elements of them, zeros
// past those.
template <bool BF16>
struct Vector {
    static constexpr int N = BF16 ? 8 : 4;
    using Raw = std::conditional_t<BF16, unsigned short, unsigned>;
    Raw v[N];

    __device__ void load(const Raw *p, int64_t left)
    {
        if (left >= N) {
            __builtin_memcpy(v, p, 16);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = i < left ? p[i] : Raw(0);
        }
    }
    __device__ void store(Raw *p, int64_t left) const
    {
        if (left >= N) {
            __builtin_memcpy(p, v, 16);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < left)
                    p[i] = v[i];
        }
    }
    __device__ float get(int i) const { return __uint_as_float(BF16 ? unsigned(v[i]) << 16 : unsigned(v[i])); }
    __device__ void scale(float by)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (BF16)
                v[i] = __builtin_bit_cast(unsigned short, (__bf16)(get(i) * by));
            else
                v[i] = __float_as_uint(get(i) * by);
        }
    }
};

// f(tensor, first element) for the tiles of workgroup b of `blocks`.
template <bool BF16, typename F>
__device__ __forceinline__ void each_tile(const ClipTensor *t, int tensors, int b, int blocks, F f)
{
    constexpr int64_t es = BF16 ? 2 : 4;
    int64_t all = 0;
    for (int i = 0; i < tensors; ++i)
        all += tiles_of(t[i].count, es);
    int64_t at = all * b / blocks, end = all * (b + 1) / blocks;
    for (int i = 0; i < tensors && end > 0; ++i) {
        const int64_t n = tiles_of(t[i].count, es);
        for (; at < n && at < end; ++at)
            f(t[i], at * (kTileBytes / es));
        at = at > n ? at - n : 0;
        end -= n;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void square_sum_kernel(SquareSumArgs a)
{
    using V = Vector<BF16>;
    __shared__ double sums[kThreads / 64];
    double sum = 0.0;
    each_tile<BF16>(a.t, a.tensors, int(blockIdx.x), a.blocks, [&](const ClipTensor &t, int64_t first) {
        const auto *in = static_cast<const typename V::Raw *>(t.in);
        V v[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int64_t at = first + (i * kThreads + int(threadIdx.x)) * V::N;
            v[i].load(in + at, t.count - at);
        }
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
            for (int n = 0; n < V::N; ++n)
                sum = __builtin_fma(double(v[i].get(n)), double(v[i].get(n)), sum);
    });
    sum = across<64>(sum, [](double x, double y) { return x + y; });
    if (threadIdx.x % 64 == 0)
        sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; ++w)
            sum += sums[w];
        a.part[blockIdx.x] = sum;
    }
}

constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void sum_parts_kernel(SumPartsArgs a)
{
    __shared__ double sums[kSumThreads / 64];
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += kSumThreads)
        sum += a.part[i];
    sum = across<64>(sum, [](double x, double y) { return x + y; });
    if (threadIdx.x % 64 == 0)
        sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kSumThreads / 64; ++w)
            sum += sums[w];
        a.sum[0] = sum;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void clip_kernel(ClipArgs a)
{
    using V = Vector<BF16>;
    double sum = 0.0;
    for (int i = 0; i < a.n_sums; ++i)
        sum += a.sums[i][0];
    const double norm = sqrt(sum);
    const float by = norm > a.max_norm && norm < INFINITY ? float(a.max_norm / norm) : 1.0f;
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0)
        a.norm[0] = float(norm);
    each_tile<BF16>(a.t, a.tensors, int(blockIdx.x), a.blocks, [&](const ClipTensor &t, int64_t first) {
        if (by == 1.0f && t.in == t.out)
            return;
        const auto *in = static_cast<const typename V::Raw *>(t.in);
        auto *out = static_cast<typename V::Raw *>(t.out);
        V v[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int64_t at = first + (i * kThreads + int(threadIdx.x)) * V::N;
            v[i].load(in + at, t.count - at);
        }
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int64_t at = first + (i * kThreads + int(threadIdx.x)) * V::N;
            v[i].scale(by);
            v[i].store(out + at, t.count - at);
        }
    });
}

}  // namespace

int32_t square_blocks(const int64_t *count, int32_t tensors, int64_t es)
{
    int64_t n = 0;
    for (int32_t i = 0; i < tensors; ++i)
        n += tiles_of(count[i], es);
    return int32_t(n < 1 ? 1 : n < 2048 ? n : 2048);
}

hipError_t launch_square_sum(const Op &op, hipStream_t stream)
{
    const SquareSumArgs a = op.get<SquareSumArgs>();
    (void)hipGetLastError();
    if (a.bf16)
        square_sum_kernel<true><<<dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a);
    else
        square_sum_kernel<false><<<dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a);
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
    if (a.bf16)
        clip_kernel<true><<<dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a);
    else
        clip_kernel<false><<<dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace rr
