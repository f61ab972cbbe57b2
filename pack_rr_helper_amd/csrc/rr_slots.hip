// rr_slots.hip -- gfx950 kernels around the experts' products: the slot map of the
// choices, the matrices in 8 bits, the weighted sum back to rows and its gradient.
// All but the slot map are bound by their bytes.
#include "rr_expert.h"
#include "rr_lanes.h"

namespace rr {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Slots: a counting sort that keeps the order of the choices.  A workgroup has a
// piece of the choices, each of its waves a contiguous part of that, 64 at a time:
// a choice's place is its segment's start, the choices of the same expert in
// earlier pieces, in earlier waves, before this 64 and in lower lanes.
// ---------------------------------------------------------------------------

constexpr int kSlotThreads = 1024;
// Choices that one workgroup places alone, which takes one launch (3200 choices 5.1 us, by
// two 6.9 us; 8000 choices 10.1 us, by eight 6.7 us), and else a workgroup's at the least (16384
// choices 6.9 us, with 2048 each 7.9 us).
constexpr int kOnePiece = 4096, kPiece = 1024;

__host__ __device__ inline int piece_of(int choices, int blocks)
{
    const int64_t per = (int64_t(choices) + blocks - 1) / blocks;
    return int((per + kSlotThreads - 1) / kSlotThreads * kSlotThreads);
}

__global__ __launch_bounds__(kThreads) void slots_count_kernel(SlotsArgs a)
{
    __shared__ int n[RR_MAX_EXPERTS];
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        n[e] = 0;
    __syncthreads();
    const int piece = piece_of(a.choices, a.blocks);
    const int64_t lo = int64_t(blockIdx.x) * piece, hi = lo + piece < a.choices ? lo + piece : a.choices;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const unsigned e = unsigned(a.choice[i]) - unsigned(a.first);
        if (e < unsigned(a.experts))
            atomicAdd(&n[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        a.part[int64_t(blockIdx.x) * a.experts + e] = n[e];
}

__global__ __launch_bounds__(kSlotThreads) void slots_kernel(SlotsArgs a)
{
    constexpr int kWaves = kSlotThreads / 64;
    __shared__ int cursor[kWaves][RR_MAX_EXPERTS];
    __shared__ int all[RR_MAX_EXPERTS], start[RR_MAX_EXPERTS + 1], earlier[RR_MAX_EXPERTS];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int piece = piece_of(a.choices, a.blocks), per = piece / kWaves;  // a multiple of 64
    for (int e = lane; e < a.experts; e += 64)
        cursor[wave][e] = 0;
    __syncthreads();
    const int64_t lo = int64_t(blockIdx.x) * piece + int64_t(wave) * per;
    const int64_t hi = lo + per < a.choices ? lo + per : a.choices;
    for (int64_t i = lo + lane; i < hi; i += 64) {
        const unsigned e = unsigned(a.choice[i]) - unsigned(a.first);
        if (e < unsigned(a.experts))
            atomicAdd(&cursor[wave][e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) {
        int here = 0, total = 0, before = 0;
        for (int w = 0; w < kWaves; ++w)
            here += cursor[w][e];
        if (a.blocks > 1) {
#pragma unroll 8
            for (int b = 0; b < a.blocks; ++b) {
                const int n = a.part[int64_t(b) * a.experts + e];
                total += n;
                before += b < int(blockIdx.x) ? n : 0;
            }
        } else {
            total = here;
        }
        all[e] = total;
        earlier[e] = before;
    }
    __syncthreads();
    if (wave == 0) {
        int base = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int n = e0 + lane < a.experts ? (all[e0 + lane] + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK * RR_QUANT_BLOCK : 0;
            int sum = n;
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(sum, d);
                sum += lane >= d ? o : 0;
            }
            if (e0 + lane < a.experts)
                start[e0 + lane] = base + sum - n;
            base += __shfl(sum, 63);
        }
        if (lane == 0)
            start[a.experts] = base;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) {
        int at = start[e] + earlier[e];
        for (int w = 0; w < kWaves; ++w) {
            const int n = cursor[w][e];
            cursor[w][e] = at;
            at += n;
        }
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.experts; e += kSlotThreads) {
            a.offset[e] = start[e];
            if (e < a.experts)
                a.count[e] = all[e];
        }
    // what no choice takes: the segments' ends, and the positions behind the last
    for (int e = int(blockIdx.x) * kWaves + wave; e < a.experts; e += a.blocks * kWaves)
        for (int p = start[e] + all[e] + lane; p < start[e + 1]; p += 64)
            a.source[p] = -1;
    for (int64_t p = start[a.experts] + int64_t(blockIdx.x) * kSlotThreads + threadIdx.x; p < a.capacity;
         p += int64_t(a.blocks) * kSlotThreads)
        a.source[p] = -1;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int64_t i = i0 + lane;
        const unsigned e = i < hi ? unsigned(a.choice[i]) - unsigned(a.first) : ~0u;
        const bool own = e < unsigned(a.experts);
        unsigned long long same = __ballot(own);
        for (int bit = 1; bit < a.experts; bit *= 2) {
            const unsigned long long set = __ballot(own && (e & bit));
            same &= (e & bit) ? set : ~set;
        }
        int p = -1;
        if (own) {
            p = cursor[wave][e] + __popcll(same & ((1ull << lane) - 1));
            a.source[p] = int(i);
        }
        // one wave's LDS operations keep their order; so has the compiler to
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (own && (same >> lane) == 1)  // the highest lane of its expert
            cursor[wave][e] = p + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (i < hi)
            a.slot[i] = p;
    }
}

// ---------------------------------------------------------------------------
// Eight bits
// ---------------------------------------------------------------------------

constexpr unsigned kNotFinite = 0x7f800000u;

// The byte of the power for a block whose largest magnitude has these bits: the
// least 2^e with it <= 448 * 2^e = 1.75 * 2^(e + 8), e >= -127; 255 for a block that is not
// finite.
__device__ __forceinline__ unsigned power_byte(unsigned largest)
{
    if (largest >= kNotFinite)
        return 255;
    const int b = int(largest >> 23) - 8 + ((largest & 0x7fffffu) > 0x600000u);
    return b > 0 ? unsigned(b) : 0;
}

// What a block's elements are multiplied by; its bits are those of 2^(127 - byte).
__device__ __forceinline__ float inverse_power(unsigned byte) { return __uint_as_float((254u - byte) << 23); }

// Four elements to e4m3.
__device__ __forceinline__ unsigned eight_bits(const float *v, unsigned byte)
{
    const float by = inverse_power(byte);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * by, v[1] * by, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * by, v[3] * by, w, true);
    return byte == 255 ? 0x7f7f7f7fu : unsigned(w);
}

__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// What is read where a matrix has not as many bytes.
__device__ const u32x4 kNothing = {0, 0, 0, 0};

// 4, 8 or 16 bytes at any element.
template <int BYTES>
struct Words {
    typedef unsigned T __attribute__((ext_vector_type(BYTES / 4)));
    typedef T Unaligned __attribute__((aligned(2)));
};

// A matrix of rows of `dim` elements, read by COLS side by side: fetch() loads, under no
// condition, as a load under one is waited for where that ends; take() gives the elements,
// zeros past the row.  WHOLE: rows start at, and are, multiples of 16 bytes.  Others are
// loaded at any element, from the matrix' last bytes at most; what those do not hold,
// then loaded one by one, is its last row's end (3300 x 2211 fp32 elements summed to rows:
// 14 us; by elements 61 us).
template <bool BF16, bool WHOLE, int COLS = 8>
struct Matrix {
    static constexpr int kSize = BF16 ? 2 : 4, N = COLS * kSize > 16 ? 16 / kSize : COLS, kLoads = COLS / N;
    using Element = std::conditional_t<BF16, unsigned short, unsigned>;
    using W = Words<N * kSize>;
    struct Raw {
        typename W::T w[kLoads];
    };
    const Element *x;
    int64_t total;       // elements
    int dim;

    __device__ Matrix(const void *p, int64_t rows, int dim) : x(static_cast<const Element *>(p)), total(rows * dim), dim(dim) {}

    // The element that load n from column `at` of row r starts at; the row's first for one past
    // the row.
    __device__ int64_t first(int64_t r, int at, int n) const { return r * dim + (at + n * N < dim ? at + n * N : 0); }
    // STREAM: not to be kept in the caches
    template <bool STREAM = false>
    __device__ void fetch(int64_t r, int at, Raw &raw) const
    {
        using P = std::conditional_t<WHOLE, typename W::T, typename W::Unaligned>;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int64_t e = first(r, at, n);
            const auto *p = reinterpret_cast<const P *>(WHOLE ? x + e
                                                        : total < N ? reinterpret_cast<const Element *>(&kNothing)
                                                                    : x + (e < total - N ? e : total - N));
            raw.w[n] = STREAM ? __builtin_nontemporal_load(p) : *p;
        }
    }
    __device__ void take(int64_t r, int at, const Raw &raw, float *v) const
    {
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            // a whole row ends where a load does
            const int left = WHOLE ? (at + n * N < dim ? N : 0) : dim - at - n * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const unsigned w = raw.w[n][i * kSize / 4], u = !BF16 ? w : i % 2 ? w & 0xffff0000u : w << 16;
                v[n * N + i] = __uint_as_float(i < left ? u : 0);
            }
            if constexpr (!WHOLE) {
                const int64_t e = first(r, at, n);
                if (left > 0 && e > total - N)
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        v[n * N + i] = __uint_as_float(i < left ? unsigned(x[e + i]) << (BF16 ? 16 : 0) : 0);
            }
        }
    }
};

// A block of a row by sixteen lanes.
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantizeRowsArgs a, int blocks)
{
    using M = Matrix<BF16, WHOLE>;
    const M x(a.x, a.rows, a.dim);
    const int lane = threadIdx.x % 16;
    const int64_t n = a.rows * blocks;
    for (int64_t i = int64_t(blockIdx.x) * (kThreads / 16) + threadIdx.x / 16; i < n; i += int64_t(gridDim.x) * (kThreads / 16)) {
        const int64_t r = i / blocks;
        const int b = int(i - r * blocks), at = b * RR_QUANT_BLOCK + lane * 8;
        float v[8];
        typename M::Raw raw;
        x.fetch(r, at, raw);
        x.take(r, at, raw, v);
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, magnitude(v[e]));
        const unsigned byte = power_byte(across<16>(top, [](unsigned x, unsigned y) { return x > y ? x : y; }));
        const uint2 q{eight_bits(v, byte), eight_bits(v + 4, byte)};
        *reinterpret_cast<uint2 *>(a.to.values + r * a.to.ld + at) = q;
        if (lane == 0)
            a.to.powers[r * a.to.lds + b] = (unsigned char)byte;
    }
}

// A tile of 128 x 128 elements: sixteen lanes a row, a thread has rows
// [8 (t / 16), + 8) and eight columns.  Transposed, its eight rows are eight bytes
// of a column, which go through LDS at places exchanged by the column's lane.
struct Turned {
    unsigned char t[RR_QUANT_BLOCK * RR_QUANT_BLOCK];

    __device__ uint2 *at(int column, int part) { return reinterpret_cast<uint2 *>(t + column * RR_QUANT_BLOCK + ((part ^ (column / 8)) & 15) * 8); }
};

// The transposed tile from LDS to rows [0, rows) of out.  STREAM: past the caches.
template <bool STREAM>
__device__ __forceinline__ void store_turned(Turned &t, unsigned char *out, int64_t ld, int rows)
{
    using W = Words<8>::T;
    for (int i = threadIdx.x; i < RR_QUANT_BLOCK * 16; i += kThreads)
        if (i / 16 < rows) {
            const W v = __builtin_bit_cast(W, *t.at(i / 16, i % 16));
            W *to = reinterpret_cast<W *>(out + i / 16 * ld + i % 16 * 8);
            if constexpr (STREAM)
                __builtin_nontemporal_store(v, to);
            else
                *to = v;
        }
}

// STREAM: more than the last level cache holds.  What is transposed then leaves past the
// caches, and w comes past them (32 experts of 4096 x 2048 in bf16 in a training step: 170 us,
// 6.3 TB/s, and 200 us with none of it past them.  Alone, and of zeros: 146 us and 207 us, the
// loads alone past them 208 us, the other stores too 193 us).  What the cache holds is read from
// it by the next product.
template <bool BF16, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(QuantizeWeightArgs a, int blocks_n, int blocks_k)
{
    __shared__ __attribute__((aligned(16))) Turned turned;
    __shared__ unsigned largest;
    const int lane = threadIdx.x % 16, part = threadIdx.x / 16;
    const int bk = blockIdx.x % blocks_k, bn = blockIdx.x / blocks_k % blocks_n, e = blockIdx.x / blocks_k / blocks_n;
    const int n0 = bn * RR_QUANT_BLOCK, k0 = bk * RR_QUANT_BLOCK;
    if (threadIdx.x == 0)
        largest = 0;
    __syncthreads();
    using M = Matrix<BF16, WHOLE>;
    const M matrix(a.w, int64_t(a.experts) * a.n, a.k);
    const auto row_of = [&](int i) { return int64_t(e) * a.n + (n0 + part * 8 + i < a.n ? n0 + part * 8 + i : 0); };
    float v[8][8];
    typename M::Raw w[8];
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        matrix.template fetch<STREAM>(row_of(i), k0 + lane * 8, w[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        matrix.take(row_of(i), k0 + lane * 8, w[i], v[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            v[i][c] = n0 + part * 8 + i < a.n ? v[i][c] : 0.0f;
            top = max(top, magnitude(v[i][c]));
        }
    }
    top = across<64>(top, [](unsigned x, unsigned y) { return x > y ? x : y; });
    if (threadIdx.x % 64 == 0)
        atomicMax(&largest, top);
    __syncthreads();
    const unsigned byte = power_byte(largest);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = n0 + part * 8 + i;
        if (row < a.n)
            *reinterpret_cast<uint2 *>(a.to.values + (int64_t(e) * a.n + row) * a.to.ld + k0 + lane * 8) =
                uint2{eight_bits(v[i], byte), eight_bits(v[i] + 4, byte)};
    }
    if (threadIdx.x == 0) {
        a.to.powers[(int64_t(e) * blocks_n + bn) * a.to.lds + bk] = (unsigned char)byte;
        if (a.turned.values)
            a.turned.powers[(int64_t(e) * blocks_k + bk) * a.turned.lds + bn] = (unsigned char)byte;
    }
    if (!a.turned.values)
        return;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float col[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            col[i] = v[i][c];
        *turned.at(lane * 8 + c, part) = uint2{eight_bits(col, byte), eight_bits(col + 4, byte)};
    }
    __syncthreads();
    store_turned<STREAM>(turned, a.turned.values + (int64_t(e) * a.k + k0) * a.turned.ld + n0, a.turned.ld, a.k - k0);
}

// The stores past the caches, as above, gain nothing inside a layer (65536 positions x 4096: 145
// us both ways) and cost the next product what the cache would have held (16384 choices of 16
// experts, 2048 x 1408: forward and backward 437 us instead of 423 us).
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_slots_kernel(QuantizeSlotsArgs a, int blocks_d)
{
    __shared__ __attribute__((aligned(16))) Turned turned;
    __shared__ unsigned largest[RR_QUANT_BLOCK];
    const int lane = threadIdx.x % 16, part = threadIdx.x / 16;
    const int bd = blockIdx.x % blocks_d, bp = a.block0 + blockIdx.x / blocks_d;
    const int p0 = bp * RR_QUANT_BLOCK, d0 = bd * RR_QUANT_BLOCK;
    if (p0 >= a.offset[a.experts])
        return;
    for (int i = threadIdx.x; i < RR_QUANT_BLOCK; i += kThreads)
        largest[i] = 0;
    __syncthreads();
    using M = Matrix<BF16, WHOLE>;
    const M x(a.x, a.gather ? a.rows : a.capacity, a.dim);
    float v[8][8], by[8];
    typename M::Raw w[8];
    int row[8];
    bool in[8];
    unsigned top[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int p = p0 + part * 8 + i, n = a.source[p];
        const int of = n < 0 ? -1 : int((__umulhi(a.topk_mul, unsigned(n)) + unsigned(n)) >> a.topk_shift);
        in[i] = of >= 0 && of < a.rows;
        row[i] = !in[i] ? 0 : a.gather ? of : p;
        x.fetch(row[i], d0 + lane * 8, w[i]);
        by[i] = a.weight ? a.weight[in[i] ? n : 0] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x.take(row[i], d0 + lane * 8, w[i], v[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            v[i][c] = in[i] ? v[i][c] * by[i] : 0.0f;
            top[c] = max(top[c], magnitude(v[i][c]));
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        atomicMax(&largest[lane * 8 + c], top[c]);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const unsigned byte = power_byte(largest[lane * 8 + c]);
        float col[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            col[i] = v[i][c];
        *turned.at(lane * 8 + c, part) = uint2{eight_bits(col, byte), eight_bits(col + 4, byte)};
    }
    for (int i = threadIdx.x; i < RR_QUANT_BLOCK && d0 + i < a.dim; i += kThreads)
        a.to.powers[int64_t(d0 + i) * a.to.lds + bp] = (unsigned char)power_byte(largest[i]);
    __syncthreads();
    store_turned<false>(turned, a.to.values + int64_t(d0) * a.to.ld + p0, a.to.ld, a.dim - d0);
}

// ---------------------------------------------------------------------------
// Rows of sums
// ---------------------------------------------------------------------------

// COLS elements to column `at` of a row of `dim` that starts at element `first` of y, past
// the caches.
template <bool BF16, bool WHOLE, int COLS>
__device__ __forceinline__ void store_row(void *y, int64_t first, int at, int dim, const float *v)
{
    using M = Matrix<BF16, WHOLE, COLS>;
    using P = std::conditional_t<WHOLE, typename M::W::T, typename M::W::Unaligned>;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    auto *row = static_cast<typename M::Element *>(y) + first + at;
#pragma unroll
    for (int n = 0; n < M::kLoads; ++n) {
        const float *of = v + n * M::N;
        typename M::W::T w;
#pragma unroll
        for (int i = 0; i < M::N * M::kSize / 4; ++i)
            w[i] = BF16 ? __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{of[2 * i % M::N], of[(2 * i + 1) % M::N]}, bf16x2))
                        : __float_as_uint(of[i]);
        const int left = dim - at - n * M::N;
        if (left >= M::N) {
            __builtin_nontemporal_store(w, reinterpret_cast<P *>(row + n * M::N));
        } else if (!WHOLE) {
#pragma unroll
            for (int i = 0; i < M::N - 1; ++i)
                if (i < left)
                    row[n * M::N + i] = typename M::Element(w[i * M::kSize / 4] >> (BF16 ? i % 2 * 16 : 0));
        }
    }
}

// Choices whose rows are on their way at a time.
constexpr int kWide = 8;

// The positions of a row's choices from k0 on, -1 for none, and elements of each on their
// way.
template <typename M>
__device__ __forceinline__ void fetch_slots(const M &values, const int32_t *slot, int k0, int topk, int capacity, int at,
                                            int *p, typename M::Raw *w)
{
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
        p[k] = slot[k0 + k < topk ? k0 + k : 0];
        p[k] = k0 + k < topk && unsigned(p[k]) < unsigned(capacity) ? p[k] : -1;
    }
#pragma unroll
    for (int k = 0; k < kWide; ++k)
        values.fetch(p[k] < 0 ? 0 : p[k], at, w[k]);
}

// Columns of a row that a thread has: 16 bytes of the values, which lie side by side across
// the lanes.
template <bool FROM>
constexpr int kCols = FROM ? 8 : 4;

template <bool FROM, bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(CombineRowsArgs a, int chunks)
{
    constexpr int COLS = kCols<FROM>;
    using M = Matrix<FROM, WHOLE, COLS>;
    const M values(a.values, a.capacity, a.dim);
    const int64_t n = a.rows * chunks;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
        const int64_t r = i / chunks;
        const int at = int(i - r * chunks) * COLS;
        float sum[COLS] = {};
        for (int k0 = 0; k0 < a.topk; k0 += kWide) {
            int p[kWide];
            float by[kWide], v[COLS];
            typename M::Raw w[kWide];
            fetch_slots(values, a.slot + r * a.topk, k0, a.topk, a.capacity, at, p, w);
#pragma unroll
            for (int k = 0; k < kWide; ++k)
                by[k] = a.weight ? a.weight[r * a.topk + (k0 + k < a.topk ? k0 + k : 0)] : 1.0f;
#pragma unroll
            for (int k = 0; k < kWide; ++k) {
                values.take(p[k] < 0 ? 0 : p[k], at, w[k], v);
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    sum[c] = p[k] >= 0 ? __builtin_fmaf(by[k], v[c], sum[c]) : sum[c];
            }
        }
        store_row<BF16, WHOLE, COLS>(a.y, r * a.dim, at, a.dim, sum);
    }
}

// A row by a wave, eight choices at a time.
template <bool FROM, bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs a)
{
    constexpr int COLS = kCols<FROM>;
    using M = Matrix<FROM, WHOLE, COLS>;
    using D = Matrix<BF16, WHOLE, COLS>;
    const M values(a.values, a.capacity, a.dim);
    const D grad(a.dy, a.rows, a.dim);
    const int lane = threadIdx.x % 64;
    for (int64_t r = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64; r < a.rows; r += int64_t(gridDim.x) * (kThreads / 64))
        for (int k0 = 0; k0 < a.topk; k0 += kWide) {
            float dot[kWide] = {};
            for (int at = lane * COLS; at < a.dim; at += 64 * COLS) {
                int p[kWide];
                float v[COLS], dy[COLS];
                typename M::Raw w[kWide];
                typename D::Raw of_dy;
                grad.fetch(r, at, of_dy);
                fetch_slots(values, a.slot + r * a.topk, k0, a.topk, a.capacity, at, p, w);
                grad.take(r, at, of_dy, dy);
#pragma unroll
                for (int k = 0; k < kWide; ++k) {
                    values.take(p[k] < 0 ? 0 : p[k], at, w[k], v);
#pragma unroll
                    for (int c = 0; c < COLS; ++c)
                        dot[k] = p[k] < 0 ? 0.0f : __builtin_fmaf(dy[c], v[c], dot[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < kWide; ++k) {
                const float d = lanes_sum<64>(dot[k]);
                if (lane == 0 && k0 + k < a.topk)
                    a.grad_weight[r * a.topk + k0 + k] = d;
            }
        }
}

// Rows that start at, and are a multiple of, 16 bytes.
bool whole(const void *p, int64_t dim, bool bf16) { return in_chunks(p, dim, bf16 ? 2 : 4); }

// f(bf16, whole) as compile-time values.
template <typename F>
hipError_t with_form(bool bf16, bool w, F f)
{
    using Yes = std::true_type;
    using No = std::false_type;
    return bf16 ? (w ? f(Yes{}, Yes{}) : f(Yes{}, No{})) : (w ? f(No{}, Yes{}) : f(No{}, No{}));
}

unsigned grid_of(int64_t n, int64_t per, unsigned most)
{
    const int64_t b = (n + per - 1) / per;
    return unsigned(b < most ? b : most);
}

}  // namespace

int32_t slots_blocks(int64_t choices)
{
    if (choices <= kOnePiece)
        return 1;
    // each workgroup reads the counts of all (524288 choices 19 us, by 256 of them 23 us)
    const int64_t n = (choices + kPiece - 1) / kPiece;
    return int32_t(n < 128 ? n : 128);
}

hipError_t launch_slots_count(const Op &op, hipStream_t stream)
{
    const SlotsArgs a = op.get<SlotsArgs>();
    (void)hipGetLastError();
    slots_count_kernel<<<dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_slots(const Op &op, hipStream_t stream)
{
    const SlotsArgs a = op.get<SlotsArgs>();
    (void)hipGetLastError();
    slots_kernel<<<dim3(unsigned(a.blocks)), dim3(kSlotThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(const Op &op, hipStream_t stream)
{
    const QuantizeRowsArgs a = op.get<QuantizeRowsArgs>();
    const int blocks = (a.dim + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    (void)hipGetLastError();
    return with_form(a.bf16, whole(a.x, a.dim, a.bf16), [&](auto bf16, auto w) {
        quantize_rows_kernel<decltype(bf16)::value, decltype(w)::value>
            <<<dim3(grid_of(a.rows * blocks, kThreads / 16, 8192)), dim3(kThreads), 0, stream>>>(a, blocks);
        return hipGetLastError();
    });
}

hipError_t launch_quantize_slots(const Op &op, hipStream_t stream)
{
    const QuantizeSlotsArgs a = op.get<QuantizeSlotsArgs>();
    const int blocks = (a.dim + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    (void)hipGetLastError();
    return with_form(a.bf16, whole(a.x, a.dim, a.bf16), [&](auto bf16, auto w) {
        quantize_slots_kernel<decltype(bf16)::value, decltype(w)::value>
            <<<dim3(unsigned(blocks) * unsigned(a.blocks)), dim3(kThreads), 0, stream>>>(a, blocks);
        return hipGetLastError();
    });
}

hipError_t launch_quantize_weight(const Op &op, hipStream_t stream)
{
    const QuantizeWeightArgs a = op.get<QuantizeWeightArgs>();
    const int n = (a.n + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK, k = (a.k + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    (void)hipGetLastError();
    return with_form(a.bf16, whole(a.w, a.k, a.bf16), [&](auto bf16, auto w) {
        const dim3 grid(unsigned(n) * unsigned(k) * unsigned(a.experts));
        if (int64_t(a.experts) * a.n * a.k * (a.bf16 ? 2 : 4) > kCacheBytes)
            quantize_weight_kernel<decltype(bf16)::value, decltype(w)::value, true><<<grid, dim3(kThreads), 0, stream>>>(a, n, k);
        else
            quantize_weight_kernel<decltype(bf16)::value, decltype(w)::value, false><<<grid, dim3(kThreads), 0, stream>>>(a, n, k);
        return hipGetLastError();
    });
}

hipError_t launch_combine_rows(const Op &op, hipStream_t stream)
{
    const CombineRowsArgs a = op.get<CombineRowsArgs>();
    const int cols = a.from_bf16 ? kCols<true> : kCols<false>, chunks = (a.dim + cols - 1) / cols;
    const bool w = whole(a.values, a.dim, a.from_bf16) && whole(a.y, a.dim, a.bf16);
    (void)hipGetLastError();
    return with_form(a.bf16, w, [&](auto bf16, auto all) {
        const dim3 grid(grid_of(a.rows * chunks, kThreads, 16384));
        if (a.from_bf16)
            combine_rows_kernel<true, decltype(bf16)::value, decltype(all)::value><<<grid, dim3(kThreads), 0, stream>>>(a, chunks);
        else
            combine_rows_kernel<false, decltype(bf16)::value, decltype(all)::value><<<grid, dim3(kThreads), 0, stream>>>(a, chunks);
        return hipGetLastError();
    });
}

hipError_t launch_combine_grad(const Op &op, hipStream_t stream)
{
    const CombineGradArgs a = op.get<CombineGradArgs>();
    const bool w = whole(a.values, a.dim, a.from_bf16) && whole(a.dy, a.dim, a.bf16);
    (void)hipGetLastError();
    return with_form(a.bf16, w, [&](auto bf16, auto all) {
        const dim3 grid(grid_of(a.rows, kThreads / 64, 16384));
        if (a.from_bf16)
            combine_grad_kernel<true, decltype(bf16)::value, decltype(all)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
        else
            combine_grad_kernel<false, decltype(bf16)::value, decltype(all)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace rr
