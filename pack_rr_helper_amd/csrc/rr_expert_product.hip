// rr_expert_product.hip -- gfx950 products of matrices in 8 bits with a power of two
// for each block of 128 along k, over the segments of an expert layer.
//
// One matrix instruction multiplies 16 x 128 by 128 x 16 elements and applies the
// operands' powers itself, so that a block of k is one instruction and costs no
// vector instruction; sums over blocks are held in 32 bits.  Which bytes of a block
// a lane holds does not matter as long as both operands agree, its power being one.
//
// Within a block that instruction keeps about 17 bits below its largest product
// (measured: 1.6e-5 of a sum of 128 normal products, whatever is added to), less than
// the 2^-9 of a result in bf16 and more than a result in 32 bits may be off.  Results in
// 32 bits therefore take the operands as bf16, which holds e4m3 times a power of two
// exactly from 2^-117 on (below 2^-126 it has multiples of 2^-133), through the bf16
// instructions (1e-8, at half the rate: 1060 us, 1030 TFLOP/s, for the product below): FULL.
#include "rr_expert.h"
#include "rr_product.h"

#include <math.h>

namespace rr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// c += a b, a lane's powers being byte PA of pa and byte PB of pb.
template <int PA, int PB>
__device__ __forceinline__ void multiply(const i32x8 &a, const i32x8 &b, f32x4 &c, unsigned pa, unsigned pb)
{
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, PA, int(pa), PB, int(pb));
}

// A lane's 32 elements times 2^(power - 127), in bf16.
struct Wide {
    bf16x8 v[4];

    __device__ __forceinline__ void set(const i32x8 &from, unsigned power)
    {
        const float by = __uint_as_float((power & 255u) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[2 * h] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(from[2 * i + h]), by, false));
                w[2 * h + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(from[2 * i + h]), by, true));
            }
            v[i] = __builtin_bit_cast(bf16x8, w);
        }
    }
};

__device__ __forceinline__ void multiply(const Wide &a, const Wide &b, f32x4 &c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
}

struct Place {
    int e, i, j;  // expert, and tile in its matrix and in its segment
};

// Which tile of the experts' segments a workgroup computes, or none.  Every wave
// finds out by itself.
__device__ __forceinline__ bool place_of(const int32_t *count, int experts, int wide, int tiles_i, Place &at)
{
    const int lane = threadIdx.x % 64;
    int total = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        int n = e0 + lane < experts ? (count[e0 + lane] + wide - 1) / wide : 0;
        for (int d = 32; d > 0; d /= 2)
            n += __shfl_xor(n, d);
        total += n;
    }
    if (int64_t(blockIdx.x) >= int64_t(total) * tiles_i)
        return false;
    int j;
    tile_at(int(blockIdx.x), total * tiles_i, tiles_i, total, at.i, j);
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int n = e0 + lane < experts ? (count[e0 + lane] + wide - 1) / wide : 0;
        int sum = n;
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            sum += lane >= d ? o : 0;
        }
        const unsigned long long past = __ballot(before + sum > j);
        if (past) {
            const int l = __ffsll(past) - 1;
            at.e = __builtin_amdgcn_readfirstlane(e0 + l);
            at.j = __builtin_amdgcn_readfirstlane(j - before - (__shfl(sum, l) - __shfl(n, l)));
            return true;
        }
        before += __shfl(sum, 63);
    }
    return false;
}

// The row of x at a position, -1 past the expert's choices.
__device__ __forceinline__ int row_of(const ExpertProductArgs &a, int p, bool in)
{
    if (!in)
        return -1;
    if (!a.gather)
        return p;
    const int n = a.source[p];
    return unsigned(n) < unsigned(a.choices) ? n / a.topk : -1;
}

__device__ __forceinline__ float weight_of(const ExpertProductArgs &a, int p, bool in)
{
    if (!in || !a.weight)
        return 1.0f;
    const int n = a.source[p];
    return unsigned(n) < unsigned(a.choices) ? a.weight[n] : 0.0f;
}

// ---------------------------------------------------------------------------
// Few positions a segment: KS waves stream FI * 16 rows of the weights from memory to
// registers, past all positions of the tile, a block of k each in turns.  Bound by the
// weights' bytes, and by how many are under way: x is read again for every 16 rows, so
// that four such per wave take 32 us where one takes 47 us (96 x 6 choices of 64 experts,
// 2048 x 1408); two waves to a workgroup 32 us, four 34 us.
// ---------------------------------------------------------------------------

// Block b of a row of k; a lane has its chunks g and g + 4.
struct Block {
    i32x8 v;
    unsigned p;   // its power in the low byte

    __device__ __forceinline__ void load(const unsigned char *row, const unsigned char *powers, int b)
    {
        typedef u32x4 Half __attribute__((aligned(16)));
        const unsigned char *at = row + int64_t(b) * RR_QUANT_BLOCK;
        const u32x4 lo = *reinterpret_cast<const Half *>(at), hi = *reinterpret_cast<const Half *>(at + 64);
        v = i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
        p = powers[b];
    }
};

template <int FJ, bool FULL, int KS, int FI>
__global__ __launch_bounds__(KS * 64) void narrow_kernel(ExpertProductArgs a, int tiles_i)
{
    constexpr int TJ = 16 * FJ;
    __shared__ __attribute__((aligned(16))) f32x4 sums[KS][FI * FJ][64];
    Place at;
    if (!place_of(a.count, a.experts, TJ, tiles_i, at))
        return;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 16, g = lane / 16;
    const int blocks = int(a.w.ld / RR_QUANT_BLOCK), blocks_n = (a.n + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    const int i0 = at.i * 16 * FI, k0 = wave < blocks ? wave : blocks - 1;
    const unsigned char *wv[FI], *wp[FI];
    Block w[FI], x[FJ];
    // the weights are what takes long: on their way before the rows of x are known
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        const int i = i0 + f * 16 + r, row_i = i < a.n ? i : a.n - 1;
        wv[f] = a.w.values + (int64_t(at.e) * a.n + row_i) * a.w.ld + g * 16;
        wp[f] = a.w.powers + (int64_t(at.e) * blocks_n + row_i / RR_QUANT_BLOCK) * a.w.lds;
        w[f].load(wv[f], wp[f], k0);
    }
    const int j0 = at.j * TJ, live = a.count[at.e] - j0, first = a.offset[at.e] + j0;
    const unsigned char *xv[FJ], *xp[FJ];
#pragma unroll
    for (int f = 0; f < FJ; ++f) {
        const int j = f * 16 + r, row = row_of(a, first + j, j < live), in = row < 0 ? 0 : row;
        xv[f] = a.x.values + int64_t(in) * a.x.ld + g * 16;
        xp[f] = a.x.powers + int64_t(in) * a.x.lds;
        x[f].load(xv[f], xp[f], k0);
    }
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = wave; b < blocks; b += KS) {
        Block w0[FI], x0[FJ];
#pragma unroll
        for (int f = 0; f < FI; ++f)
            w0[f] = w[f];
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            x0[f] = x[f];
        const int next = b + KS < blocks ? b + KS : b;
#pragma unroll
        for (int f = 0; f < FI; ++f)
            w[f].load(wv[f], wp[f], next);
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            x[f].load(xv[f], xp[f], next);
        if constexpr (FULL) {
            Wide wide[FI];
#pragma unroll
            for (int i = 0; i < FI; ++i)
                wide[i].set(w0[i].v, w0[i].p);
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                Wide of_x;
                of_x.set(x0[j].v, x0[j].p);
#pragma unroll
                for (int i = 0; i < FI; ++i)
                    multiply(wide[i], of_x, acc[i][j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    multiply<0, 0>(w0[i].v, x0[j].v, acc[i][j], w0[i].p, x0[j].p);
        }
    }
#pragma unroll
    for (int n = 0; n < FI * FJ; ++n)
        sums[wave][n][lane] = acc[n / FJ][n % FJ];
    __syncthreads();
    for (int f = wave; f < FI * FJ; f += KS) {
        f32x4 s = sums[0][f][lane];
#pragma unroll
        for (int n = 1; n < KS; ++n)
            s += sums[n][f][lane];
        const int j = f % FJ * 16 + r, i = i0 + f / FJ * 16 + g * 4;
        if (j >= live || i >= a.n)
            continue;
        s *= weight_of(a, first + j, true);
        const int64_t to = int64_t(first + j) * a.n + i;
        if constexpr (FULL) {
            store_chunk<4>(static_cast<char *>(a.out) + to * 4, __builtin_bit_cast(u32x4, s), (a.n - i) * 4);
        } else {
            auto *out = static_cast<unsigned short *>(a.out) + to;
            const u32x2 v{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
            if (i + 3 < a.n) {
                __builtin_memcpy(out, &v, 8);
            } else {
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    if (i + n < a.n)
                        out[n] = (unsigned short)(v[n / 2] >> 16 * (n % 2));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------

// A workgroup's tile, the same in all its lanes.
struct Span {
    int e, i0, j0;       // expert; first row of A and of B, or of the segment
    int first, live;     // product: first position, positions from there on
    int s0, s1;          // steps of k
};

// Where the workgroup's tables lie in LDS: of every expert the tiles of the experts before
// it, its first position and its choices; the choices of two tiles, the weights of four;
// what the workgroup's tiles are, as finding that out takes longer than looking it up.
struct Tables {
    int *before, *offset, *count, *list;
    float *weight;
    int4 *span;          // the workgroup's first kSpans tiles: e, i0, then j0 or first, live
};
constexpr int kSpans = 256;

// Fills the tables; the number of segments' tiles, `wide` positions each.
__device__ __forceinline__ int fill_tables(const Tables &t, const int32_t *offset, const int32_t *count, int experts, int wide)
{
    const int lane = threadIdx.x % 64;
    int total = 0;
    // every wave finds the total, the first one writes
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane, n = e < experts ? count[e] : 0, m = (n + wide - 1) / wide;
        int sum = m;
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            sum += lane >= d ? o : 0;
        }
        if (threadIdx.x < 64 && e < experts) {
            t.before[e] = total + sum - m;
            t.offset[e] = offset[e];
            t.count[e] = n;
        }
        total += __shfl(sum, 63);
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(total);
}

// A workgroup computes tiles of C[j][i] = sum_k A[i][k] B[j][k] one after the other.
// Steps of 128 elements of k, of one tile and then of the next, are loaded two ahead
// into two places in LDS (the layout of Tile, rr_product.h; a lane's 32 bytes of a row are
// its chunks g and g + 4), so that the matrix units do not wait where tiles change:
// 8192 x 8 choices of 32 experts, 4096 x 2048, took 712 us with a workgroup for each tile
// and the memory operations at the steps' ends, 594 us as it is (1850 TFLOP/s; one
// dense product of 8192^3 2600).  What is left is the power that the matrix units draw: a
// loop of nothing but their instructions reaches 4650 TFLOP/s on constant and 3630 on random
// data; and a fifth of a tile's time, its results' way out between two tiles.
// Powers come four steps at a time, a word for each row of the tile.
// A step is computed in two halves of the rows i.  While the first runs, the
// second's fragments are read; into the second, one barrier says that this step has
// been read by all and that the next one has arrived.
// BLOCK_A: the rows of a wave share one power.
template <int TI_, int TJ_, int WI, int WJ, bool BLOCK_A, bool FULL>
struct Tile8 {
    static constexpr int TI = TI_, TJ = TJ_, kWaves = WI * WJ, kThreads = kWaves * 64;
    static constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16, H = FI / 2;
    static constexpr int kRows = 8 * kWaves, kLoadBytes = kRows * kRowBytes;
    static constexpr int kLoadsA = TI / kRows, kLoadsB = TJ / kRows, kLoadsP = (TI + TJ) / kThreads;
    static constexpr int kStageBytes = (TI + TJ) * kRowBytes, kPowerBytes = (TI + TJ) * 4;
    static constexpr int kFixedBytes = 2 * kStageBytes + 3 * kPowerBytes + 6 * TJ * 4 + kSpans * 16;
    // workgroups on a compute unit (of 512 experts at most), and waves on a SIMD, which
    // its registers are divided by
    static constexpr int kPerUnit = 160 * 1024 / (kFixedBytes + 12 * 512), kPerSimd = kPerUnit * kWaves / 4;
    static constexpr bool kFull = FULL;  // results in 32 bits
    static_assert(kLoadsP * kThreads == TI + TJ && TI % 64 == 0, "a wave loads the powers of one operand");
    static_assert(!BLOCK_A || RR_QUANT_BLOCK % (FI * 16) == 0, "");
    static_assert(FJ >= 4 && H >= 1, "");
    // results leave as those of a product in bf16 and fp32 do
    using Out = Tile<!FULL, TI, TJ, WI, WJ, 2, true>;

    static int lds_bytes(int experts) { return kFixedBytes + 12 * experts; }
    __device__ static Tables tables(char *lds, int experts)
    {
        int *t = reinterpret_cast<int *>(lds + 2 * kStageBytes + 3 * kPowerBytes), *e = t + 6 * TJ + 4 * kSpans;
        return Tables{e, e + experts, e + 2 * experts, t, reinterpret_cast<float *>(t + 2 * TJ), reinterpret_cast<int4 *>(t + 6 * TJ)};
    }

    // Bytes of a buffer from its first row on, below kNowhere.
    __device__ static __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t bytes)
    {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0,
                                                 int(bytes < kNowhere ? bytes : kNowhere), kBufferFormat);
    }
    __device__ static int wave() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64); }
    __device__ static int wave_i() { return wave() % WI * (FI * 16); }
    __device__ static int wave_j() { return wave() / WI * (FJ * 16); }

    // The steps of a tile that are still to be loaded.
    struct Source {
        __amdgpu_buffer_rsrc_t a, b, power[kLoadsP];
        int off_a[kLoadsA], off_b[kLoadsB], off_power[kLoadsP];
        int s, s1, group;  // group: of powers, counted over all tiles
        bool words;        // this step's powers begin a word, or a tile

        // ra(i), rb(j): the rows in the buffers of the tile's rows, -1 for none; pa: the same
        // in A's powers.
        template <typename RA, typename RB, typename PA>
        __device__ void open(const Eight &x, int64_t bytes_a, int64_t power_a, const Eight &y, int64_t bytes_b,
                             int64_t power_b, RA ra, RB rb, PA pa, const Span &span)
        {
            const int lane = threadIdx.x % 64;
            s = span.s0;
            s1 = span.s1;
            group += s < s1;  // a tile without steps has no powers
            words = true;
            a = buffer(x.values, bytes_a);
            b = buffer(y.values, bytes_b);
            const int row0 = wave() * 8 + lane / 8, chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
#pragma unroll
            for (int l = 0; l < kLoadsA; ++l) {
                const int r = ra(l * kRows + row0);
                off_a[l] = r >= 0 ? r * int(x.ld) + chunk : kNowhere;
            }
#pragma unroll
            for (int l = 0; l < kLoadsB; ++l) {
                const int r = rb(l * kRows + row0);
                off_b[l] = r >= 0 ? r * int(y.ld) + chunk : kNowhere;
            }
#pragma unroll
            for (int l = 0; l < kLoadsP; ++l) {
                const int row = l * kThreads + int(threadIdx.x);
                const bool of_a = l * kThreads + wave() * 64 < TI;
                power[l] = of_a ? buffer(x.powers, power_a) : buffer(y.powers, power_b);
                const int r = of_a ? pa(row) : rb(row - TI);
                off_power[l] = r >= 0 ? r * int(of_a ? x.lds : y.lds) : kNowhere;
            }
        }
        // No more tiles: loads give zeros.
        __device__ void close()
        {
            s = 0;
            s1 = 1 << 30;
            ++group;
            words = false;
            a = buffer(nullptr, 0);
            b = buffer(nullptr, 0);
#pragma unroll
            for (int l = 0; l < kLoadsP; ++l)
                power[l] = buffer(nullptr, 0);
        }
        static constexpr int kLoads = kLoadsP + kLoadsA + kLoadsB;
        // Load l of the next step, to place `stage` in LDS.
        __device__ void load(int l, char *lds, int stage) const
        {
            char *to = lds + stage * kStageBytes + wave() * 1024;
            if (l < kLoadsA)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(a, lds_pointer(to + l * kLoadBytes), 16, off_a[l], s * kRowBytes, 0, 0);
            else if (l < kLoadsA + kLoadsB)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds_pointer(to + l * kLoadBytes), 16, off_b[l - kLoadsA], s * kRowBytes, 0, 0);
            else
                // a word holds four steps.  In the other three the load reads nothing (64
                // rows of 4 bytes cost as much as 64 rows of 128) and leaves zeros where
                // nothing lies.
                __builtin_amdgcn_raw_ptr_buffer_load_lds(power[l - kLoadsA - kLoadsB],
                    lds_pointer(lds + 2 * kStageBytes + (words ? group % 2 : 2) * kPowerBytes + wave() * 256 + (l - kLoadsA - kLoadsB) * kThreads * 4), 4,
                    words ? off_power[l - kLoadsA - kLoadsB] : kNowhere, s / 4 * 4, 0, 0);
        }
        __device__ void next()
        {
            ++s;
            words = s % 4 == 0;
            group += words && s < s1;
        }
    };

    // A lane's 32 bytes of a row of 16, read in two halves.
    struct Fragment {
        u32x4 half[2];

        __device__ void read(const char *stage, int f, int h)
        {
            const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
            half[h] = *reinterpret_cast<const u32x4 *>(stage + (f + r) * kRowBytes + ((4 * h + g) ^ (r >> 1)) * 16);
        }
        __device__ i32x8 value() const { return __builtin_bit_cast(i32x8, half); }
    };
    __device__ static void read_a(Fragment *fa, const char *lds, int stage, int n)
    {
        fa[n / 2].read(lds + stage * kStageBytes, wave_i() + n / 2 * 16, n % 2);
    }
    __device__ static void read_b(Fragment *fb, const char *lds, int stage, int n)
    {
        fb[n / 2].read(lds + stage * kStageBytes + kLoadsA * kLoadBytes, wave_j() + n / 2 * 16, n % 2);
    }

    static constexpr int kPowersA = BLOCK_A ? 1 : FI;
    struct Powers {
        unsigned a[kPowersA], b[FJ];

        __device__ void read(const char *lds, int group)
        {
            const unsigned *at = reinterpret_cast<const unsigned *>(lds + 2 * kStageBytes + group % 2 * kPowerBytes) + threadIdx.x % 16;
#pragma unroll
            for (int f = 0; f < kPowersA; ++f)
                a[f] = at[wave_i() + f * 16];
#pragma unroll
            for (int f = 0; f < FJ; ++f)
                b[f] = at[TI + wave_j() + f * 16];
        }
        // Those of step s in the low bytes.
        __device__ Powers of(int s) const
        {
            Powers p;
#pragma unroll
            for (int f = 0; f < kPowersA; ++f)
                p.a[f] = a[f] >> s % 4 * 8;
#pragma unroll
            for (int f = 0; f < FJ; ++f)
                p.b[f] = b[f] >> s % 4 * 8;
            return p;
        }
    };
    struct Acc {
        f32x4 c[FI][FJ];

        __device__ void clear()
        {
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };

    // A workgroup's tiles, `tiles` of them.  job.span(n): the n-th; job.first(): before it
    // is opened; job.open(source, n, last): its source; job.end(span, n, acc): its results.
    // A tile of one step is opened right after the one before it.
    template <typename Job>
    __device__ static void run(const Job &job, int tiles, char *lds)
    {
        Source source;
        source.s = source.s1 = 0;
        source.group = -1;
        int opened = 0, stage = 0, group = 0;
        const auto refill = [&] {
            while (source.s == source.s1) {
                if (opened >= tiles) {
                    source.close();
                    return;
                }
                job.open(source, opened, opened + 1 == tiles);
                ++opened;
            }
        };
        if (tiles <= 0)
            return;
        job.first();
        Acc acc;
        Fragment fa[FI], fb[FJ];
        Powers raw;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            refill();
#pragma unroll
            for (int l = 0; l < Source::kLoads; ++l)
                source.load(l, lds, f);
            source.next();
            if (f == 0 || opened > 1) {
                // between any two calls of open() stands a wait and a barrier, here as in the
                // loop below: what the next tile's source needs, loaded by all waves, is there,
                // and all waves have read what the next call overwrites
                wait_loads<0>();
                __builtin_amdgcn_s_barrier();
            }
        }
#pragma unroll
        for (int h = 0; h < 2 * FJ; ++h)
            read_b(fb, lds, 0, h);
#pragma unroll
        for (int h = 0; h < 2 * (FULL ? FI : H); ++h)
            read_a(fa, lds, 0, h);
        raw.read(lds, 0);
        for (int n = 0; n < tiles; ++n) {
            const Span span = job.span(n);
            acc.clear();
            for (int s = span.s0; s < span.s1; ++s, stage ^= 1) {
                refill();
                // one block without branches from here on: memory operations in the
                // shadow of matrix instructions, a few at a time
                const Powers at = raw.of(s);
                group += (s + 1) % 4 == 0 || s + 1 == span.s1;
                if constexpr (FULL) {
                    Wide wb[FJ];
#pragma unroll
                    for (int j = 0; j < FJ; ++j)
                        wb[j].set(fb[j].value(), at.b[j]);
#pragma unroll
                    for (int i = 0; i < FI; ++i) {
                        Wide wa;
                        wa.set(fa[i].value(), at.a[BLOCK_A ? 0 : i]);
                        if (i == 0) {
                            // this step has been read by all, and the next one has arrived
                            wait_loads<0>();
                            __builtin_amdgcn_s_barrier();
                        }
#pragma unroll
                        for (int j = 0; j < FJ; ++j) {
                            multiply(wa, wb[j], acc.c[i][j]);
                            constexpr int kPer = (Source::kLoads + FJ - 1) / FJ;
                            if (i == 0)
#pragma unroll
                                for (int l = j * kPer; l < j * kPer + kPer && l < Source::kLoads; ++l)
                                    source.load(l, lds, stage);
                            if (i == 1)
#pragma unroll
                                for (int h = j * 2; h < j * 2 + 2; ++h)
                                    read_b(fb, lds, stage ^ 1, h);
                            if (i >= FI / 2 && j < 4) {
                                constexpr int kRead = FI / (FI - FI / 2);
#pragma unroll
                                for (int h = ((i - FI / 2) * 4 + j) * kRead / 2; h < ((i - FI / 2) * 4 + j + 1) * kRead / 2; ++h)
                                    if (h < 2 * i)
                                        read_a(fa, lds, stage ^ 1, h);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    read_a(fa, lds, stage ^ 1, 2 * FI - 2);
                    read_a(fa, lds, stage ^ 1, 2 * FI - 1);
                    raw.read(lds, group);
                } else {
                    constexpr int kHalf = H * FJ, kBarrier = kHalf - kHalf / 8;
#pragma unroll
                    for (int m = 0; m < 2 * kHalf; ++m) {
                        const int j = m % kHalf / H, i = m / kHalf * H + m % H;
                        multiply<0, 0>(fa[i].value(), fb[j].value(), acc.c[i][j], at.a[BLOCK_A ? 0 : i], at.b[j]);
                        // a's second half, every other time
                        if (m % 2 == 1 && m / 2 < 2 * (FI - H))
                            read_a(fa, lds, stage, 2 * H + m / 2);
                        if (m == kBarrier) {
                            // this step has been read by all, and the next one has arrived
                            wait_loads<0>();
                            __builtin_amdgcn_s_barrier();
                        }
                        if (m >= kBarrier && m - kBarrier < Source::kLoads)
                            source.load(m - kBarrier, lds, stage);
                        // b's columns once they have been used, with them a's first half
                        if (m >= kHalf && m % H == H - 1) {
                            read_b(fb, lds, stage ^ 1, 2 * j);
                            read_b(fb, lds, stage ^ 1, 2 * j + 1);
                        }
                        if (m >= kHalf && m % H < 2 && (m - kHalf) / H * 2 + m % H < 2 * H)
                            read_a(fa, lds, stage ^ 1, (m - kHalf) / H * 2 + m % H);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    raw.read(lds, group);
                }
                source.next();
            }
            job.end(span, n, acc);
        }
        wait_loads<0>();
    }
};

// A tile's results times by(column of the tile) to out, from its first row and column on:
// `rows` and `left` columns of them, ld elements a row.  Where rows lie in 16-byte chunks
// a chunk is stored or not as a whole, without branches.
template <typename T, typename BY>
__device__ __forceinline__ void store(const typename T::Acc &acc, void *out, int64_t ld, int rows, int left, BY by)
{
    constexpr int es = T::kFull ? 4 : 2, kChunks = T::kFull ? T::FI : T::FI / 2, kPer = 16 / es;
    const int g = threadIdx.x % 64 / 16;
    if (in_chunks(out, ld, es)) {
        const __amdgpu_buffer_rsrc_t to = T::buffer(out, kNowhere);
        int at[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            // the columns that store_row gives a lane
            const int i = T::wave_i() + (T::kFull ? c * 16 + g * 4 : (2 * c + g % 2) * 16 + g / 2 * 8);
            at[c] = i < left ? i * es : kNowhere;
        }
        static_assert(kPer == (T::kFull ? 4 : 8), "");
#pragma unroll
        for (int f = 0; f < T::FJ; ++f) {
            const int j = T::wave_j() + f * 16 + int(threadIdx.x % 16);
            const int row = j < rows ? j * int(ld * es) : kNowhere;
            const float w = by(j);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                u32x4 v;
                if constexpr (T::kFull) {
                    v = __builtin_bit_cast(u32x4, f32x4(acc.c[c][f] * w));
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const f32x4 lo = acc.c[2 * c][f] * w, hi = acc.c[2 * c + 1][f] * w;
                        const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16(lo[2 * n], lo[2 * n + 1]),
                                                                        pack_bf16(hi[2 * n], hi[2 * n + 1]), false, false);
                        v[n] = s[0];
                        v[2 + n] = s[1];
                    }
                }
                __builtin_amdgcn_raw_buffer_store_b128(v, to, int(unsigned(row) + unsigned(at[c])), 0, 0);
            }
        }
        return;
    }
#pragma unroll
    for (int f = 0; f < T::FJ; ++f) {
        const int j = T::wave_j() + f * 16 + int(threadIdx.x % 16);
        const float w = by(j);
        f32x4 v[T::FI];
#pragma unroll
        for (int i = 0; i < T::FI; ++i)
            v[i] = acc.c[i][f] * w;
        T::Out::store_row(static_cast<char *>(out) + j * ld * es, v, j < rows ? left : 0);
    }
}

template <typename T>
struct ProductJob {
    const ExpertProductArgs &a;
    Tables tables;
    int tiles_i, tiles_j;

    // The n-th tile of the workgroup, by its thread: expert, first column, first position,
    // positions from there on.
    __device__ int4 find(int n) const
    {
        int i, j;
        tile_at(int(blockIdx.x) + n * int(gridDim.x), tiles_i * tiles_j, tiles_i, tiles_j, i, j);
        // the last expert with at most j tiles before it
        int e = 0;
        for (int step = 512; step > 0; step /= 2)
            if (e + step < a.experts && tables.before[e + step] <= j)
                e += step;
        const int j0 = (j - tables.before[e]) * T::TJ;
        return int4{e, i * T::TI, tables.offset[e] + j0, tables.count[e] - j0};
    }
    __device__ Span span(int n) const
    {
        const int4 v = n < kSpans ? tables.span[n] : find(n);
        return Span{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y), 0,
                    __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w), 0, int(a.w.ld / RR_QUANT_BLOCK)};
    }
    // Row of x, of choice n.
    __device__ int row_of(int n) const { return n < 0 ? -1 : int((__umulhi(a.topk_mul, unsigned(n)) + unsigned(n)) >> a.topk_shift); }
    // The choices of a tile, to list n; a wave for 64 of them.
    __device__ void fetch_list(const Span &s, int n) const
    {
        if (T::wave() * 64 < T::TJ)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                T::buffer(a.source + s.first, int64_t(s.live) * 4),
                lds_pointer(reinterpret_cast<char *>(tables.list + n % 2 * T::TJ + T::wave() * 64)), 4, int(threadIdx.x) * 4, 0, 0, 0);
    }
    __device__ bool listed() const { return a.gather || a.weight; }
    __device__ void first() const
    {
        if (listed()) {
            fetch_list(span(0), 0);
            wait_loads<0>();
            __syncthreads();
        }
    }
    __device__ void open(typename T::Source &source, int n, bool last) const
    {
        const Span s = span(n);
        const int *list = tables.list + n % 2 * T::TJ;
        const int blocks_n = (a.n + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK, rows_i = a.n - s.i0;
        // from the tile's first row on; gathered rows may be anywhere
        const Eight w{a.w.values + (int64_t(s.e) * a.n + s.i0) * a.w.ld,
                      a.w.powers + (int64_t(s.e) * blocks_n + s.i0 / RR_QUANT_BLOCK) * a.w.lds, a.w.ld, a.w.lds};
        const int base = a.gather ? 0 : s.first;
        const Eight x{a.x.values + base * a.x.ld, a.x.powers + base * a.x.lds, a.x.ld, a.x.lds};
        const int64_t rows_x = a.gather ? a.rows : s.live;
        source.open(w, rows_i * w.ld, (blocks_n - s.i0 / RR_QUANT_BLOCK) * w.lds, x, rows_x * x.ld, rows_x * x.lds,
                    [&](int i) { return i < rows_i ? i : -1; },
                    [&](int j) {
                        if (j >= s.live)
                            return -1;
                        if (!a.gather)
                            return j;
                        const int r = row_of(list[j]);
                        return r < a.rows ? r : -1;
                    },
                    [&](int i) { return i < rows_i ? i / RR_QUANT_BLOCK : -1; }, s);
        if (a.weight && T::wave() * 64 < T::TJ) {
            const int j = int(threadIdx.x), at = j < s.live ? list[j] : -1;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                T::buffer(a.weight, int64_t(a.choices) * 4),
                lds_pointer(reinterpret_cast<char *>(tables.weight + n % 4 * T::TJ + T::wave() * 64)), 4, at >= 0 ? at * 4 : kNowhere, 0, 0, 0);
        }
        if (listed() && !last)
            fetch_list(span(n + 1), n + 1);
    }
    __device__ void end(const Span &s, int n, const typename T::Acc &acc) const
    {
        void *out = static_cast<char *>(a.out) + (int64_t(s.first) * a.n + s.i0) * (T::kFull ? 4 : 2);
        const float *by = a.weight ? tables.weight + n % 4 * T::TJ : nullptr;
        store<T>(acc, out, a.n, s.live, a.n - s.i0, [=](int j) { return by ? by[j] : 1.0f; });
    }
};

// Tiles of the workgroup, of n in all; their spans to the table.
template <typename Job>
__device__ __forceinline__ int own_tiles(const Job &job, int n)
{
    const int own = int(blockIdx.x) < n ? (n - int(blockIdx.x) - 1) / int(gridDim.x) + 1 : 0;
    for (int i = threadIdx.x; i < kSpans && i < own; i += blockDim.x)
        job.tables.span[i] = job.find(i);
    __syncthreads();
    return own;
}

template <typename T>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void product_kernel(ExpertProductArgs a, int tiles_i)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const Tables tables = T::tables(lds, a.experts);
    const int tiles_j = fill_tables(tables, a.offset, a.count, a.experts, T::TJ);
    const ProductJob<T> job{a, tables, tiles_i, tiles_j};
    T::run(job, own_tiles(job, tiles_i * tiles_j), lds);
}

// dw[e][j][i] = sum over the segment's positions of x[i][p] dy[j][p].
template <typename T>
struct GradJob {
    const ExpertGradArgs &a;
    Tables tables;
    int tiles_i, tiles_j;

    __device__ int4 find(int n) const
    {
        const int t = int(blockIdx.x) + n * int(gridDim.x), e = t / (tiles_i * tiles_j);
        int i, j;
        tile_at(t - e * tiles_i * tiles_j, tiles_i * tiles_j, tiles_i, tiles_j, i, j);
        const int s0 = tables.offset[e] / RR_QUANT_BLOCK;
        return int4{e, i * T::TI | j * T::TJ << 16, s0, s0 + (tables.count[e] + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK};
    }
    __device__ Span span(int n) const
    {
        static_assert(RR_MAX_WIDTH <= 1 << 16, "a tile's first row and column take a word");
        const int4 v = n < kSpans ? tables.span[n] : find(n);
        const unsigned ij = unsigned(__builtin_amdgcn_readfirstlane(v.y));
        return Span{__builtin_amdgcn_readfirstlane(v.x), int(ij & 0xffff), int(ij >> 16), 0, 0,
                    __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
    }
    __device__ void first() const {}
    __device__ void open(typename T::Source &source, int n, bool) const
    {
        const Span s = span(n);
        const int rows_i = a.k - s.i0, rows_j = a.n - s.j0;
        const Eight x{a.x.values + s.i0 * a.x.ld, a.x.powers + s.i0 * a.x.lds, a.x.ld, a.x.lds};
        const Eight dy{a.dy.values + s.j0 * a.dy.ld, a.dy.powers + s.j0 * a.dy.lds, a.dy.ld, a.dy.lds};
        source.open(x, rows_i * x.ld, rows_i * x.lds, dy, rows_j * dy.ld, rows_j * dy.lds,
                    [&](int i) { return i < rows_i ? i : -1; }, [&](int j) { return j < rows_j ? j : -1; },
                    [&](int i) { return i < rows_i ? i : -1; }, s);
    }
    __device__ void end(const Span &s, int, const typename T::Acc &acc) const
    {
        void *out = static_cast<char *>(a.dw) + ((int64_t(s.e) * a.n + s.j0) * a.k + s.i0) * (T::kFull ? 4 : 2);
        store<T>(acc, out, a.k, a.n - s.j0, a.k - s.i0, [](int) { return 1.0f; });
    }
};

template <typename T>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void grad_kernel(ExpertGradArgs a, int tiles_i, int tiles_j)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const Tables tables = T::tables(lds, a.experts);
    fill_tables(tables, a.offset, a.count, a.experts, T::TJ);
    const GradJob<T> job{a, tables, tiles_i, tiles_j};
    T::run(job, own_tiles(job, tiles_i * tiles_j * a.experts), lds);
}

int tiles(int n, int per) { return n / per + (n % per != 0); }

template <bool BLOCK_A> using Big = Tile8<256, 256, 2, 2, BLOCK_A, false>;
template <bool BLOCK_A, bool FULL> using Mid = Tile8<128, 128, 2, 2, BLOCK_A, FULL>;

// Tiles of segments, at most: each expert with a choice may have one that is not full.
int64_t most_tiles(const ExpertProductArgs &a, int ti, int tj)
{
    return (a.choices / tj + (a.experts < a.choices ? a.experts : a.choices)) * int64_t(tiles(a.n, ti));
}

// As many workgroups as the 256 compute units hold at a time.
template <typename T>
unsigned grid_for(int64_t n)
{
    return unsigned(n < 256 * T::kPerUnit ? n : 256 * T::kPerUnit);
}

template <int FJ, int KS, int FI>
hipError_t narrow(const ExpertProductArgs &a, hipStream_t stream)
{
    const dim3 grid(unsigned(most_tiles(a, 16 * FI, 16 * FJ))), threads(KS * 64);
    if (a.bf16)
        narrow_kernel<FJ, false, KS, FI><<<grid, threads, 0, stream>>>(a, tiles(a.n, 16 * FI));
    else
        narrow_kernel<FJ, true, KS, FI><<<grid, threads, 0, stream>>>(a, tiles(a.n, 16 * FI));
    return hipGetLastError();
}

template <int FJ>
hipError_t narrow(const ExpertProductArgs &a, hipStream_t stream)
{
    // where that would leave compute units idle, smaller tiles and more parts of k (8
    // experts, 2048 x 1024: 6.8 us against 9 us)
    const int used = a.experts < a.choices ? a.experts : a.choices;
    return int64_t(used) * tiles(a.n, 64) >= 512 ? narrow<FJ, 2, 4>(a, stream) : narrow<FJ, 4, 2>(a, stream);
}

template <typename T>
hipError_t product(const ExpertProductArgs &a, hipStream_t stream)
{
    product_kernel<T><<<dim3(grid_for<T>(most_tiles(a, T::TI, T::TJ))), dim3(T::kThreads), T::lds_bytes(a.experts), stream>>>(a, tiles(a.n, T::TI));
    return hipGetLastError();
}

template <typename T>
hipError_t grad(const ExpertGradArgs &a, hipStream_t stream)
{
    const int ti = tiles(a.k, T::TI), tj = tiles(a.n, T::TJ);
    grad_kernel<T><<<dim3(grid_for<T>(int64_t(ti) * tj * a.experts)), dim3(T::kThreads), T::lds_bytes(a.experts), stream>>>(a, ti, tj);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_product(const Op &op, hipStream_t stream)
{
    const ExpertProductArgs a = op.get<ExpertProductArgs>();
    // choices of an expert, were they even
    const int used = a.experts < a.choices ? a.experts : a.choices, per = a.choices / used;
    (void)hipGetLastError();
    // Streaming wins where tiles through LDS would be too few for the 256 compute units:
    // 8 experts of 2048 x 1024, one choice each: 6.5 us and 15.2 us; 576 choices of 64 experts,
    // 2048 x 1408: 31 us and 22 us; with more choices each it reads them too often: 64 of each
    // of 8, 2048 x 2048: 35 us and 17 us, of 2, 2048 x 1024: 9.5 us and 13.9 us.
    // Counts are known on the device only, so that the rule takes them to be even.  Others cost
    // streaming up to 1.6 times as long (32 choices of 8 experts, 2048 x 1024: 6.4 us, half of
    // them one expert's 10.2 us, all of them 6.9 us), tiles next to nothing (16384 of 16, 2048 x
    // 1408: 61 us, 57 us and 56 us; 65536 of 32, 4096 x 2048: 510 us, 534 us and 459 us).
    if (per <= 64 && int64_t(used) * tiles(a.n, 128) <= (per <= 16 ? 512 : 96))
        return per <= 16 ? narrow<1>(a, stream) : per <= 32 ? narrow<2>(a, stream) : narrow<4>(a, stream);
    if (!a.bf16)
        return product<Mid<true, true>>(a, stream);
    // The busiest of 256 compute units has so many tiles; segments end in the middle of
    // one.  A large tile takes as long as 3.4 small ones, of which two share a unit: one alone
    // takes as long as 1.6 (65536 x 4096 x 2048 in 32 segments: 611 us with large tiles, 702 us
    // with small; 16384 x 2048 x 1408 in 16: 67 us and 59 us).
    const auto busy = [&](int t) {
        return ceil((double(a.choices) / t + 0.5 * used) * tiles(a.n, t) / 256);
    };
    const double large = 3.4 * busy(256), small = busy(128) > 1 ? busy(128) : 1.6;
    return large < small ? product<Big<true>>(a, stream) : product<Mid<true, false>>(a, stream);
}

hipError_t launch_expert_grad(const Op &op, hipStream_t stream)
{
    const ExpertGradArgs a = op.get<ExpertGradArgs>();
    (void)hipGetLastError();
    if (!a.bf16)
        return grad<Mid<false, true>>(a, stream);
    // Large tiles where each compute unit has eight or more: 65536 x 4096 x 2048 for 32 experts
    // 631 us, with small ones 794 us; for 16 experts of 2048 x 1408, three a unit, 81 us and
    // 69 us.
    if (int64_t(tiles(a.n, 256)) * tiles(a.k, 256) * a.experts < 2048)
        return grad<Mid<false, false>>(a, stream);
    return grad<Big<false>>(a, stream);
}

}  // namespace rr
