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
// exactly, through the bf16 instructions (1e-8, at half the rate): FULL.
#include "rr_expert.h"
#include "rr_product.h"

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
    const int r = a.source[p] / a.topk;
    return r >= 0 && r < a.rows ? r : -1;
}

__device__ __forceinline__ float weight_of(const ExpertProductArgs &a, int p, bool in)
{
    if (!in || !a.weight)
        return 1.0f;
    const int n = a.source[p];
    return n >= 0 && n / a.topk < a.rows ? a.weight[n] : 0.0f;
}

// ---------------------------------------------------------------------------
// Few positions a segment: each of eight waves streams its share of k for 32 rows of
// the weights from memory to registers, and the sums are joined in LDS.
// ---------------------------------------------------------------------------

constexpr int kNarrowWaves = 8, kNarrowThreads = kNarrowWaves * 64, kNarrowI = 32;

struct Piece {
    i32x8 v;
    unsigned p;

    __device__ __forceinline__ void load(const unsigned char *at, const unsigned char *power)
    {
        u32x4 lo, hi;
        __builtin_memcpy(&lo, __builtin_assume_aligned(at, 16), 16);
        __builtin_memcpy(&hi, __builtin_assume_aligned(at + 16, 16), 16);
        v = i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
        p = *power;
    }
};

template <int FJ, bool FULL>
__global__ __launch_bounds__(kNarrowThreads) void narrow_kernel(ExpertProductArgs a, int tiles_i)
{
    constexpr int FI = kNarrowI / 16, TJ = 16 * FJ;
    __shared__ __attribute__((aligned(16))) f32x4 sums[kNarrowWaves][FI * FJ][64];
    Place at;
    if (!place_of(a.count, a.experts, TJ, tiles_i, at))
        return;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 16, g = lane / 16;
    const int blocks = int(a.w.ld / RR_QUANT_BLOCK), blocks_n = (a.n + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    const int i0 = at.i * kNarrowI, j0 = at.j * TJ, live = a.count[at.e] - j0, first = a.offset[at.e] + j0;
    const unsigned char *wv[FI], *wp[FI], *xv[FJ], *xp[FJ];
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        const int i = i0 + f * 16 + r < a.n ? i0 + f * 16 + r : a.n - 1;
        wv[f] = a.w.values + (int64_t(at.e) * a.n + i) * a.w.ld + g * 32;
        wp[f] = a.w.powers + (int64_t(at.e) * blocks_n + i / RR_QUANT_BLOCK) * a.w.lds;
    }
#pragma unroll
    for (int f = 0; f < FJ; ++f) {
        const int j = f * 16 + r, row = row_of(a, first + j, j < live), in = row < 0 ? 0 : row;
        xv[f] = a.x.values + int64_t(in) * a.x.ld + g * 32;
        xp[f] = a.x.powers + int64_t(in) * a.x.lds;
    }
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Piece wf[FI], xf[FJ];
    const auto load = [&](int b) {
#pragma unroll
        for (int f = 0; f < FI; ++f)
            wf[f].load(wv[f] + int64_t(b) * RR_QUANT_BLOCK, wp[f] + b);
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            xf[f].load(xv[f] + int64_t(b) * RR_QUANT_BLOCK, xp[f] + b);
    };
    if (wave < blocks)
        load(wave);
    for (int b = wave; b < blocks; b += kNarrowWaves) {
        Piece w0[FI], x0[FJ];
#pragma unroll
        for (int f = 0; f < FI; ++f)
            w0[f] = wf[f];
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            x0[f] = xf[f];
        if (b + kNarrowWaves < blocks)
            load(b + kNarrowWaves);
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
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            sums[wave][i * FJ + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = threadIdx.x; t < FI * FJ * 64; t += kNarrowThreads) {
        const int f = t / 64, l = t % 64, j = f % FJ * 16 + l % 16, i = i0 + f / FJ * 16 + l / 16 * 4;
        if (j >= live || i >= a.n)
            continue;
        f32x4 s = sums[0][f][l];
#pragma unroll
        for (int w = 1; w < kNarrowWaves; ++w)
            s += sums[w][f][l];
        s *= weight_of(a, first + j, true);
        const int64_t to = int64_t(first + j) * a.n + i;
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (i + n < a.n) {
                if constexpr (!FULL)
                    static_cast<unsigned short *>(a.out)[to + n] = (unsigned short)pack_bf16(s[n], 0.0f);
                else
                    static_cast<float *>(a.out)[to + n] = s[n];
            }
    }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------

// One tile of C[j][i] = sum_k A[i][k] B[j][k].  Two steps of k, of 128 elements each,
// lie in LDS in the layout of Tile (rr_product.h); a lane's 32 bytes of a row are its
// chunks g and g + 4.  Powers come four steps at a time, a word for each row of the
// tile.  A step is computed in two halves of the rows i.  While the first runs, the
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
    static constexpr int kLdsBytes = 2 * kStageBytes + 2 * kPowerBytes;
    // waves a SIMD has room for, which the registers are divided by
    static constexpr int kPerSimd = 160 * 1024 / kLdsBytes * kWaves / 4;
    static_assert(kLoadsP * kThreads == TI + TJ && TI % 64 == 0, "a wave loads the powers of one operand");
    static_assert(!BLOCK_A || RR_QUANT_BLOCK % (FI * 16) == 0, "");
    static_assert(FJ >= 4 && H >= 1, "");
    static constexpr bool kFull = FULL;  // results in 32 bits
    // results leave as those of a product in bf16 and fp32 do
    template <bool BF16>
    using Out = Tile<BF16, TI, TJ, WI, WJ, 2, true>;

    __amdgpu_buffer_rsrc_t a, b, power[kLoadsP];
    int off_a[kLoadsA], off_b[kLoadsB], off_power[kLoadsP];
    char *lds;
    int s0, s1;

    // Bytes of a buffer from its first row on, below kNowhere.
    __device__ static __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t bytes)
    {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0,
                                                 int(bytes < kNowhere ? bytes : kNowhere), kBufferFormat);
    }

    // ra(i), rb(j): the rows in the buffers of the tile's rows, -1 for none; pa: the same in
    // A's powers.
    template <typename RA, typename RB, typename PA>
    __device__ void start(const Eight &x, int64_t bytes_a, int64_t power_a, const Eight &y, int64_t bytes_b,
                          int64_t power_b, RA ra, RB rb, PA pa, int first, int last, char *buffer_lds)
    {
        const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
        lds = buffer_lds;
        s0 = first;
        s1 = last;
        a = buffer(x.values, bytes_a);
        b = buffer(y.values, bytes_b);
        const int row0 = wave * 8 + lane / 8, chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;
#pragma unroll
        for (int l = 0; l < kLoadsA; ++l) {
            const int r = ra(l * kRows + row0);
            off_a[l] = r >= 0 ? int(r * x.ld) + chunk : kNowhere;
        }
#pragma unroll
        for (int l = 0; l < kLoadsB; ++l) {
            const int r = rb(l * kRows + row0);
            off_b[l] = r >= 0 ? int(r * y.ld) + chunk : kNowhere;
        }
#pragma unroll
        for (int l = 0; l < kLoadsP; ++l) {
            const int row = l * kThreads + int(threadIdx.x);
            const bool of_a = l * kThreads + __builtin_amdgcn_readfirstlane(wave) * 64 < TI;
            power[l] = of_a ? buffer(x.powers, power_a) : buffer(y.powers, power_b);
            const int r = of_a ? pa(row) : rb(row - TI);
            off_power[l] = r >= 0 ? int(r * (of_a ? x.lds : y.lds)) : kNowhere;
        }
        fetch_powers(s0 / 4);
        if (s0 % 4 == 3)
            fetch_powers(s0 / 4 + 1);
        fetch(s0);
        fetch(s0 + 1);
    }
    __device__ void fetch(int s) const
    {
        char *to = lds + s % 2 * kStageBytes + threadIdx.x / 64 * 1024;
        const bool in = s < s1;
        const int k = in ? s * kRowBytes : 0;
#pragma unroll
        for (int l = 0; l < kLoadsA; ++l)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a, lds_pointer(to + l * kLoadBytes), 16, in ? off_a[l] : kNowhere, k, 0, 0);
#pragma unroll
        for (int l = 0; l < kLoadsB; ++l)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds_pointer(to + (kLoadsA + l) * kLoadBytes), 16,
                                                     in ? off_b[l] : kNowhere, k, 0, 0);
    }
    __device__ char *powers(int group) const { return lds + 2 * kStageBytes + group % 2 * kPowerBytes; }
    // Four steps' powers, from step 4 * group on.
    __device__ void fetch_powers(int group) const
    {
        const bool in = 4 * group < s1;
#pragma unroll
        for (int l = 0; l < kLoadsP; ++l)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(power[l], lds_pointer(powers(group) + (l * kThreads + threadIdx.x / 64 * 64) * 4), 4,
                                                     in ? off_power[l] : kNowhere, in ? group * 4 : 0, 0, 0);
    }

    __device__ static int wave_i() { return (threadIdx.x / 64) % WI * (FI * 16); }
    __device__ static int wave_j() { return (threadIdx.x / 64) / WI * (FJ * 16); }

    __device__ static i32x8 fragment(const char *stage, int f)
    {
        const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
        struct {
            u32x4 lo, hi;
        } v;
        v.lo = *reinterpret_cast<const u32x4 *>(stage + (f + r) * kRowBytes + (g ^ (r >> 1)) * 16);
        v.hi = *reinterpret_cast<const u32x4 *>(stage + (f + r) * kRowBytes + ((4 + g) ^ (r >> 1)) * 16);
        return __builtin_bit_cast(i32x8, v);
    }
    __device__ i32x8 read_a(int s, int f) const { return fragment(lds + s % 2 * kStageBytes, wave_i() + f * 16); }
    __device__ i32x8 read_b(int s, int f) const
    {
        return fragment(lds + s % 2 * kStageBytes + kLoadsA * kLoadBytes, wave_j() + f * 16);
    }

    static constexpr int kPowersA = BLOCK_A ? 1 : FI;
    struct Powers {
        unsigned a[kPowersA], b[FJ];
    };
    __device__ void read_powers(int s, Powers &p) const
    {
        const unsigned *at = reinterpret_cast<const unsigned *>(powers(s / 4)) + threadIdx.x % 16;
#pragma unroll
        for (int f = 0; f < kPowersA; ++f)
            p.a[f] = at[wave_i() + f * 16];
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            p.b[f] = at[TI + wave_j() + f * 16];
    }
    // The powers of step s in the low bytes.
    __device__ static void shift(const Powers &from, int s, Powers &to)
    {
#pragma unroll
        for (int f = 0; f < kPowersA; ++f)
            to.a[f] = from.a[f] >> s % 4 * 8;
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            to.b[f] = from.b[f] >> s % 4 * 8;
    }
    struct Acc {
        f32x4 c[FI][FJ];
    };

    // This step has been read by all, and the next one has arrived.
    __device__ void advance(int s, Powers &raw) const
    {
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        fetch(s + 2);
        if ((s + 2) % 4 == 0)
            fetch_powers((s + 2) / 4);
        if ((s + 1) % 4 == 0)
            read_powers(s + 1, raw);
    }

    // acc += the products of steps [s0, s1), of which there is at least one
    __device__ void finish(Acc &acc) const
    {
        i32x8 fa[FI], fb[FJ];
        Powers raw, at;
        wait_loads<kLoadsA + kLoadsB>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            fb[f] = read_b(s0, f);
#pragma unroll
        for (int f = 0; f < (FULL ? FI : H); ++f)
            fa[f] = read_a(s0, f);
        read_powers(s0, raw);
        if constexpr (FULL) {
            for (int s = s0; s < s1; ++s) {
                shift(raw, s, at);
                Wide wb[FJ];
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    wb[j].set(fb[j], at.b[j]);
#pragma unroll
                for (int i = 0; i < FI; ++i) {
                    Wide wa;
                    wa.set(fa[i], at.a[BLOCK_A ? 0 : i]);
#pragma unroll
                    for (int j = 0; j < FJ; ++j)
                        multiply(wa, wb[j], acc.c[i][j]);
                    if (i == 0)
                        advance(s, raw);
                    if (i == 0 || i == 1) {
#pragma unroll
                        for (int f = i * FJ / 2; f < (i + 1) * FJ / 2; ++f)
                            fb[f] = read_b(s + 1, f);
                    }
                    fa[i] = read_a(s + 1, i);
                }
            }
        } else {
            for (int s = s0; s < s1; ++s) {
                shift(raw, s, at);
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        multiply<0, 0>(fa[i], fb[j], acc.c[i][j], at.a[BLOCK_A ? 0 : i], at.b[j]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (j < (H + 1) / 2) {
#pragma unroll
                        for (int f = H + 2 * j; f < H + 2 * j + 2 && f < FI; ++f)
                            fa[f] = read_a(s, f);
                    }
                }
                constexpr int kAt = FJ / 4 - 1;  // the barrier: after this column of the second half
#pragma unroll
                for (int j = 0; j < FJ; ++j) {
#pragma unroll
                    for (int i = H; i < FI; ++i)
                        multiply<0, 0>(fa[i], fb[j], acc.c[i][j], at.a[BLOCK_A ? 0 : i], at.b[j]);
                    if (j == kAt) {
                        advance(s, raw);
#pragma unroll
                        for (int f = 0; f < kAt; ++f)
                            fb[f] = read_b(s + 1, f);
                    }
                    if (j >= kAt) {
                        fb[j] = read_b(s + 1, j);
                        constexpr int kOver = FJ - 1 - kAt;  // a's first half over the columns left
#pragma unroll
                        for (int f = (j - kAt) * H / kOver; f < (j - kAt + 1) * H / kOver && f < H; ++f)
                            fa[f] = read_a(s + 1, f);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // the loads past s1 have written zeros: LDS is free after this
        wait_loads<0>();
        __syncthreads();
    }
};

// The lane's results of row j (fragment f, of the wave's) to out, the tile's first i.
template <typename T>
__device__ __forceinline__ void store(const typename T::Acc &acc, int f, void *out, int64_t at, int left, float by)
{
    f32x4 v[T::FI];
#pragma unroll
    for (int i = 0; i < T::FI; ++i)
        v[i] = acc.c[i][f] * by;
    T::template Out<!T::kFull>::store_row(static_cast<char *>(out) + at * (T::kFull ? 4 : 2), v, left);
}

template <typename T>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void product_kernel(ExpertProductArgs a, int tiles_i)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    Place at;
    if (!place_of(a.count, a.experts, T::TJ, tiles_i, at))
        return;
    const int blocks_n = (a.n + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    const int i0 = at.i * T::TI, j0 = at.j * T::TJ, live = a.count[at.e] - j0, first = a.offset[at.e] + j0;
    const int rows_i = a.n - i0;
    // from the tile's first row on; gathered rows may be anywhere
    const Eight w{a.w.values + (int64_t(at.e) * a.n + i0) * a.w.ld,
                  a.w.powers + (int64_t(at.e) * blocks_n + i0 / RR_QUANT_BLOCK) * a.w.lds, a.w.ld, a.w.lds};
    const int base = a.gather ? 0 : first;
    const Eight x{a.x.values + base * a.x.ld, a.x.powers + base * a.x.lds, a.x.ld, a.x.lds};
    const int64_t rows_x = a.gather ? a.rows : live;
    T t;
    t.start(w, rows_i * w.ld, (blocks_n - i0 / RR_QUANT_BLOCK) * w.lds, x, rows_x * x.ld, rows_x * x.lds,
            [&](int i) { return i < rows_i ? i : -1; },
            [&](int j) {
                const int r = row_of(a, first + j, j < live);
                return r < 0 ? -1 : r - base;
            },
            [&](int i) { return i < rows_i ? i / RR_QUANT_BLOCK : -1; }, 0, int(a.w.ld / RR_QUANT_BLOCK), lds);
    typename T::Acc acc;
#pragma unroll
    for (int i = 0; i < T::FI; ++i)
#pragma unroll
        for (int j = 0; j < T::FJ; ++j)
            acc.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    t.finish(acc);
#pragma unroll
    for (int f = 0; f < T::FJ; ++f) {
        const int j = T::wave_j() + f * 16 + int(threadIdx.x % 16);
        const int p = first + j, left = j < live ? rows_i : 0;
        const float by = weight_of(a, p, j < live);
        const int64_t to = int64_t(p) * a.n + i0;
        store<T>(acc, f, a.out, to, left, by);
    }
}

// dw[e][j][i] = sum over the segment's positions of x[i][p] dy[j][p].
template <typename T>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void grad_kernel(ExpertGradArgs a, int tiles_i, int tiles_j)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int e = blockIdx.x / (tiles_i * tiles_j);
    int ti, tj;
    tile_at(int(blockIdx.x) - e * tiles_i * tiles_j, tiles_i * tiles_j, tiles_i, tiles_j, ti, tj);
    const int i0 = ti * T::TI, j0 = tj * T::TJ, rows_i = a.k - i0, rows_j = a.n - j0;
    const int s0 = a.offset[e] / RR_QUANT_BLOCK, steps = (a.count[e] + RR_QUANT_BLOCK - 1) / RR_QUANT_BLOCK;
    typename T::Acc acc;
#pragma unroll
    for (int i = 0; i < T::FI; ++i)
#pragma unroll
        for (int j = 0; j < T::FJ; ++j)
            acc.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (steps > 0) {
        const Eight x{a.x.values + i0 * a.x.ld, a.x.powers + i0 * a.x.lds, a.x.ld, a.x.lds};
        const Eight dy{a.dy.values + j0 * a.dy.ld, a.dy.powers + j0 * a.dy.lds, a.dy.ld, a.dy.lds};
        T t;
        t.start(x, rows_i * x.ld, rows_i * x.lds, dy, rows_j * dy.ld, rows_j * dy.lds,
                [&](int i) { return i < rows_i ? i : -1; }, [&](int j) { return j < rows_j ? j : -1; },
                [&](int i) { return i < rows_i ? i : -1; }, s0, s0 + steps, lds);
        t.finish(acc);
    }
#pragma unroll
    for (int f = 0; f < T::FJ; ++f) {
        const int j = j0 + T::wave_j() + f * 16 + int(threadIdx.x % 16);
        const int left = j < a.n ? rows_i : 0;
        const int64_t to = (int64_t(e) * a.n + j) * a.k + i0;
        store<T>(acc, f, a.dw, to, left, 1.0f);
    }
}

int tiles(int n, int per) { return n / per + (n % per != 0); }

template <bool BLOCK_A> using Big = Tile8<256, 256, 2, 2, BLOCK_A, false>;
template <bool BLOCK_A, bool FULL> using Mid = Tile8<128, 128, 2, 2, BLOCK_A, FULL>;

// Tiles of segments: each expert with a choice may have one that is not full.
unsigned grid_of(const ExpertProductArgs &a, int ti, int tj)
{
    const int64_t j = a.choices / tj + (a.experts < a.choices ? a.experts : a.choices);
    return unsigned(j * tiles(a.n, ti));
}

template <int FJ>
hipError_t narrow(const ExpertProductArgs &a, hipStream_t stream)
{
    const dim3 grid(grid_of(a, kNarrowI, 16 * FJ)), threads(kNarrowThreads);
    if (a.bf16)
        narrow_kernel<FJ, false><<<grid, threads, 0, stream>>>(a, tiles(a.n, kNarrowI));
    else
        narrow_kernel<FJ, true><<<grid, threads, 0, stream>>>(a, tiles(a.n, kNarrowI));
    return hipGetLastError();
}

template <typename T>
hipError_t product(const ExpertProductArgs &a, hipStream_t stream)
{
    product_kernel<T><<<dim3(grid_of(a, T::TI, T::TJ)), dim3(T::kThreads), T::kLdsBytes, stream>>>(a, tiles(a.n, T::TI));
    return hipGetLastError();
}

template <typename T>
hipError_t grad(const ExpertGradArgs &a, hipStream_t stream)
{
    const int ti = tiles(a.k, T::TI), tj = tiles(a.n, T::TJ);
    grad_kernel<T><<<dim3(unsigned(ti) * unsigned(tj) * unsigned(a.experts)), dim3(T::kThreads), T::kLdsBytes, stream>>>(a, ti, tj);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_product(const Op &op, hipStream_t stream)
{
    const ExpertProductArgs a = op.get<ExpertProductArgs>();
    // choices of an expert, were they even
    const int per = a.choices / (a.experts < a.choices ? a.experts : a.choices);
    (void)hipGetLastError();
    if (per <= 16)
        return narrow<1>(a, stream);
    if (per <= 32)
        return narrow<2>(a, stream);
    if (per <= 64)
        return narrow<4>(a, stream);
    if (!a.bf16)
        return product<Mid<true, true>>(a, stream);
    if (per <= 192)
        return product<Mid<true, false>>(a, stream);
    return product<Big<true>>(a, stream);
}

hipError_t launch_expert_grad(const Op &op, hipStream_t stream)
{
    const ExpertGradArgs a = op.get<ExpertGradArgs>();
    (void)hipGetLastError();
    if (!a.bf16)
        return grad<Mid<false, true>>(a, stream);
    if (int64_t(a.n) * a.k * a.experts < int64_t(256) * 256 * 256)
        return grad<Mid<false, false>>(a, stream);
    return grad<Big<false>>(a, stream);
}

}  // namespace rr
