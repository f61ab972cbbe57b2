// rr_product.h -- one output tile of C[j][i] = sum_k A[i][k] B[j][k] on the
// gfx950 matrix cores.  Either operand lies with contiguous k, or "tall", with
// contiguous i or j.
//
// A workgroup of WI x WJ waves computes TI x TJ results in registers.  k goes
// by in steps of 64 bf16 or 32 fp32.  STAGES steps of both operands are held in
// LDS; loads write LDS directly (buffer_load ... lds) without passing through
// registers.  A step is computed in two halves.  While the first runs, the
// second's fragments are read; a quarter into the second, one barrier says that
// this step has been read by all and that the next one has arrived, the loads
// of step s + STAGES go out and the next first half's fragments are read, so
// that the matrix instructions find theirs in registers.
//
// LDS layout of a step with contiguous k: 128 bytes per row, the eight 16-byte
// chunks at chunk c ^ ((row >> 1) & 7); sixteen consecutive rows of one logical
// chunk then cover all 64 banks, which is what one fragment read touches.
// Tall: one row per k as wide as the tile, chunk c at c ^ f(k).  bf16 fragments
// are read transposed (ds_read_b64_tr_b16: sixteen lanes read four rows of 32
// bytes, each lane gets a column), f(k) = 2 (k % 4 + 4 (k / 8 % 2)) sets eight
// such rows side by side; fp32 ones by the element, f(k) = 4 (k / 4 % 4).
//
// Measured: logits of 8192 x 4096 x 128000 in bf16 in 6.2 ms, 1376 TFLOP/s, the
// matrix units busy 62% of the time at the 1.9 GHz that the card then
// holds; with the fragments read where they are used, and the barrier between
// steps, 6.8 ms.  fp32 2048 x 1024 x 16384: 116 TFLOP/s.
//
// fp32 elements go through the fp32 matrix instructions.  A lane's 16-byte
// fragment holds four consecutive k there, used by four instructions in turn;
// both operands are permuted alike, which leaves the sum as it is.
#pragma once

#include "rr_loss.h"

namespace rr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRowBytes = 128;
constexpr int kBufferFormat = 0x00020000;  // raw buffer: 32-bit data format, no swizzle
constexpr int kNowhere = 0x7fff0000;       // a byte offset past the end of every buffer

// At most N vector memory operations outstanding, and no LDS operation.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N < 64, "");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4 | 0 << 8);
}

// The LDS address of a generic pointer into LDS (its low half).
__device__ __forceinline__ __attribute__((address_space(3))) void *lds_pointer(char *p)
{
    return reinterpret_cast<__attribute__((address_space(3))) void *>(uint32_t(reinterpret_cast<uintptr_t>(p)));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 *LdsTile;

// Sixteen lanes read four rows of 32 bytes, 8 bytes each; a lane gets its column
// of the four.  The restricted pointer tells the compiler that loads into LDS
// under way do not concern this read, for which it would wait otherwise.
__device__ __forceinline__ s16x4 read_transposed(LdsTile __restrict p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// Sixteen bytes at any element alignment, zeros from byte `left` on.
template <int ES>
__device__ __forceinline__ u32x4 load_chunk(const char *p, int left)
{
    u32x4 v{0, 0, 0, 0};
    if (left >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 16 / ES - 1; ++e)
            if (e * ES < left) {
                if constexpr (ES == 2)
                    v[e / 2] |= unsigned(reinterpret_cast<const unsigned short *>(p)[e]) << 16 * (e % 2);
                else
                    v[e] = reinterpret_cast<const unsigned *>(p)[e];
            }
    }
    return v;
}

// Sixteen bytes to any element alignment, the first `left` of them.
template <int ES>
__device__ __forceinline__ void store_chunk(char *p, u32x4 v, int left)
{
    if (left >= 16) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 16 / ES - 1; ++e)
            if (e * ES < left) {
                if constexpr (ES == 2)
                    reinterpret_cast<unsigned short *>(p)[e] = (unsigned short)(v[e / 2] >> 16 * (e % 2));
                else
                    reinterpret_cast<unsigned *>(p)[e] = v[e];
            }
    }
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Which tile a workgroup computes.  Consecutive workgroups go to the eight
// dies in turn; each die gets a contiguous range of an order that walks i for
// kGroup rows of tiles at a time, so that the tiles a die runs at once share
// their operands in its L2.
constexpr int kGroup = 4;

__device__ __forceinline__ void tile_at(int b, int n, int tiles_i, int tiles_j, int &i, int &j)
{
    const int per = n / 8, id = b < per * 8 ? b % 8 * per + b / 8 : b;
    const int group = id / (kGroup * tiles_i), in = id - group * kGroup * tiles_i;
    const int left = tiles_j - group * kGroup, wide = left < kGroup ? left : kGroup;
    i = in / wide;
    j = group * kGroup + in % wide;
}

template <bool BF16, int TI_, int TJ_, int WI, int WJ, int STAGES, bool DIRECT, bool TALL_A = false, bool TALL_B = false>
struct Tile {
    static constexpr int TI = TI_, TJ = TJ_, kWaves = WI * WJ, kThreads = kWaves * 64;
    static constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;  // 16 x 16 results per wave
    static constexpr int kEs = BF16 ? 2 : 4, kStep = kRowBytes / kEs;
    static constexpr int kRows = 8 * kWaves;                    // rows of one load of the workgroup
    static constexpr int kLoadBytes = kRows * kRowBytes;
    static constexpr int kLoadsA = TI / kRows, kLoadsB = (TJ + kRows - 1) / kRows;
    static constexpr int kLoads = kLoadsA + kLoadsB;
    static constexpr int kStageBytes = kLoads * kLoadBytes;
    static constexpr int kLdsBytes = STAGES * kStageBytes;
    static_assert(TI % kRows == 0 && FI * WI * 16 == TI && FJ * WJ * 16 == TJ, "");
    static_assert(DIRECT || !(TALL_A || TALL_B), "");
    static_assert(!TALL_A || TI * kEs >= 256, "a tall row has to hold the swizzle");
    static_assert(!TALL_B || (TJ * kEs >= 256 && TJ % kRows == 0), "");

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

    // First row of the wave's results, and of the lane's.
    __device__ static int wave_i() { return (threadIdx.x / 64) % WI * (FI * 16); }
    __device__ static int wave_j() { return (threadIdx.x / 64) / WI * (FJ * 16); }
    __device__ static int lane_i(int f) { return wave_i() + f * 16 + threadIdx.x % 64 / 16 * 4; }
    __device__ static int lane_j(int f) { return wave_j() + f * 16 + threadIdx.x % 16; }

    // One operand: W rows of the tile, n in all from row r0 on.
    template <bool TALL, int W, int LOADS>
    struct Side {
        const char *base;
        int64_t ld;       // bytes
        int off[LOADS];   // this lane's byte offsets within a step
        int chunk;        // of k, TALL: unused
        int left;         // bytes of base: of all steps, TALL: of the row
        int nk;
        __amdgpu_buffer_rsrc_t whole;

        __device__ void init(const void *p, int64_t stride, int n, int64_t r0, int k)
        {
            const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
            ld = stride * kEs;
            nk = k;
            const int rows = int(n - r0 < W ? n - r0 : W);
            if constexpr (TALL) {
                constexpr int kWide = W * kEs;
                base = static_cast<const char *>(p) + r0 * kEs;
                left = (rows * kEs + 15) / 16 * 16;
#pragma unroll
                for (int l = 0; l < LOADS; ++l) {
                    const int at = l * kLoadBytes + wave * 1024 + lane * 16, row = at / kWide;
                    const int f = BF16 ? 2 * (row % 4 + 4 * (row / 8 % 2)) : 4 * (row / 4 % 4);
                    const int c = ((at % kWide / 16) ^ f) * 16;
                    off[l] = c < left && row * ld < kNowhere - kRowBytes * W ? int(row * ld) + c : kNowhere;
                }
                chunk = 0;
            } else {
                base = static_cast<const char *>(p) + r0 * ld;
                const int row0 = wave * 8 + lane / 8;
                chunk = ((lane % 8) ^ ((row0 >> 1) & 7)) * 16;   // kRows is a multiple of 16
#pragma unroll
                for (int l = 0; l < LOADS; ++l) {
                    const int row = l * kRows + row0;
                    off[l] = row < rows ? int(row * ld) + chunk : kNowhere;
                }
                left = int(rows * ld);
                whole = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), (short)0, left, kBufferFormat);
            }
        }
        // Step s to LDS; what lies past k, past the operand, or in a step that
        // is not wanted becomes zeros.
        __device__ void fetch(int s, bool wanted, char *to) const
        {
            if constexpr (TALL) {
                const int64_t k0 = int64_t(s) * kStep;
                const int rows = nk - k0 < kStep ? int(nk - k0) : kStep;
                // bytes from this step's first to the operand's last
                const int have = wanted && rows > 0 ? int((rows - 1) * ld) + left : 0;
                const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<char *>(base + (wanted ? k0 * ld : 0)), (short)0, have, kBufferFormat);
#pragma unroll
                for (int l = 0; l < LOADS; ++l)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_pointer(to + l * kLoadBytes), 16, off[l], 0, 0, 0);
            } else {
                const int k = s * kRowBytes;
                const bool in = k + chunk < nk * kEs && wanted;
#pragma unroll
                for (int l = 0; l < LOADS; ++l)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(whole, lds_pointer(to + l * kLoadBytes), 16,
                                                             in ? off[l] : kNowhere, k, 0, 0);
            }
        }
        // The same through registers, for operands at any element alignment.
        __device__ void hold(int s, bool wanted, u32x4 *held) const
        {
            const int k = s * kRowBytes, end = nk * kEs;
#pragma unroll
            for (int l = 0; l < LOADS; ++l) {
                held[l] = u32x4{0, 0, 0, 0};
                if (k + chunk < end && wanted && off[l] != kNowhere)
                    held[l] = load_chunk<kEs>(base + off[l] + k, end - k - chunk);
            }
        }
        // This lane's part of 16 rows from row f on, of half h.
        __device__ static u32x4 fragment(const char *stage, int f, int h)
        {
            const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
            if constexpr (!TALL) {
                return *reinterpret_cast<const u32x4 *>(stage + (f + r) * kRowBytes + ((4 * h + g) ^ (r >> 1)) * 16);
            } else if constexpr (BF16) {
                const char *at = stage + (32 * h + 8 * g + r / 4) * (W * 2) +
                                 ((f / 8) ^ (2 * (r / 4 + 4 * (g % 2)))) * 16 + r % 4 * 8;
                struct {
                    s16x4 lo, hi;
                } v;
                v.lo = read_transposed((LdsTile)lds_pointer(const_cast<char *>(at)));
                v.hi = read_transposed((LdsTile)lds_pointer(const_cast<char *>(at + 4 * W * 2)));
                return __builtin_bit_cast(u32x4, v);
            } else {
                const char *at = stage + (16 * h + 4 * g) * (W * 4) + ((f / 4) ^ (4 * g)) * 16 + r * 4;
                u32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = *reinterpret_cast<const unsigned *>(at + e * W * 4);
                return v;
            }
        }
    };

    __device__ static void multiply(const u32x4 &a, const u32x4 &b, f32x4 &c)
    {
        if constexpr (BF16) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
        }
    }

    // Steps [s0, s1) of k of the tile at (i0, j0): start() sends its first loads,
    // finish() computes it.  What needs none of the tile's LDS can stand between.
    struct Pipe {
        Side<TALL_A, TI, kLoadsA> a;
        Side<TALL_B, TJ, kLoadsB> b;
        char *lds;
        int s0, s1;

        __device__ void fetch(int s) const
        {
            char *to = lds + s % STAGES * kStageBytes + threadIdx.x / 64 * 1024;
            a.fetch(s, s < s1, to);
            b.fetch(s, s < s1, to + kLoadsA * kLoadBytes);
        }
        __device__ void hold(int s, u32x4 *ha, u32x4 *hb) const
        {
            a.hold(s, s < s1, ha);
            b.hold(s, s < s1, hb);
        }
        __device__ void commit(int s, const u32x4 *ha, const u32x4 *hb) const
        {
            char *to = lds + s % STAGES * kStageBytes + threadIdx.x * 16;
#pragma unroll
            for (int l = 0; l < kLoadsA; ++l)
                *reinterpret_cast<u32x4 *>(to + l * kLoadBytes) = ha[l];
#pragma unroll
            for (int l = 0; l < kLoadsB; ++l)
                *reinterpret_cast<u32x4 *>(to + (kLoadsA + l) * kLoadBytes) = hb[l];
        }
        // Fragment n of a half: first B's, then A's.
        __device__ void read(int s, int h, u32x4 *fa, u32x4 *fb, int n) const
        {
            const char *stage = lds + s % STAGES * kStageBytes;
            if (n < FJ)
                fb[n] = decltype(b)::fragment(stage + kLoadsA * kLoadBytes, wave_j() + n * 16, h);
            else if (n < FJ + FI)
                fa[n - FJ] = decltype(a)::fragment(stage, wave_i() + (n - FJ) * 16, h);
        }

        __device__ void start(const Product &p, int64_t i0, int64_t j0, int first, int last, char *buffer)
        {
            lds = buffer;
            s0 = first;
            s1 = last;
            a.init(p.a, p.lda, p.ni, i0, p.nk);
            b.init(p.b, p.ldb, p.nj, j0, p.nk);
            if constexpr (DIRECT) {
#pragma unroll
                for (int s = 0; s < STAGES; ++s)
                    fetch(s0 + s);
            } else {
                u32x4 ha[kLoadsA], hb[kLoadsB];
                hold(s0, ha, hb);
                commit(s0, ha, hb);
            }
        }

        // acc += the tile's products
        __device__ void finish(Acc &acc) const
        {
            constexpr int kReads = FI + FJ;
            if constexpr (DIRECT) {
                constexpr int kAt = (FI + 3) / 4 - 1;  // the barrier: after this row of the second half
                constexpr int kPer = (kReads + FI - 1) / FI, kPerNext = (kReads + FI - 2 - kAt) / (FI - 1 - kAt);
                u32x4 a0[FI], b0[FJ], a1[FI], b1[FJ];
                wait_loads<(STAGES - 1) * kLoads>();
                __builtin_amdgcn_s_barrier();
#pragma unroll
                for (int n = 0; n < kReads; ++n)
                    read(s0, 0, a0, b0, n);
                for (int s = s0; s < s1; ++s) {
#pragma unroll
                    for (int i = 0; i < FI; ++i) {
#pragma unroll
                        for (int j = 0; j < FJ; ++j)
                            multiply(a0[i], b0[j], acc.c[i][j]);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int n = 0; n < kPer; ++n)
                            read(s, 1, a1, b1, i * kPer + n);
                    }
#pragma unroll
                    for (int i = 0; i < FI; ++i) {
#pragma unroll
                        for (int j = 0; j < FJ; ++j)
                            multiply(a1[i], b1[j], acc.c[i][j]);
                        if (i == kAt) {
                            wait_loads<(STAGES - 2) * kLoads>();
                            __builtin_amdgcn_s_barrier();
                            fetch(s + STAGES);
                        }
                        if (i >= kAt) {
#pragma unroll
                            for (int n = 0; n < kPerNext; ++n)
                                read(s + 1, 0, a0, b0, (i - kAt) * kPerNext + n);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            } else {
                for (int s = s0; s < s1; ++s) {
                    u32x4 ha[kLoadsA], hb[kLoadsB];
                    __syncthreads();
                    hold(s + 1, ha, hb);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        u32x4 fa[FI], fb[FJ];
#pragma unroll
                        for (int n = 0; n < kReads; ++n)
                            read(s, h, fa, fb, n);
#pragma unroll
                        for (int i = 0; i < FI; ++i)
#pragma unroll
                            for (int j = 0; j < FJ; ++j)
                                multiply(fa[i], fb[j], acc.c[i][j]);
                    }
                    commit(s + 1, ha, hb);
                }
            }
            // the loads past s1 have written zeros: LDS is free after this
            wait_loads<0>();
            __syncthreads();
        }
    };

    // The lane's row j of the wave's results, v, to out (at the tile's first
    // i), `left` of them from there on.  bf16 lanes 16 apart swap halves of two
    // neighbouring fragments, which makes 16 bytes per lane and 64 per row.
    __device__ static void store_row(char *out, const f32x4 *v, int left)
    {
        const int g = threadIdx.x % 64 / 16;
        if constexpr (BF16) {
#pragma unroll
            for (int f = 0; f < FI; f += 2) {
                u32x4 w;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16(v[f][2 * n], v[f][2 * n + 1]),
                                                                    pack_bf16(v[f + 1][2 * n], v[f + 1][2 * n + 1]), false, false);
                    w[n] = s[0];
                    w[2 + n] = s[1];
                }
                const int i = wave_i() + (f + g % 2) * 16 + g / 2 * 8;
                if (i < left)
                    store_chunk<2>(out + i * 2, w, (left - i) * 2);
            }
        } else {
#pragma unroll
            for (int f = 0; f < FI; ++f) {
                const int i = wave_i() + f * 16 + g * 4;
                if (i < left)
                    store_chunk<4>(out + i * 4, __builtin_bit_cast(u32x4, v[f]), (left - i) * 4);
            }
        }
    }
    // Whether store_row has this lane write result i of the wave's.
    __device__ static bool stores(int i)
    {
        const int g = threadIdx.x % 64 / 16;
        return i >= 0 && i < FI * 16 && g == (BF16 ? i / 16 % 2 + i % 16 / 8 * 2 : i % 16 / 4);
    }
};

}  // namespace
}  // namespace rr
