// rr_product.h -- one output tile of C[j][i] = sum_k A[i][k] B[j][k] on the
// gfx950 matrix cores, both operands with contiguous k.
//
// A workgroup of WI x WJ waves computes TI x TJ results in registers.  k goes
// by in steps of 128 bytes per row (64 bf16, 32 fp32).  STAGES steps of both
// operands are held in LDS; the loads of step t + STAGES - 1 are issued before
// step t is computed, and write LDS directly (buffer_load ... lds) without
// passing through registers.  A row's eight 16-byte chunks lie in LDS at chunk
// c ^ ((row >> 1) & 7): sixteen consecutive rows of one logical chunk then
// cover all 64 banks, which is what one fragment read touches.
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

// At most n vector memory operations outstanding.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4 | 15 << 8);
}

// The LDS address of a generic pointer into LDS (its low half).
__device__ __forceinline__ __attribute__((address_space(3))) void *lds_pointer(char *p)
{
    return reinterpret_cast<__attribute__((address_space(3))) void *>(uint32_t(reinterpret_cast<uintptr_t>(p)));
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

template <bool BF16, int TI_, int TJ_, int WI, int WJ, int STAGES, bool DIRECT>
struct Tile {
    static constexpr int TI = TI_, TJ = TJ_, kWaves = WI * WJ, kThreads = kWaves * 64;
    static constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;  // 16 x 16 results per wave
    static constexpr int kEs = BF16 ? 2 : 4, kStep = kRowBytes / kEs;
    static constexpr int kRows = 8 * kWaves;                    // rows of one load of the workgroup
    static constexpr int kLoadsA = TI / kRows, kLoadsB = (TJ + kRows - 1) / kRows;
    static constexpr int kLoads = kLoadsA + kLoadsB;
    static constexpr int kStageBytes = kLoads * kRows * kRowBytes;
    static constexpr int kLdsBytes = STAGES * kStageBytes;
    static_assert(TI % kRows == 0 && FI * WI * 16 == TI && FJ * WJ * 16 == TJ, "");

    struct Acc {
        f32x4 c[FI][FJ];
    };

    // First row of the wave's results, and of the lane's.
    __device__ static int wave_i() { return (threadIdx.x / 64) % WI * (FI * 16); }
    __device__ static int wave_j() { return (threadIdx.x / 64) / WI * (FJ * 16); }
    __device__ static int lane_i(int f) { return wave_i() + f * 16 + threadIdx.x % 64 / 16 * 4; }
    __device__ static int lane_j(int f) { return wave_j() + f * 16 + threadIdx.x % 16; }

    // Steps [s0, s1) of k of the tile at (i0, j0).
    __device__ static void run(const Product &p, int64_t i0, int64_t j0, int s0, int s1, char *lds, Acc &acc)
    {
        const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                acc.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        const int64_t lda = p.lda * kEs, ldb = p.ldb * kEs;
        const int rows_a = int(p.ni - i0 < TI ? p.ni - i0 : TI), rows_b = int(p.nj - j0 < TJ ? p.nj - j0 : TJ);
        const char *base_a = static_cast<const char *>(p.a) + i0 * lda, *base_b = static_cast<const char *>(p.b) + j0 * ldb;
        const int end = p.nk * kEs;
        // this lane's rows and chunks of each load
        int off[kLoads], chunk[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const bool is_a = n < kLoadsA;
            const int row = (is_a ? n : n - kLoadsA) * kRows + wave * 8 + lane / 8;
            chunk[n] = ((lane % 8) ^ ((row >> 1) & 7)) * 16;
            off[n] = row < (is_a ? rows_a : rows_b) ? int(row * (is_a ? lda : ldb)) + chunk[n] : kNowhere;
        }
        const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(base_a), (short)0, int(rows_a * lda), kBufferFormat);
        const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(base_b), (short)0, int(rows_b * ldb), kBufferFormat);

        u32x4 held[DIRECT ? 1 : kLoads];
        // Step s into its LDS buffer (DIRECT) or into registers; chunks past
        // the end of k and rows past the end of an operand become zeros.
        auto fetch = [&](int s) {
            const int k = s * kRowBytes;
            char *to = lds + s % STAGES * kStageBytes + wave * 1024;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const bool in = k + chunk[n] < end && s < s1;
                if constexpr (DIRECT) {
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(n < kLoadsA ? ra : rb, lds_pointer(to + n * kRows * kRowBytes),
                                                             16, in ? off[n] : kNowhere, k, 0, 0);
                } else {
                    held[n] = u32x4{0, 0, 0, 0};
                    if (in && off[n] != kNowhere)
                        held[n] = load_chunk<kEs>((n < kLoadsA ? base_a : base_b) + off[n] + k, end - k - chunk[n]);
                }
            }
        };
        auto commit = [&](int s) {
            char *to = lds + s % STAGES * kStageBytes + wave * 1024 + lane * 16;
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                *reinterpret_cast<u32x4 *>(to + n * kRows * kRowBytes) = held[DIRECT ? 0 : n];
        };
        // fragment reads: this lane's row and chunk in each half of a step
        const int frow = lane % 16;
        const int swz = (frow >> 1) & 7;
        const int at0 = frow * kRowBytes + ((lane / 16) ^ swz) * 16, at1 = frow * kRowBytes + ((4 + lane / 16) ^ swz) * 16;

        if constexpr (DIRECT) {
#pragma unroll
            for (int s = 0; s < STAGES - 1; ++s)
                fetch(s0 + s);
        } else {
            fetch(s0);
            commit(s0);
        }
        for (int s = s0; s < s1; ++s) {
            if constexpr (DIRECT) {
                wait_loads<(STAGES - 2) * kLoads>();
                __builtin_amdgcn_s_barrier();
                fetch(s + STAGES - 1);
            } else {
                __syncthreads();
                fetch(s + 1);
            }
            const char *stage = lds + s % STAGES * kStageBytes;
            const char *sa = stage + wave_i() * kRowBytes, *sb = stage + (kLoadsA * kRows + wave_j()) * kRowBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = h ? at1 : at0;
                u32x4 a[FI], b[FJ];
#pragma unroll
                for (int i = 0; i < FI; ++i)
                    a[i] = *reinterpret_cast<const u32x4 *>(sa + at + i * 16 * kRowBytes);
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    b[j] = *reinterpret_cast<const u32x4 *>(sb + at + j * 16 * kRowBytes);
#pragma unroll
                for (int i = 0; i < FI; ++i)
#pragma unroll
                    for (int j = 0; j < FJ; ++j) {
                        if constexpr (BF16) {
                            acc.c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, a[i]), __builtin_bit_cast(bf16x8, b[j]), acc.c[i][j], 0, 0, 0);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc.c[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(a[i][e]), __uint_as_float(b[j][e]), acc.c[i][j], 0, 0, 0);
                        }
                    }
            }
            if constexpr (!DIRECT)
                commit(s + 1);
        }
        // the loads past s1 have written zeros: LDS is free after this
        wait_loads<0>();
        __syncthreads();
    }
};

}  // namespace
}  // namespace rr
