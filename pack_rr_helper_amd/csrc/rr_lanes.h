// rr_lanes.h -- values exchanged and combined between the lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>

namespace rr {
namespace {

template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned v)
{
    return unsigned(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, false));
}

// The value of the lane that step STEP of an exchange over G lanes pairs this
// one with: its neighbour, the other pair, the mirror lane of 8, of 16, and
// the lanes 16 and 32 away.
template <int STEP>
__device__ __forceinline__ unsigned other(unsigned v)
{
    if constexpr (STEP == 0)
        return dpp<0xb1>(v);
    else if constexpr (STEP == 1)
        return dpp<0x4e>(v);
    else if constexpr (STEP == 2)
        return dpp<0x141>(v);
    else if constexpr (STEP == 3)
        return dpp<0x140>(v);
    else
        return unsigned(__shfl_xor(int(v), 1 << STEP));
}
template <int STEP>
__device__ __forceinline__ float other(float v)
{
    return __uint_as_float(other<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double other(double v)
{
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    return __builtin_bit_cast(double, (unsigned long long)other<STEP>(unsigned(u >> 32)) << 32 | other<STEP>(unsigned(u)));
}

// f over G lanes side by side, the result in every lane.  f commutes, and both
// sides of each exchange combine the same two values, so all lanes get the
// same bits.
template <int G, int STEP = 0, typename T, typename F>
__device__ __forceinline__ T across(T v, F f)
{
    if constexpr (1 << STEP == G)
        return v;
    else
        return across<G, STEP + 1>(f(v, other<STEP>(v)), f);
}

template <int G>
__device__ __forceinline__ float lanes_sum(float v)
{
    return across<G>(v, [](float a, float b) { return a + b; });
}

template <int G>
__device__ __forceinline__ float lanes_max(float v)
{
    return across<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
}  // namespace rr
