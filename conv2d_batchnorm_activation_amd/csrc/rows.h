// rows.h -- device helpers of the operators on rows (the norm, the gated activation):
// vectors of a row, reductions over its threads, 8-bit codes.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "tokens.h"

namespace cvx {

typedef _Float16 half_t;
typedef __bf16 bf16_t;

// the largest value of an 8-bit type
template <int OUT>
constexpr double kTop = OUT == kXE4m3 ? 448.0 : 127.0;

template <typename T, int N>
struct Vec {
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};
typedef unsigned u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned u32x1u __attribute__((aligned(1)));

__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// e4m3 takes fp32 values; a 64-bit value goes there rounded to odd (its last bit
// set if anything is cut), which the rounding to four bits sees as it is.
__device__ __forceinline__ float to_odd(double v)
{
    unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = (unsigned)b;
    const unsigned cut = (lo & 0xe0000000u) | ((lo & 0x1fffffffu) ? 0x20000000u : 0u);
    b = (b & 0xffffffff00000000ull) | cut;
    return (float)__builtin_bit_cast(double, b);
}

// A value on its way to a code, the nearest to it: for e4m3 the bits of an fp32 value,
// else an integer's, the low bits of a sum that leaves none below one (of a NaN they
// say nothing).
template <int OUT>
__device__ __forceinline__ unsigned code_part(double v)
{
#pragma clang fp contract(off)  // v is a rounded product: fused into the sum, borders would be missed by a hair
    if constexpr (OUT == kXE4m3) return __builtin_bit_cast(unsigned, to_odd(v));
    const double at_ones = v + 0x1.8p52;
    return (unsigned)__builtin_bit_cast(unsigned long long, at_ones);
}
template <int OUT>
__device__ __forceinline__ unsigned pack_codes(unsigned a, unsigned b, unsigned c, unsigned d)
{
    auto f = [](unsigned v) { return __builtin_bit_cast(float, v); };
    if constexpr (OUT == kXE4m3) return pack_e4m3(f(a), f(b), f(c), f(d));
    return (a & 255u) | (b & 255u) << 8 | (c & 255u) << 16 | d << 24;
}
// Channels i0 to i0+VEC-1 of a row of c codes, those there are.
template <int VEC>
__device__ __forceinline__ void store_codes(unsigned char* y, int i0, int c, const unsigned (&w)[VEC / 4])
{
    if (i0 + VEC <= c) {
        if constexpr (VEC == 8) {
            u32x2u w2;
            w2[0] = w[0];
            w2[1] = w[1];
            *reinterpret_cast<u32x2u*>(y + i0) = w2;
        } else {
            *reinterpret_cast<u32x1u*>(y + i0) = w[0];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (i0 + e < c) y[i0 + e] = (unsigned char)(w[e / 4] >> (8 * (e % 4)));
    }
}

// The value of another lane of the same 16 (a DPP control), or of lane L.
template <int CTRL>
__device__ __forceinline__ double lane_move(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_mov_dpp((int)b, CTRL, 0xf, 0xf, true);
    const unsigned hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
template <int L>
__device__ __forceinline__ double lane_value(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_readlane((int)b, L), hi = __builtin_amdgcn_readlane((int)(b >> 32), L);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// op over the 64 lanes of a wave, whole: within 16 lanes by DPP (neighbour, pair,
// mirrored half, mirrored row: lanes that hold the same value are interchangeable),
// then the four rows.  A quarter of the latency of six shuffles by way of LDS.
template <typename OP>
__device__ __forceinline__ double wave_all(double v, OP op)
{
    v = op(v, lane_move<0xb1>(v));
    v = op(v, lane_move<0x4e>(v));
    v = op(v, lane_move<0x141>(v));
    v = op(v, lane_move<0x140>(v));
    return op(op(lane_value<0>(v), lane_value<16>(v)), op(lane_value<32>(v), lane_value<48>(v)));
}

// The largest of the values of a row's TPR threads (8, 16 or whole waves), none of them a
// NaN.  S: which of a kernel's exchanges by way of LDS this is.
template <int TPR, int S, typename V>
__device__ __forceinline__ V row_top(V v)
{
    constexpr bool F = sizeof(V) == 4;
    auto move = [](V x, auto ctrl) {
        if constexpr (F)
            return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
        else
            return lane_move<decltype(ctrl)::value>(x);
    };
    auto larger = [](V x, V y) {
        if constexpr (F)
            return fmaxf(x, y);
        else
            return fmax(x, y);
    };
    v = larger(v, move(v, std::integral_constant<int, 0xb1>()));
    v = larger(v, move(v, std::integral_constant<int, 0x4e>()));
    v = larger(v, move(v, std::integral_constant<int, 0x141>()));
    if constexpr (TPR > 8) v = larger(v, move(v, std::integral_constant<int, 0x140>()));
    if constexpr (TPR > 16) {
        auto of = [&](auto lane) {
            if constexpr (F)
                return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), decltype(lane)::value));
            else
                return lane_value<decltype(lane)::value>(v);
        };
        v = larger(larger(of(std::integral_constant<int, 0>()), of(std::integral_constant<int, 16>())),
                   larger(of(std::integral_constant<int, 32>()), of(std::integral_constant<int, 48>())));
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __shared__ V tops[W];
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) v = larger(v, tops[i]);
    }
    return v;
}

// Row sums over TPR threads of `s` and maxima of `m`; every thread gets both.
template <int TPR, bool MAX>
__device__ __forceinline__ void row_reduce(double& s, double& m)
{
    s = wave_all(s, [](double a, double b) { return a + b; });
    if (MAX) m = wave_all(m, [](double a, double b) { return fmax(a, b); });
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __shared__ double ls[W];
        __shared__ double lm[W];
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            ls[wave] = s;
            if (MAX) lm[wave] = m;
        }
        __syncthreads();
        s = 0.0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s += ls[i];
            if (MAX) m = fmax(m, lm[i]);
        }
    }
}

}  // namespace cvx
