// lin_common.h -- device helpers the projection's kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "bufio.h"
#include "epilogue.h"
#include "tokens.h"

namespace cvx {

typedef _Float16 half_t;
typedef __bf16 bf16_t;
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef half_t h8 __attribute__((ext_vector_type(8)));
typedef half_t h4 __attribute__((ext_vector_type(4)));
typedef bf16_t b8 __attribute__((ext_vector_type(8)));
typedef bf16_t b4 __attribute__((ext_vector_type(4)));

template <typename T>
struct V16 {  // vectors of a 16-bit type
    static constexpr bool BF = std::is_same<T, bf16_t>::value;
    typedef typename std::conditional<BF, b8, h8>::type v8;
    typedef typename std::conditional<BF, b4, h4>::type v4;
};

__device__ __forceinline__ u32x4 bload128(rsrc_t r, unsigned off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ u32x2 bload64(rsrc_t r, unsigned off)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
}

// 16x16 block += A (16 rows x 32 of k) * B (32 of k x 16 columns), 16-bit operands:
// lane l holds row/column l%16, eight values of k from 8*(l/16).
template <typename T>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (V16<T>::BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// 32x32 block, 16 of k a step: lane l holds row/column l%32, eight values of k from 8*(l/32).
template <typename T>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (V16<T>::BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// eight e4m3 values -> eight 16-bit values, exactly
template <typename T>
__device__ __forceinline__ u32x4 widen8(u32x2 q)
{
    typename V16<T>::v8 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
        o[4 * i] = (T)lo[0];
        o[4 * i + 1] = (T)lo[1];
        o[4 * i + 2] = (T)hi[0];
        o[4 * i + 3] = (T)hi[1];
    }
    return __builtin_bit_cast(u32x4, o);
}

typedef __attribute__((address_space(3))) void lds_void;

// Waits until at most N of this wave's vector-memory operations (fetches into LDS
// among them) are under way and what it read from LDS is here; no memory access
// moves across it.
template <int N>
__device__ __forceinline__ void wait_arrived()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// A barrier that waits for nothing: a wave waits before it for what the others may
// rely on (wait_arrived).  A fence here would wait for every fetch under way.
__device__ __forceinline__ void stage_barrier() { asm volatile("s_barrier" ::: "memory"); }

// An adapter of this token, or -1.
__device__ __forceinline__ int adapter_of(const LinArgs& a, int token)
{
    if (token >= a.tokens) return -1;
    const int d = a.lora_id[token];
    return d >= 0 && d < a.n_adapters ? d : -1;
}

// Ranks r to r+7 of v of a token with adapter d: its slices added, in order, times
// the adapter's factor.
__device__ __forceinline__ void lora_values(const LinArgs& a, int d, long token, int r, float (&v)[8])
{
    const float* p = a.part + token * a.rank + r;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    for (int s = 0; s < a.slices; s += 4) {
        f32x4 p0[4], p1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float* q = p + (long)(s + k) * a.tokens * a.rank;
            p0[k] = p1[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (s + k < a.slices) {
                p0[k] = *reinterpret_cast<const f32x4*>(q);
                p1[k] = *reinterpret_cast<const f32x4*>(q + 4);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] += p0[k][e];
                v[4 + e] += p1[k][e];
            }
    }
    const float alpha = a.lora_alpha ? a.lora_alpha[d] : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= alpha;
}

// The largest |v| of eight.
__device__ __forceinline__ float lora_top(const float (&v)[8])
{
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
    return top;
}

// fp16: the power of two a token's v is multiplied by, 2^-e, e the exponent of its largest |v|.
__device__ __forceinline__ float lora_factor(float top)
{
    int e = (int)((__builtin_bit_cast(unsigned, top) >> 23) & 255u) - 127;
    e = e < -24 ? -24 : e > 120 ? 120 : e;
    return __builtin_bit_cast(float, (unsigned)(127 - e) << 23);
}

// v as the sum of two 16-bit values.
template <typename T>
__device__ __forceinline__ void lora_parts(const float (&v)[8], u32x4& high, u32x4& low)
{
    typename V16<T>::v8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = (T)v[e];
        l[e] = __builtin_isfinite((float)h[e]) ? (T)(v[e] - (float)h[e]) : (T)0.0f;
    }
    high = __builtin_bit_cast(u32x4, h);
    low = __builtin_bit_cast(u32x4, l);
}

// The activation of a projection.  A NaN stays one (what marks a token as bad passes
// on), so ReLU is the maximum that keeps it, one instruction like the other one.
__device__ __forceinline__ float apply_act_nan(float v, int act)
{
    return act == CVX_ACT_RELU ? __builtin_elementwise_maximum(v, 0.0f) : apply_act_fast(v, act);
}

// z (scale, bias, adapters in it) -> y
__device__ __forceinline__ float finish(float z, float r, int act, int res_mode)
{
    if (res_mode == CVX_RES_BEFORE_ACT) z += r;
    z = apply_act_nan(z, act);
    if (res_mode == CVX_RES_AFTER_ACT) z += r;
    return z;
}

}  // namespace cvx
