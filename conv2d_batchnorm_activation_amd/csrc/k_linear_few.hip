// k_linear_few.hip -- projection of few tokens (up to 64), the form for
// generated tokens: bound by the stream of the weights.
//
// A workgroup takes 16 output channels and all tokens; its eight waves take
// 256-byte pieces of the weight rows in turn, straight from memory into the
// matrix instruction's A operand (16 rows x 64 bytes a load), with the tokens'
// values of the same channels as the B operand: a lane is a token, so the
// columns of tokens that are not there cost no traffic.  The waves' sums meet
// in LDS and are added in a fixed order.  The low-rank term is a few thousand
// multiply-adds a workgroup and is taken in fp32 on the vector units: v from
// LDS, the adapters' rows of these 16 channels from memory.
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

constexpr int kFewWaves = 8;

// 16x16 block, 64 bytes of k a row.  e4m3 values are widened to 16 bits, exactly:
// the 8-bit matrix instructions drop what lies 2^-13 below the largest of eight
// products, and here the stream of the weights leaves time for better.
template <typename T, bool X8>
__device__ __forceinline__ f32x4 mma_piece(u32x4 w, u32x4 x, f32x4 c)
{
    if constexpr (X8) {
        c = mma16<T>(widen8<T>(u32x2{w[0], w[1]}), widen8<T>(u32x2{x[0], x[1]}), c);
        return mma16<T>(widen8<T>(u32x2{w[2], w[3]}), widen8<T>(u32x2{x[2], x[3]}), c);
    } else {
        return mma16<T>(w, x, c);
    }
}

template <typename T, bool X8, int NT>
__global__ void __launch_bounds__(64 * kFewWaves) k_linear_few(LinArgs a)
{
    typedef typename V16<T>::v8 v8;
    constexpr unsigned XB = X8 ? 1 : 2;
    __shared__ f32x4 red[kFewWaves][NT][64];
    extern __shared__ float vlds[];  // [tokens][rank]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c0 = blockIdx.x * 16;
    const int q = lane >> 4;
    const unsigned cb = (unsigned)a.cin * XB;  // bytes of a weight row
    const unsigned pitch = (unsigned)a.xs * XB;
    const int rows = a.cout - c0 < 16 ? a.cout - c0 : 16;
    const rsrc_t rw = make_rsrc(static_cast<const char*>(a.w) + (long)c0 * cb, (unsigned)rows * cb);
    const rsrc_t rx = make_rsrc(a.x, (unsigned)(a.tokens - 1) * pitch + cb);
    const unsigned wrow = (unsigned)(lane & 15) * cb;
    unsigned xrow[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xrow[n] = (unsigned)(16 * n + (lane & 15)) * pitch;

    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int chunks = (int)((cb + 255) / 256);
    for (int ch = wave; ch < chunks; ch += kFewWaves) {
        u32x4 wv[4], xv[NT][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const unsigned k = (unsigned)ch * 256 + 64 * s + 16 * q;
            const bool live = k < cb;
            wv[s] = bload128(rw, live ? wrow + k : kOOB);
#pragma unroll
            for (int n = 0; n < NT; ++n) xv[n][s] = bload128(rx, live ? xrow[n] + k : kOOB);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] = mma_piece<T, X8>(wv[s], xv[n][s], acc[n]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][n][lane] = acc[n];
    if (a.rank) {
        // the tokens' low-rank values: slices added in order, times the adapter's factor
        for (int i = tid; i < a.tokens * a.rank; i += 64 * kFewWaves) {
            const int t = i / a.rank;
            const int d = adapter_of(a, t);
            float v = 0.0f;
            for (int s = 0; s < a.slices; ++s) v += a.part[(long)s * a.tokens * a.rank + i];
            vlds[i] = d >= 0 && a.lora_alpha ? v * a.lora_alpha[d] : v;
        }
    }
    __syncthreads();
    for (int i = tid; i < NT * 256; i += 64 * kFewWaves) {
        const int ch = i & 15, t = i >> 4;
        const int c = c0 + ch;
        if (t >= a.tokens || c >= a.cout) continue;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) z += red[w][t >> 4][(ch >> 2) * 16 + (t & 15)][ch & 3];
        if (a.scale) z *= a.scale[c];
        if constexpr (X8) z *= a.x_scale[t];
        if (a.bias) z += a.bias[c];
        if (a.rank) {
            const int d = adapter_of(a, t);
            if (d >= 0) {
                const T* b = static_cast<const T*>(a.lora_b) + ((long)d * a.cout + c) * a.rank;
                const float* v = vlds + t * a.rank;
                float u = 0.0f;
                for (int r = 0; r < a.rank; r += 8) {
                    const v8 bv = *reinterpret_cast<const v8*>(b + r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u = fmaf((float)bv[e], v[r + e], u);
                }
                z += u;
            }
        }
        const float r = a.res ? (float)static_cast<const T*>(a.res)[(long)t * a.rs + c] : 0.0f;
        static_cast<T*>(a.y)[(long)t * a.ys + c] = (T)finish(z, r, a.act, a.res_mode);
    }
}

template <typename T, bool X8>
hipError_t launch_few_t(const LinArgs& a, const LinPlan& p, hipStream_t s)
{
    const dim3 grid((unsigned)((a.cout + 15) / 16)), block(64 * kFewWaves);
    const size_t lds = (size_t)a.tokens * a.rank * sizeof(float);
    if (p.nt == 1)
        hipLaunchKernelGGL((k_linear_few<T, X8, 1>), grid, block, lds, s, a);
    else if (p.nt == 2)
        hipLaunchKernelGGL((k_linear_few<T, X8, 2>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((k_linear_few<T, X8, 4>), grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_few(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s)
{
    if (a.tokens > 16 * p.nt) return hipErrorInvalidValue;
    if (dtype == CVX_DT_F16) return x8 ? launch_few_t<half_t, true>(a, p, s) : launch_few_t<half_t, false>(a, p, s);
    return x8 ? launch_few_t<bf16_t, true>(a, p, s) : launch_few_t<bf16_t, false>(a, p, s);
}

}  // namespace cvx
