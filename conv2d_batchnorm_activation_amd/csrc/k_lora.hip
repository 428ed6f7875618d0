// k_lora.hip -- the first product of the low-rank adapters,
//     v_t[r] = x_scale[t] * sum_i A_d[r][i] * x_t[i],   d = the token's adapter,
// for tokens of many adapters at once.
//
// A wave holds 16 tokens' values of 256 channels in registers as the matrix
// instruction's B operand, and goes through the distinct adapters of its 16
// tokens: each adapter's 16 x 256 block of A streams past once, and the lanes
// (one token each) whose token names that adapter keep the product.  So a block
// of tokens of one request costs one pass, 16 tokens of 16 requests cost the 16
// adapters' bytes they cannot do without, and a value of another adapter never
// enters a token's sum.  The four waves of a workgroup take the four quarters
// of 1024 channels and add their sums in LDS in a fixed order; a workgroup
// covers `slice_chunks` such steps, and the slices of c_in that make up the
// grid when there are few tokens are added, in order, by the kernel that reads
// them.
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

template <typename T, bool X8>
__global__ void __launch_bounds__(256) k_lora_down(LinArgs a)
{
    __shared__ f32x4 red[4][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = blockIdx.x * 16;
    const int token = t0 + (lane & 15);
    const int r0 = blockIdx.z * 16;
    const int q = lane >> 4;
    const int id = adapter_of(a, token);
    constexpr unsigned XB = X8 ? 1 : 2;  // bytes of an x value
    const int rows = a.tokens - t0 < 16 ? a.tokens - t0 : 16;
    const rsrc_t rx = make_rsrc(static_cast<const char*>(a.x) + (long)t0 * a.xs * XB,
                                (unsigned)(((rows - 1) * a.xs + a.cin) * XB));
    const unsigned xrow = (lane & 15) < rows ? (unsigned)((lane & 15) * a.xs * XB) : kOOB;
    const int ar = r0 + (lane & 15);  // row of A this lane holds

    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int ch = 0; ch < a.slice_chunks; ++ch) {
        const int k0 = (blockIdx.y * a.slice_chunks + ch) * kLoraChunk + wave * 256;
        if (k0 >= a.cin) break;  // later steps are past it too
        u32x4 xv[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            const unsigned off = k < a.cin && xrow != kOOB ? xrow + (unsigned)k * XB : kOOB;
            if constexpr (X8)
                xv[s] = widen8<T>(bload64(rx, off));
            else
                xv[s] = bload128(rx, off);
        }
        unsigned long long todo = __ballot(id >= 0) & 0xffffull;
        while (todo) {  // each pass clears at least its first bit
            const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            const bool mine = id == d;
            todo &= ~__ballot(mine);
            const rsrc_t ra = make_rsrc(static_cast<const T*>(a.lora_a) + (long)d * a.rank * a.cin,
                                        (unsigned)a.rank * (unsigned)a.cin * 2u);
            f32x4 c = acc;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = k0 + 32 * s + 8 * q;
                const unsigned off = k < a.cin && ar < a.rank ? ((unsigned)ar * (unsigned)a.cin + (unsigned)k) * 2u : kOOB;
                c = mma16<T>(bload128(ra, off), xv[s], c);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = mine ? c[i] : acc[i];
        }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        const f32x4 s0 = red[0][lane], s1 = red[1][lane], s2 = red[2][lane], s3 = red[3][lane];
        const int r = r0 + 4 * q;
        if (token < a.tokens && r < a.rank) {
            const float xs = X8 ? a.x_scale[token] : 1.0f;
            f32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = id >= 0 ? xs * (((s0[i] + s1[i]) + s2[i]) + s3[i]) : 0.0f;
            float* dst = a.part + ((long)blockIdx.y * a.tokens + token) * a.rank + r;
            *reinterpret_cast<f32x4*>(dst) = o;  // rank is a multiple of 8: whole, aligned vectors
        }
    }
}

}  // namespace

hipError_t launch_lora_down(const LinArgs& a, int dtype, int x8, hipStream_t s)
{
    const dim3 grid((unsigned)((a.tokens + 15) / 16), (unsigned)a.slices, (unsigned)((a.rank + 15) / 16));
    if (dtype == CVX_DT_F16) {
        if (x8)
            hipLaunchKernelGGL((k_lora_down<half_t, true>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_lora_down<half_t, false>), grid, dim3(256), 0, s, a);
    } else {
        if (x8)
            hipLaunchKernelGGL((k_lora_down<bf16_t, true>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_lora_down<bf16_t, false>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace cvx
