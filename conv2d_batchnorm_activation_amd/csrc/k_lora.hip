// k_lora.hip -- the first product of the low-rank adapters,
//     v_t[r] = x_scale[t] * sum_i A_d[r][i] * x_t[i],   d = the token's adapter,
// for tokens of many adapters at once.
//
// A wave holds 16*NB tokens' values of 256 channels in registers as the matrix
// instruction's B operands, and goes through the distinct adapters of its tokens:
// each adapter's 16 x 256 block of A streams past once, and the lanes (one token
// each) whose token names that adapter keep the product.  So a block of tokens
// of one request costs one pass, tokens of many requests cost their adapters'
// bytes, and a value of another adapter never enters a token's sum.  Where there
// are few tokens, each likely of a request of its own, a block is one token:
// the passes over adapters are then workgroups side by side.  The four waves of a workgroup take the four quarters
// of 1024 channels and add their sums in LDS in a fixed order; a workgroup
// covers `slice_chunks` such steps, and the slices of c_in that make up the
// grid when there are few tokens are added, in order, by the kernel that reads
// them.
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

// A block is 16*NB tokens, or a single one (NB = 0); a workgroup takes RC times 16 ranks.
template <typename T, bool X8, int NB, int RC>
__global__ void __launch_bounds__(256) k_lora_down(LinArgs a)
{
    constexpr int B = NB ? NB : 1, TOK = NB ? 16 * NB : 1;
    constexpr unsigned XB = X8 ? 1 : 2;  // bytes of an x value
    __shared__ f32x4 red[4][RC * B][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Consecutive blocks of tokens, which share adapters, on one XCD (workgroups go
    // to the eight in turn), so that its cache holds the adapters of its tokens.
    const int xcd = blockIdx.x & 7, per = gridDim.x >> 3, rest = gridDim.x & 7;
    const int t0 = (xcd * per + (xcd < rest ? xcd : rest) + (int)(blockIdx.x >> 3)) * TOK;
    const int r0 = blockIdx.z * 16 * RC;
    const int q = lane >> 4, l16 = lane & 15;
    const int rows = a.tokens - t0 < TOK ? a.tokens - t0 : TOK;
    const rsrc_t rx = make_rsrc(static_cast<const char*>(a.x) + (long)t0 * a.xs * XB,
                                (unsigned)(((rows - 1) * a.xs + a.cin) * XB));
    int id[B];
    unsigned xrow[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int t = 16 * b + l16;
        id[b] = t < rows ? adapter_of(a, t0 + t) : -1;
        xrow[b] = t < rows ? (unsigned)(t * a.xs * XB) : kOOB;
    }

    f32x4 acc[RC][B];
#pragma unroll
    for (int r = 0; r < RC; ++r)
#pragma unroll
        for (int b = 0; b < B; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int ch = 0; ch < a.slice_chunks; ++ch) {
        const int k0 = (blockIdx.y * a.slice_chunks + ch) * kLoraChunk + wave * 256;
        if (k0 >= a.cin) break;  // later steps are past it too
        u32x4 xv[B][8];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = k0 + 32 * s + 8 * q;
                const unsigned off = k < a.cin && xrow[b] != kOOB ? xrow[b] + (unsigned)k * XB : kOOB;
                if constexpr (X8)
                    xv[b][s] = widen8<T>(bload64(rx, off));
                else
                    xv[b][s] = bload128(rx, off);
            }
        unsigned long long todo[B];
#pragma unroll
        for (int b = 0; b < B; ++b) todo[b] = __ballot(id[b] >= 0) & 0xffffull;
        for (;;) {  // each pass clears at least one bit
            int d = -1;
#pragma unroll
            for (int b = B - 1; b >= 0; --b)
                if (todo[b]) d = __builtin_amdgcn_readlane(id[b], __builtin_ctzll(todo[b]));
            if (d < 0) break;
            const rsrc_t ra = make_rsrc(static_cast<const T*>(a.lora_a) + (long)d * a.rank * a.cin,
                                        (unsigned)a.rank * (unsigned)a.cin * 2u);
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                const int ar = r0 + 16 * r + l16;  // row of A this lane holds
                u32x4 av[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int k = k0 + 32 * s + 8 * q;
                    const unsigned off =
                        k < a.cin && ar < a.rank ? ((unsigned)ar * (unsigned)a.cin + (unsigned)k) * 2u : kOOB;
                    av[s] = bload128(ra, off);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const bool mine = id[b] == d;
                    if (__ballot(mine) == 0) continue;
                    f32x4 c = acc[r][b];
#pragma unroll
                    for (int s = 0; s < 8; ++s) c = mma16<T>(av[s], xv[b][s], c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][b][i] = mine ? c[i] : acc[r][b][i];
                }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) todo[b] &= ~__ballot(id[b] == d);
        }
    }
#pragma unroll
    for (int r = 0; r < RC; ++r)
#pragma unroll
        for (int b = 0; b < B; ++b) red[wave][r * B + b][lane] = acc[r][b];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RC; ++r)
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if ((r * B + b) % 4 != wave) continue;
            const f32x4 s0 = red[0][r * B + b][lane], s1 = red[1][r * B + b][lane], s2 = red[2][r * B + b][lane],
                        s3 = red[3][r * B + b][lane];
            const int t = 16 * b + l16, rank = r0 + 16 * r + 4 * q;
            if (t < rows && rank < a.rank) {
                const float xs = X8 ? a.x_scale[t0 + t] : 1.0f;
                f32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = id[b] >= 0 ? xs * (((s0[i] + s1[i]) + s2[i]) + s3[i]) : 0.0f;
                // rank is a multiple of 8: whole, aligned vectors
                *reinterpret_cast<f32x4*>(a.part + ((long)blockIdx.y * a.tokens + t0 + t) * a.rank + rank) = o;
            }
        }
}

template <typename T, bool X8>
hipError_t launch_down_t(const LinArgs& a, const LinPlan& p, hipStream_t s)
{
    const int tok = p.down_nb ? 16 * p.down_nb : 1;
    const dim3 grid((unsigned)((a.tokens + tok - 1) / tok), (unsigned)a.slices,
                    (unsigned)((a.rank + 16 * p.down_rc - 1) / (16 * p.down_rc)));
    if (p.down_nb == 0)
        hipLaunchKernelGGL((k_lora_down<T, X8, 0, 1>), grid, dim3(256), 0, s, a);
    else if (p.down_nb == 1)
        hipLaunchKernelGGL((k_lora_down<T, X8, 1, 1>), grid, dim3(256), 0, s, a);
    else if (p.down_rc == 1)
        hipLaunchKernelGGL((k_lora_down<T, X8, 2, 1>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_lora_down<T, X8, 2, 4>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_down(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s)
{
    if (dtype == CVX_DT_F16) return x8 ? launch_down_t<half_t, true>(a, p, s) : launch_down_t<half_t, false>(a, p, s);
    return x8 ? launch_down_t<bf16_t, true>(a, p, s) : launch_down_t<bf16_t, false>(a, p, s);
}

}  // namespace cvx
