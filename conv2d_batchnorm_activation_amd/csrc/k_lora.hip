// k_lora.hip -- the first product of the low-rank adapters,
//     v_t[r] = x_scale[t] * sum_i A_d[r][i] * x_t[i],   d = the token's adapter,
// for tokens of many adapters at once.
//
// A wave holds 16 tokens' values of 256 channels in registers as the matrix
// instruction's B operand, and goes through the distinct adapters of its tokens:
// each adapter's 16 x 256 block of A streams past once, and the lanes (one token
// each) whose token names that adapter keep the product.  So a block of tokens of
// one request costs one pass, tokens of many requests cost their adapters' bytes,
// and a value of another adapter never enters a token's sum.  Where there are few
// tokens, each likely of a request of its own, a block is one token: the passes
// over adapters are then workgroups side by side.  The four waves of a workgroup
// take the four quarters of 1024 channels and add their sums in LDS in a fixed
// order; a workgroup covers a slice of whole such steps, and the slices of c_in
// that make up the grid when there are few tokens are added, in order, by the
// kernel that reads them.
//
// Latency bounds the small ones, the address unit the larger.  Measured, 4096
// channels bf16: 48 tokens of as many adapters, rank 32, 5.5 us; 512 tokens, rank
// 16, 5.7; 4096 tokens in 64s (k_lora_down_many), rank 16, 10.5 (14.5 in registers,
// with consecutive blocks on all XCDs); 8192 tokens of e4m3, rank 64, 29.  Joining
// the slices: 2.5 to 5 us.
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

// Workgroups go to the eight XCDs in turn: consecutive blocks of tokens, which share
// adapters, on one, so that its cache holds the adapters of its tokens.
__device__ __forceinline__ int xcd_run(unsigned block, unsigned blocks)
{
    const unsigned xcd = block & 7, per = blocks >> 3, rest = blocks & 7;
    return (int)(xcd * per + (xcd < rest ? xcd : rest) + (block >> 3));
}

// A block is 16 tokens, or a single one (NB = 0).
template <typename T, int X, int NB>
__global__ void __launch_bounds__(256) k_lora_down(LinArgs a)
{
    constexpr int TOK = NB ? 16 : 1;
    constexpr bool X8 = X != kX16;       // e4m3 or integers: exact in 16 bits
    constexpr unsigned XB = X8 ? 1 : 2;  // bytes of an x value
    __shared__ f32x4 red[4][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = xcd_run(blockIdx.x, gridDim.x) * TOK;
    const int r0 = blockIdx.z * 16;
    const int q = lane >> 4, l16 = lane & 15;
    const int rows = a.tokens - t0 < TOK ? a.tokens - t0 : TOK;
    const rsrc_t rx = make_rsrc(static_cast<const char*>(a.x) + (long)t0 * a.xs * XB,
                                (unsigned)(((rows - 1) * a.xs + a.cin) * XB));
    const int id = l16 < rows ? adapter_of(a, t0 + l16) : -1;
    const unsigned xrow = l16 < rows ? (unsigned)(l16 * a.xs * XB) : kOOB;
    const int ar = r0 + l16;  // row of A this lane holds

    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int ch = 0; ch < a.slice_len; ch += kLoraChunk) {
        const int k0 = blockIdx.y * a.slice_len + ch + wave * 256;
        if (k0 >= a.cin) break;  // later steps are past it too
        u32x4 xv[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            const unsigned off = k < a.cin && xrow != kOOB ? xrow + (unsigned)k * XB : kOOB;
            if constexpr (X8)
                xv[s] = widen8<T, X>(bload64(rx, off));
            else
                xv[s] = bload128(rx, off);
        }
        unsigned long long todo = __ballot(id >= 0) & 0xffffull;
        while (todo) {  // each pass clears at least the first bit
            const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            const bool mine = id == d;
            todo &= ~__ballot(mine);
            const rsrc_t ra = make_rsrc(static_cast<const T*>(a.lora_a) + (long)d * a.rank * a.cin,
                                        (unsigned)a.rank * (unsigned)a.cin * 2u);
            f32x4 c = acc;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = k0 + 32 * s + 8 * q;
                const unsigned off =
                    k < a.cin && ar < a.rank ? ((unsigned)ar * (unsigned)a.cin + (unsigned)k) * 2u : kOOB;
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
        const int rank = r0 + 4 * q;
        if (id >= 0 && rank < a.rank) {  // (of a token without an adapter nothing is read)
            const float xs = X8 ? a.x_scale[t0 + l16] : 1.0f;
            f32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = xs * (((s0[i] + s1[i]) + s2[i]) + s3[i]);
            // rank is a multiple of 8: whole, aligned vectors
            *reinterpret_cast<f32x4*>(a.part + ((long)blockIdx.y * a.tokens + t0 + l16) * a.rank + rank) = o;
        }
    }
}

// Many tokens: 64 a workgroup, 16 a wave, RB times 16 ranks, both operands by way
// of LDS, 128 bytes of every row of x a stage (and as many channels of A, twice
// the bytes where x is in 8 bits), two stages a workgroup under way, and three to six
// workgroups a compute unit: short ones, as a block of several requests takes as
// many passes.  What the registers'
// form above pays is the address unit: 16 rows a load are 64 cycles of it for
// 1 KB, where a fetch of whole lines is 16.
template <typename T, int X, int RB>
__global__ void __launch_bounds__(256) k_lora_down_many(LinArgs a)
{
    constexpr bool X8 = X != kX16;
    constexpr unsigned XB = X8 ? 1 : 2;
    constexpr int KS = X8 ? 128 : 64;                  // channels a stage
    constexpr int AL = X8 ? 2 : 1;                     // 128-byte lines of a row of A a stage
    constexpr int FA = (2 * RB * AL + 3) / 4, F = 2 + FA;  // fetches of a wave: A, all
    constexpr int SB = 8192 + FA * 4096;
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[SB], buf1[SB];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = xcd_run(blockIdx.x, gridDim.x) * 64;
    const int r0 = blockIdx.z * 16 * RB;
    const int q = lane >> 4, l16 = lane & 15;
    const int rows = a.tokens - t0 < 64 ? a.tokens - t0 : 64;
    const int k0 = blockIdx.y * a.slice_len;  // this slice's channels
    const int kn = a.cin - k0 < a.slice_len ? a.cin - k0 : a.slice_len;
    const int nst = (kn + KS - 1) / KS;
    const int all = adapter_of(a, t0 + lane);  // the block's adapters, a lane each
    const int token = t0 + 16 * wave + l16;    // this lane's, as a column
    const int id = adapter_of(a, token);

    const unsigned pitch = (unsigned)a.xs * XB, ab = (unsigned)a.cin * 2u;
    const rsrc_t rx = make_rsrc(static_cast<const char*>(a.x) + (long)t0 * pitch + (long)k0 * XB,
                                (unsigned)(rows - 1) * pitch + (unsigned)kn * XB);
    // Pieces lie permuted as in the tile kernel, p at p ^ (r/2 % 8) of row r.  A
    // wave's fetches of x are of rows 8*wave and 32 + 8*wave; of A, line j of rows
    // 8*i is fetch i*AL + j, taken in turn by the waves.
    const unsigned xpiece = (unsigned)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
    const unsigned xo = (unsigned)(8 * wave + (lane >> 3)) * pitch + xpiece;
    auto issue = [&](int st, unsigned char* buf, rsrc_t ra) {
        const unsigned kb = (unsigned)st * 128;
        const bool xlive = st < nst && kb + xpiece < (unsigned)kn * XB;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(buf + 1024 * (wave + 4 * i)), 16,
                                                     xlive ? xo + 32 * i * pitch + kb : kOOB, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int f = wave + 4 * i, row = 8 * (f / AL) + (lane >> 3);
            const unsigned piece = (unsigned)((lane & 7) ^ ((row >> 1) & 7)) * 16;
            const unsigned k = (unsigned)(st * AL + f % AL) * 128 + piece;
            const bool live = st < nst && f < 2 * RB * AL && r0 + row < a.rank && k < (unsigned)kn * 2u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_void*)(buf + 8192 + 1024 * f), 16,
                live ? (unsigned)(r0 + row) * ab + (unsigned)k0 * 2u + k : kOOB, 0, 0, 0);
        }
    };
    unsigned long long todo = __ballot(all >= 0);
    while (todo) {  // each pass clears at least the first bit
        const int d = __builtin_amdgcn_readlane(all, __builtin_ctzll(todo));
        todo &= ~__ballot(all == d);
        const rsrc_t ra = make_rsrc(static_cast<const T*>(a.lora_a) + (long)d * a.rank * a.cin, (unsigned)a.rank * ab);
        f32x4 c[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) c[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const bool any = __ballot(id == d) != 0;
        auto stage = [&](int st, unsigned char* buf) {
            wait_arrived<F>();
            stage_barrier();
            const unsigned char* px = buf + (16 * wave + l16) * 128;
            const unsigned char* pa = buf + 8192;
            const unsigned key = (unsigned)(l16 >> 1);
            u32x4 xv[2], av[X8 ? 4 : 2][RB];
#pragma unroll
            for (int s = 0; s < 2; ++s) xv[s] = *reinterpret_cast<const u32x4*>(px + ((4 * s + q) ^ key) * 16);
#pragma unroll
            for (int s = 0; s < 2 * AL; ++s)
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    // 8 bits: channels 64j + 16q + 8h of step s = 2j + h are line j, piece 2q + h
                    const int piece = X8 ? 2 * q + (s & 1) : 4 * s + q, line = X8 ? s >> 1 : 0;
                    const int row = 16 * r + l16;
                    av[s][r] = *reinterpret_cast<const u32x4*>(pa + ((row >> 3) * AL + line) * 1024 + (row & 7) * 128 +
                                                               (piece ^ (int)key) * 16);
                }
            wait_arrived<63>();
            stage_barrier();  // every wave has read the stage
            issue(st + 2, buf, ra);
            if (any) {
#pragma unroll
                for (int s = 0; s < 2 * AL; ++s) {
                    const u32x4 x = X8 ? widen8<T, X>(u32x2{xv[s / AL][2 * (s % AL)], xv[s / AL][2 * (s % AL) + 1]}) : xv[s / AL];
#pragma unroll
                    for (int r = 0; r < RB; ++r) c[r] = mma16<T>(av[s][r], x, c[r]);
                }
            }
        };
        issue(0, buf0, ra);
        issue(1, buf1, ra);
        for (int st = 0; st < nst; st += 2) {
            stage(st, buf0);
            stage(st + 1, buf1);
        }
        wait_arrived<0>();  // no fetch of this adapter is under way when the next one's begin
        stage_barrier();
        if (id == d) {
            const float xs = X8 ? a.x_scale[token] : 1.0f;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int rank = r0 + 16 * r + 4 * q;
                if (rank >= a.rank) continue;
                f32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = xs * c[r][i];
                *reinterpret_cast<f32x4*>(a.part + ((long)blockIdx.y * a.tokens + token) * a.rank + rank) = o;
            }
        }
    }
}

// v joined and taken apart into two 16-bit values, once for all the tiles of output
// channels that read them; a token's ranks are eight a lane.  Tokens without an adapter get zeros, which nothing reads.
template <typename T>
__global__ void __launch_bounds__(256) k_lora_join(LinArgs a)
{
    int lanes = 2;  // that share a token: a power of two, of whole sixteens of ranks
    while (8 * lanes < a.rank) lanes *= 2;
    const long at = (long)blockIdx.x * 256 + threadIdx.x;
    const long token = at / lanes;
    const int r8 = (int)(at & (lanes - 1)), r = 8 * r8;
    const int id = token < a.tokens ? adapter_of(a, (int)token) : -1;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (id >= 0 && r < a.rank) lora_values(a, id, token, r, v);
    if constexpr (!V16<T>::BF) {
        float top = lora_top(v);
        for (int o = 1; o < lanes; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
        const float down = lora_factor(top);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= down;
        if (r == 0 && token < a.tokens) a.down[token] = down;
    }
    if (token < a.tokens && r < (a.rank + 15) / 16 * 16) {
        u32x4* out = static_cast<u32x4*>(a.joined) + 2l * r8 * a.tokens + token;
        lora_parts<T>(v, out[0], out[a.tokens]);
    }
}

template <typename T, int X>
hipError_t launch_down_t(const LinArgs& a, const LinPlan& p, hipStream_t s)
{
    const int tok = p.down_nb ? 16 * p.down_nb : 1;
    const dim3 grid((unsigned)((a.tokens + tok - 1) / tok), (unsigned)a.slices,
                    (unsigned)((a.rank + 16 * p.down_rc - 1) / (16 * p.down_rc)));
    if (p.down_nb == 0)
        hipLaunchKernelGGL((k_lora_down<T, X, 0>), grid, dim3(256), 0, s, a);
    else if (p.down_nb == 1)
        hipLaunchKernelGGL((k_lora_down<T, X, 1>), grid, dim3(256), 0, s, a);
    else if (p.down_rc == 1)
        hipLaunchKernelGGL((k_lora_down_many<T, X, 1>), grid, dim3(256), 0, s, a);
    else if (p.down_rc == 2)
        hipLaunchKernelGGL((k_lora_down_many<T, X, 2>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_lora_down_many<T, X, 4>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_join(const LinArgs& a, int dtype, hipStream_t s)
{
    int lanes = 2;
    while (8 * lanes < a.rank) lanes *= 2;
    const dim3 grid((unsigned)(((long)a.tokens * lanes + 255) / 256));
    if (dtype == CVX_DT_F16)
        hipLaunchKernelGGL((k_lora_join<half_t>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_lora_join<bf16_t>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_lora_down(const LinArgs& a, const LinPlan& p, int dtype, int held, hipStream_t s)
{
    return by_types(dtype, held, [&](auto t, auto x) { return launch_down_t<typename decltype(t)::type, x.value>(a, p, s); });
}

}  // namespace cvx
