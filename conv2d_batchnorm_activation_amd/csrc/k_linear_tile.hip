// k_linear_tile.hip -- projection of many tokens: a tile of 64*MB output
// channels x 64*NB tokens a workgroup, on the matrix cores.
//
// The weights are the A operand (rows = output channels) and the tokens the B
// operand (columns = tokens), so a lane's accumulators are channels of one
// token.  Four waves, two by two, each 32*MB x 32*NB.  A stage is 128 bytes of
// every row of both operands, loaded straight into LDS; the 16-byte pieces of a
// row are permuted by the row's index as they are fetched, so that the lanes of
// an operand read (32 rows, the same piece) fall in different banks while every
// fetch still takes whole 128-byte lines.  Two stage buffers: stage s+1 arrives
// while s is multiplied, with one barrier a stage, which comes before the
// stage's last step so that the next stage's first operands are read under it.
//
// 8-bit operands (e4m3) are the same bytes: a stage is 128 channels instead of
// 64, and the 32x32x64 instruction takes two pieces a lane where the 16-bit
// one takes one.  Any assignment of k to lanes serves, as long as both operands
// use the same.  The 8-bit instructions align the products of eight consecutive
// channels to the largest of them and drop what lies 2^-13 below it (the sums of
// these groups are fp32): about 2^-13 of the result's size on data like normal
// values, a sixteenth of bf16's own rounding, taken for twice the rate.
//
// Adapters: once the sums stand in registers they get scale and bias, and the
// second product of the adapters is accumulated onto them by the same matrix
// instructions: for every 32 tokens, each distinct adapter's rows of B, with v
// as two 16-bit values (v = high + low, so v keeps 16 bits in bf16 and 21 in
// fp16); the lanes whose token names the adapter keep the result.  fp16, whose
// range v may leave, takes v and the sums divided by a power of two per token.
#include <stdio.h>

#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

typedef __attribute__((address_space(3))) void lds_void;

template <bool X8>
struct Op {
    typedef typename std::conditional<X8, i32x8, u32x4>::type type;
};

template <typename T, bool X8, int MB, int NB>
__global__ void __launch_bounds__(256, MB * NB >= 16 ? 1 : 2) k_linear_tile(LinArgs a)
{
    typedef typename V16<T>::v8 v8;
    typedef typename V16<T>::v4 v4;
    typedef typename Op<X8>::type op_t;
    constexpr unsigned XB = X8 ? 1 : 2;
    constexpr int BM = 64 * MB, BN = 64 * NB;
    constexpr int STEPS = X8 ? 2 : 4;
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[(BM + BN) * 128];
    __shared__ __attribute__((aligned(1024))) unsigned char buf1[(BM + BN) * 128];
    __shared__ float down_lds[V16<T>::BF ? 1 : BN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int hi = lane >> 5, l32 = lane & 31;

    // Workgroups go to the XCDs in turn: give each XCD a run of tiles, and runs
    // go through eight tiles of channels before the next tile of tokens.
    int m0, n0;
    {
        const int n = a.tiles_m * a.tiles_n;
        const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
        const int per = n >> 3, rest = n & 7;
        const int tile = xcd * per + (xcd < rest ? xcd : rest) + idx;
        const int wide = 8 * a.tiles_n;
        const int grp = tile / wide, in = tile - grp * wide;
        const int gm = a.tiles_m - 8 * grp < 8 ? a.tiles_m - 8 * grp : 8;
        const int tn = in / gm;
        m0 = (8 * grp + in - tn * gm) * BM;
        n0 = tn * BN;
    }
    const unsigned cb = (unsigned)a.cin * XB, pitch = (unsigned)a.xs * XB;
    const int mrows = a.cout - m0 < BM ? a.cout - m0 : BM;
    const int nrows = a.tokens - n0 < BN ? a.tokens - n0 : BN;
    const char* wt = static_cast<const char*>(a.w) + (long)(m0 + 8 * wave) * cb;
    const char* xt = static_cast<const char*>(a.x) + (long)(n0 + 8 * wave) * pitch;
    const unsigned piece = (unsigned)((lane & 7) ^ (lane >> 3)) * 16;
    const unsigned wo = (unsigned)(lane >> 3) * cb + piece;
    const unsigned xo = (unsigned)(lane >> 3) * pitch + piece;
    const int nst = (int)((cb + 127) / 128);

    // Eight rows a fetch.  Each has a descriptor of its own, which ends with the
    // operand's rows, so what a lane holds is one offset an operand; pieces past
    // the end of a row are sent out of range.
    auto issue = [&](int st, unsigned char* buf) {
        const unsigned kb = (unsigned)st * 128 < cb ? (unsigned)st * 128 : 0u;  // past the end: nothing is live
        const bool live = (unsigned)st * 128 + piece < cb;
        const unsigned wl = live ? wo : kOOB, xl = live ? xo : kOOB;
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i) {
            const int left = mrows - 8 * wave - 32 * i;
            const unsigned n = left <= 0 ? 0u : (unsigned)(left < 8 ? left : 8) * cb - kb;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(wt + (long)(32 * i) * cb + kb, n),
                                                     (lds_void*)(buf + 1024 * (wave + 4 * i)), 16, wl, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
            const int left = nrows - 8 * wave - 32 * i;
            const unsigned n = left <= 0 ? 0u : (unsigned)((left < 8 ? left : 8) - 1) * pitch + cb - kb;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(xt + (long)(32 * i) * pitch + kb, n),
                                                     (lds_void*)(buf + BM * 128 + 1024 * (wave + 4 * i)), 16, xl, 0, 0, 0);
        }
    };
    unsigned slot[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) slot[s] = (unsigned)(l32 * 128 + (((2 * s + hi) ^ (l32 & 7)) * 16));
    auto read = [&](const unsigned char* buf, int st, op_t (&A)[MB], op_t (&B)[NB]) {
        const unsigned char* pa = buf + wm * MB * 4096;
        const unsigned char* pb = buf + BM * 128 + wn * NB * 4096;
        auto one = [&](const unsigned char* p) {
            if constexpr (X8) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(p + slot[2 * st]);
                const u32x4 y = *reinterpret_cast<const u32x4*>(p + slot[2 * st + 1]);
                i32x8 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = (int)x[e];
                    o[4 + e] = (int)y[e];
                }
                return o;
            } else {
                return *reinterpret_cast<const u32x4*>(p + slot[st]);
            }
        };
#pragma unroll
        for (int m = 0; m < MB; ++m) A[m] = one(pa + 4096 * m);
#pragma unroll
        for (int n = 0; n < NB; ++n) B[n] = one(pb + 4096 * n);
    };

    f32x16 acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;
    op_t A0[MB], B0[NB], A1[MB], B1[NB];
    auto mul = [&](const op_t (&A)[MB], const op_t (&B)[NB]) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if constexpr (X8)
                    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A[m], B[n], acc[m][n], 0, 0, 0,
                                                                                0x7f7f7f7f, 0, 0x7f7f7f7f);
                else
                    acc[m][n] = mma32<T>(A[m], B[n], acc[m][n]);
            }
    };
    // Orders a step's instructions: the reads of the next operands and the fetches
    // of a later stage between the matrix instructions.
    auto mix = [&](auto fetches) {
        constexpr int READS = (X8 ? 2 : 1) * (MB + NB), MUL = MB * NB, F = decltype(fetches)::value;
        constexpr int OTHER = READS + F;
#pragma unroll
        for (int i = 0; i < MUL; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
#pragma unroll
            for (int o = i * OTHER / MUL; o < (i + 1) * OTHER / MUL; ++o) {
                if (o < READS)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                else
                    __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
            }
        }
    };
    typedef std::integral_constant<int, 0> no_fetch;
    typedef std::integral_constant<int, 2 * (MB + NB)> fetch;
    auto stage = [&](int st, unsigned char* cur, unsigned char* nxt) {
#pragma unroll
        for (int s = 0; s + 1 < STEPS; ++s) {
            if (s & 1) {
                read(cur, s + 1, A0, B0);
                mul(A1, B1);
            } else {
                read(cur, s + 1, A1, B1);
                mul(A0, B0);
            }
            mix(no_fetch());
        }
        __builtin_amdgcn_s_waitcnt(0);  // the next stage has arrived, this wave has read the current one
        lds_barrier();
        issue(st + 2, cur);
        read(nxt, 0, A0, B0);
        mul(A1, B1);
        mix(fetch());
    };
    // An odd number of stages ends with one of zeros; so do the fetches past the last.
    issue(0, buf0);
    __builtin_amdgcn_s_waitcnt(0);
    lds_barrier();
    issue(1, buf1);
    read(buf0, 0, A0, B0);
    for (int st = 0; st < nst; st += 2) {
        stage(st, buf0, buf1);
        stage(st + 1, buf1, buf0);
    }
    __builtin_amdgcn_s_waitcnt(0);  // no fetch is under way when LDS is used again
    lds_barrier();

    // 2^-e, e the exponent of a token's largest |v|
    auto power = [&](float top) {
        int e = (int)((__builtin_bit_cast(unsigned, top) >> 23) & 255u) - 127;
        e = e < -24 ? -24 : e > 120 ? 120 : e;
        return __builtin_bit_cast(float, (unsigned)(127 - e) << 23);
    };
    // The tile's low-rank values go to LDS as B operands, high and low part:
    // [16 ranks][part][hi][token] pieces of eight.
    const int nrs = (a.rank + 15) / 16;
    auto at = [&](int rs, int part, int half, int t) {
        unsigned char* b = rs < 4 ? buf0 + rs * 64 * BN : buf1 + (rs - 4) * 64 * BN;
        return reinterpret_cast<u32x4*>(b + (((part * 2 + half) * BN + t) * 16));
    };
    if (a.rank) {
        if (tid < BN && n0 + tid < a.tokens) {
            const int token = n0 + tid;
            const int id = adapter_of(a, token);
            if (id >= 0) {
                const float alpha = a.lora_alpha ? a.lora_alpha[id] : 1.0f;
                auto eight = [&](int r, float (&v)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                    for (int sl = 0; sl < a.slices; ++sl) {
                        const float* p = a.part + ((long)sl * a.tokens + token) * a.rank + r;
                        const f32x4 p0 = *reinterpret_cast<const f32x4*>(p);
                        const f32x4 p1 = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] += p0[e];
                            v[4 + e] += p1[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= alpha;
                };
                float down = 1.0f;
                if constexpr (!V16<T>::BF) {
                    float top = 0.0f;
                    for (int r = 0; r < a.rank; r += 8) {
                        float v[8];
                        eight(r, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
                    }
                    down = power(top);
                    down_lds[tid] = down;
                }
                for (int r = 0; r < 16 * nrs; r += 8) {
                    v8 vh, vl;
                    float v[8];
                    if (r < a.rank) {
                        eight(r, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = v[e] * down;
                        vh[e] = (T)f;
                        vl[e] = __builtin_isfinite((float)vh[e]) ? (T)(f - (float)vh[e]) : (T)0.0f;
                    }
                    *at(r >> 4, 0, (r >> 3) & 1, tid) = __builtin_bit_cast(u32x4, vh);
                    *at(r >> 4, 1, (r >> 3) & 1, tid) = __builtin_bit_cast(u32x4, vl);
                }
            }
        }
        lds_barrier();
    }

    // 32 x 32 blocks one by one; lane (hi, l32) holds channels 8j + 4hi + 0..3 of one token
    const rsrc_t rs = make_rsrc(a.scale, a.scale ? 4u * (unsigned)a.cout : 0u);
    const rsrc_t rb = make_rsrc(a.bias, a.bias ? 4u * (unsigned)a.cout : 0u);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int tt = (wn * NB + n) * 32 + l32, token = n0 + tt;
        const float sx = X8 && token < a.tokens ? a.x_scale[token] : 1.0f;
        const int id = a.rank ? adapter_of(a, token) : -1;
        const unsigned long long ids = __ballot(id >= 0) & 0xffffffffull;
        float down = 1.0f, up = 1.0f;
        if constexpr (!V16<T>::BF) {
            if (id >= 0) {
                down = down_lds[tt];
                up = 1.0f / down;  // a power of two: exact
            }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int cm = m0 + (wm * MB + m) * 32;
            f32x16 z;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = cm + 8 * j + 4 * hi;
                const unsigned off = c < a.cout ? 4u * (unsigned)c : kOOB;
                f32x4 sc = __builtin_bit_cast(f32x4, bload128(rs, off));
                const f32x4 bi = __builtin_bit_cast(f32x4, bload128(rb, off));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!a.scale) sc[i] = 1.0f;
                    z[4 * j + i] = fmaf(X8 ? acc[m][n][4 * j + i] * sx : acc[m][n][4 * j + i], sc[i], bi[i]);
                }
            }
            unsigned long long todo = ids;
            while (todo) {  // each pass clears at least its first bit
                const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
                const bool mine = id == d;
                todo &= ~__ballot(mine);
                const rsrc_t rbm = make_rsrc(static_cast<const T*>(a.lora_b) + (long)d * a.cout * a.rank,
                                             (unsigned)a.cout * (unsigned)a.rank * 2u);
                const unsigned row = cm + l32 < a.cout ? (unsigned)(cm + l32) * (unsigned)a.rank * 2u : kOOB;
                f32x16 c;
#pragma unroll
                for (int i = 0; i < 16; ++i) c[i] = V16<T>::BF ? z[i] : z[i] * down;
                for (int r16 = 0; r16 < nrs; ++r16) {
                    const int r = 16 * r16 + 8 * hi;
                    const u32x4 b = bload128(rbm, r < a.rank ? row + 2u * (unsigned)r : kOOB);
                    c = mma32<T>(b, *at(r16, 1, hi, tt), c);
                    c = mma32<T>(b, *at(r16, 0, hi, tt), c);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = mine ? (V16<T>::BF ? c[i] : c[i] * up) : z[i];
            }
            if (token < a.tokens) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = cm + 8 * j + 4 * hi;
                    if (c >= a.cout) continue;
                    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (a.res) {
                        const v4 rv = *reinterpret_cast<const v4*>(static_cast<const T*>(a.res) + (long)token * a.rs + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[i] = (float)rv[i];
                    }
                    v4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = (T)finish(z[4 * j + i], r[i], a.act, a.res_mode);
                    *reinterpret_cast<v4*>(static_cast<T*>(a.y) + (long)token * a.ys + c) = o;
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // a block at a time: its values are all that is live beside the sums
        }
    }
}

template <typename T, bool X8>
hipError_t launch_tile_t(LinArgs a, const LinPlan& p, hipStream_t s)
{
    a.tiles_m = (a.cout + 64 * p.mb - 1) / (64 * p.mb);
    a.tiles_n = (a.tokens + 64 * p.nb - 1) / (64 * p.nb);
    const long n = (long)a.tiles_m * a.tiles_n;
    if (n > (1l << 23)) return hipErrorInvalidValue;  // a grid holds fewer than 2^32 threads
    const dim3 grid((unsigned)n);
    if (p.mb == 4 && p.nb == 4)
        hipLaunchKernelGGL((k_linear_tile<T, X8, 4, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_tile<T, X8, 2, 2>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tile(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s)
{
    if (dtype == CVX_DT_F16) return x8 ? launch_tile_t<half_t, true>(a, p, s) : launch_tile_t<half_t, false>(a, p, s);
    return x8 ? launch_tile_t<bf16_t, true>(a, p, s) : launch_tile_t<bf16_t, false>(a, p, s);
}

LinPlan linear_plan(const cvx_linear_desc& d)
{
    LinPlan p;
    p.few = d.tokens <= 64;
    p.nt = d.tokens <= 16 ? 1 : d.tokens <= 32 ? 2 : 4;
    const long big = (long)((d.c_out + 255) / 256) * ((d.tokens + 255) / 256);
    p.mb = p.nb = big >= 192 ? 4 : 2;
    p.slices = p.slice_chunks = 0;
    p.ws_bytes = 0;
    if (d.rank) {
        // slices of c_in until the first product's grid fills the device
        const long chunks = (d.c_in + kLoraChunk - 1) / kLoraChunk;
        const long blocks = (long)((d.tokens + 15) / 16) * ((d.rank + 15) / 16);
        long want = (512 + blocks - 1) / blocks;
        if (want > chunks) want = chunks;
        p.slice_chunks = (int)((chunks + want - 1) / want);
        p.slices = (int)((chunks + p.slice_chunks - 1) / p.slice_chunks);
        p.ws_bytes = (size_t)p.slices * d.tokens * d.rank * sizeof(float);
    }
    return p;
}

void linear_describe(const cvx_linear_desc& d, const LinPlan& p, char* buf, int len)
{
    const char* t = d.dtype == CVX_DT_F16 ? "_Float16" : "__bf16";
    const char* x8 = d.x_dtype == CVX_DT_E4M3 ? "true" : "false";
    char lora[64] = "";
    if (d.rank) snprintf(lora, sizeof lora, " rank=%d slices=%d", d.rank, p.slices);
    if (p.few)
        snprintf(buf, len, "linear few 16x%d%s kernel=cvx::k_linear_few<%s, %s, %d>", 16 * p.nt, lora, t, x8, p.nt);
    else
        snprintf(buf, len, "linear tile %dx%d%s kernel=cvx::k_linear_tile<%s, %s, %d, %d>", 64 * p.mb, 64 * p.nb, lora,
                 t, x8, p.mb, p.nb);
}

}  // namespace cvx
