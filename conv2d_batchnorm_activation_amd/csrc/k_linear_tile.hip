// k_linear_tile.hip -- projection of many tokens: a tile of 64*MB output
// channels x 64*NB tokens a workgroup, on the matrix cores.
//
// The weights are the A operand (rows = output channels) and the tokens the B
// operand (columns = tokens), so a lane's accumulators are channels of one
// token.  A stage is 128 bytes of every row of both operands, loaded straight
// into LDS; the 16-byte pieces of a row are permuted by the row's index as they
// are fetched, so that the lanes of an operand read (32 rows, the same piece) fall
// in different banks while every fetch still takes whole 128-byte lines.  Stage
// s+1 (and, with four stage buffers, up to s+3) arrives while s is multiplied; a
// stage has one barrier, before which a wave waits for its own fetches of the next
// stage only, and which drains nothing: a fence there waited for every fetch under
// way (512 tokens, 4096 -> 4096 channels, 34 us instead of 22).
//
// Measured: 4096^3 bf16 105 to 114 us (1200 to 1310 TFLOP/s; the library's product
// 99), the matrix pipes busy half of the cycles that 2.4 GHz would give; 8192 x 4096
// x 14336 e4m3 386 to 402 us (2400 to 2490), 0.47.  512 tokens, 4096 -> 4096: 22 us,
// 256 workgroups of one tile, the pipes busy 0.31: 84 MB come past the XCDs' caches
// for 38 MB of operands, 4 TB/s, and 24 KB a stage of 0.28 us into every compute
// unit.  Tiles go in whole rounds of 256: 559 tokens of 8048 -> 7436 are 531 tiles of
// 128x128, three rounds, 192 us, the pipes at 0.15.
//
// 8-bit operands (e4m3) are the same bytes: a stage is 128 channels instead of
// 64, and the 32x32x64 instruction takes two pieces a lane where the 16-bit
// one takes one.  Any assignment of k to lanes serves, as long as both operands
// use the same.  The 8-bit instructions align the products of eight consecutive
// channels to the largest of them and drop what lies 2^-13 below it (the sums of
// these groups are fp32), in this form and in the older 32x32x16 one alike.  Measured
// before the output's rounding, 1024 channels: off by 1.5e-5 of the result's size
// (root mean square) for normal values, without a bias to either side, 5.3e-5 with
// one channel in 64 a hundred times larger (fp32 sums: 3e-8, 5e-8).  The output's
// own rounding is 1.7e-3 in bf16 and 2.1e-4 in fp16, which becomes 2.2e-4 with such
// channels.  Taken for the rate: the same product of values held in 16 bits, whose
// sums are fp32, is 726 us.
//
// Adapters: once the sums stand in registers they get scale and bias, and the
// second product of the adapters is accumulated onto them by the same matrix
// instructions: for every 32 tokens, each distinct adapter's rows of B, with v
// as two 16-bit values (v = high + low, so v keeps 16 bits in bf16 and 21 in
// fp16; k_lora_join makes them, or the tile itself); the lanes whose token names the adapter keep the
// result.  fp16, whose range v may leave, takes v divided by a power of two per
// token, and the product is added to the sums when it is whole.
#include <stdio.h>

#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

// Orders this wave's LDS accesses (which the hardware keeps in order) for the compiler.
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

template <bool X8>
struct Op {
    typedef typename std::conditional<X8, i32x8, u32x4>::type type;
};

// WM x WN waves, each MB x NB blocks of 32 x 32; D stage buffers.
template <typename T, bool X8, bool LORA, int WM, int WN, int MB, int NB, int D>
__global__ void __launch_bounds__(64 * WM * WN, D == 2 ? 2 : 1) k_linear_tile(LinArgs a)
{
    typedef typename V16<T>::v4 v4;
    typedef typename Op<X8>::type op_t;
    constexpr unsigned XB = X8 ? 1 : 2;
    constexpr int W = WM * WN, NT = 64 * W;
    constexpr int BM = 32 * WM * MB, BN = 32 * WN * NB;
    constexpr int FM = BM / (8 * W), FN = BN / (8 * W);  // fetches of eight rows a wave, per stage and operand
    constexpr int STEPS = X8 ? 2 : 4;
    constexpr int SB = (BM + BN) * 128;  // bytes of a stage
    static_assert(D == 2 || D == 4, "stage buffers");
    static_assert(W * 4096 <= SB && MB % 2 == 0, "LDS is used again after the main loop");
    // an array a stage, so that waits are for the stage read, not for every fetch
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[SB], buf1[SB], buf2[D == 4 ? SB : 16],
        buf3[D == 4 ? SB : 16];
    __shared__ __attribute__((aligned(16))) float sc_lds[BM], bi_lds[BM];
    __shared__ float sx_lds[X8 ? BN : 1];
    __shared__ int id_lds[LORA ? BN : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
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
    const char* wt = static_cast<const char*>(a.w) + (long)m0 * cb;
    const char* xt = static_cast<const char*>(a.x) + (long)n0 * pitch;
    const int nst = (int)((cb + 127) / 128);

    // A fetch is eight rows of 128 bytes, eight lanes a row.  Rows past the operand
    // are past the range of its descriptor, pieces past the end of a row are sent
    // there.  The 16-byte pieces of row r lie permuted, piece p at p ^ (r/2 % 8): the
    // sixteen lanes of an operand read that go together (0-3, 12-15, 20-27 of 32,
    // or the others) then fall in all of the banks.
    static_assert(W % 2 == 0, "a wave's fetches begin at rows 8 * wave + 16 * i");
    const unsigned piece = (unsigned)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
    static_assert(FM <= 8 && FN <= 8, "fetches a wave");
    unsigned wo[8], xo[8];
#pragma unroll
    for (int i = 0; i < FM; ++i) wo[i] = (unsigned)(8 * (wave + W * i) + (lane >> 3)) * cb + piece;
#pragma unroll
    for (int i = 0; i < FN; ++i) xo[i] = (unsigned)(8 * (wave + W * i) + (lane >> 3)) * pitch + piece;
    auto issue = [&](int st, unsigned char* buf) {
        const unsigned kb = (unsigned)st * 128 < cb ? (unsigned)st * 128 : 0u;  // past the end: nothing is live
        const unsigned dead = (unsigned)st * 128 + piece < cb ? 0u : kOOB;
        const char *wk = wt + kb, *xk = xt + kb;
        const unsigned wleft = (unsigned)mrows * cb - kb, xleft = (unsigned)(nrows - 1) * pitch + cb - kb;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(wk, wleft), (lds_void*)(buf + 1024 * (wave + W * i)), 16,
                                                     wo[i] | dead, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < FN; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(xk, xleft),
                                                     (lds_void*)(buf + BM * 128 + 1024 * (wave + W * i)), 16,
                                                     xo[i] | dead, 0, 0, 0);
    };
    unsigned slot[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) slot[s] = (unsigned)(l32 * 128 + (((2 * s + hi) ^ ((l32 >> 1) & 7)) * 16));
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
        for (int n = 0; n < NB; ++n) B[n] = one(pb + 4096 * n);
#pragma unroll
        for (int m = 0; m < MB; ++m) A[m] = one(pa + 4096 * m);
    };

    f32x16 acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;
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
    auto mix_all = [&]() {  // the same for a whole stage
        constexpr int READS = (X8 ? 2 : 1) * (MB + NB) * STEPS, MUL = MB * NB * STEPS, OTHER = READS + FM + FN;
#pragma unroll
        for (int i = 0; i < MUL; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
#pragma unroll
            for (int o = i * OTHER / MUL; o < (i + 1) * OTHER / MUL; ++o) {
                if (o % (OTHER / (FM + FN)) == 0)
                    __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
                else
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
    };
    for (int i = tid; i < BM; i += NT) {
        const bool ok = m0 + i < a.cout;
        sc_lds[i] = !a.scale ? 1.0f : ok ? a.scale[m0 + i] : 0.0f;
        bi_lds[i] = a.bias && ok ? a.bias[m0 + i] : 0.0f;
    }
    for (int i = tid; i < BN; i += NT) {
        const int token = n0 + i;
        if (X8) sx_lds[i] = token < a.tokens ? a.x_scale[token] : 0.0f;
        if (LORA) id_lds[i] = adapter_of(a, token);
    }
    // Both loops take D stages; those past the last are zeros, and so are the fetches past it.
    typedef std::integral_constant<int, FM + FN> fetch;
    if constexpr (D == 2) {
        // A step's operands are read under the step before.
        typedef std::integral_constant<int, 0> no_fetch;
        op_t A0[MB], B0[NB], A1[MB], B1[NB];
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
            wait_arrived<0>();  // the next stage has arrived, this wave has read the current one
            stage_barrier();
            issue(st + 2, cur);
            read(nxt, 0, A0, B0);
            mul(A1, B1);
            mix(fetch());
        };
        issue(0, buf0);
        wait_arrived<0>();
        stage_barrier();
        issue(1, buf1);
        read(buf0, 0, A0, B0);
        for (int st = 0; st < nst; st += 2) {
            stage(st, buf0, buf1);
            stage(st + 1, buf1, buf0);
        }
    } else {
        // One wave a SIMD: a stage's operands are all read under the stage before, as
        // a step's products (four instructions) are shorter than a read takes.
        op_t A0[STEPS][MB], B0[STEPS][NB], A1[STEPS][MB], B1[STEPS][NB];
        auto read_all = [&](const unsigned char* buf, op_t(&A)[STEPS][MB], op_t(&B)[STEPS][NB]) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) read(buf, s, A[s], B[s]);
        };
        auto stage = [&](int st, unsigned char* cur, unsigned char* nxt, op_t(&A)[STEPS][MB], op_t(&B)[STEPS][NB],
                         op_t(&An)[STEPS][MB], op_t(&Bn)[STEPS][NB]) {
            wait_arrived<2 * (FM + FN)>();  // the next stage has arrived, this wave has read the current one
            stage_barrier();
            issue(st + 4, cur);
            read_all(nxt, An, Bn);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) mul(A[s], B[s]);
            mix_all();
        };
        issue(0, buf0);
        issue(1, buf1);
        issue(2, buf2);
        issue(3, buf3);
        wait_arrived<3 * (FM + FN)>();
        stage_barrier();
        read_all(buf0, A0, B0);
        for (int st = 0; st < nst; st += 4) {
            stage(st, buf0, buf1, A0, B0, A1, B1);
            stage(st + 1, buf1, buf2, A1, B1, A0, B0);
            stage(st + 2, buf2, buf3, A0, B0, A1, B1);
            stage(st + 3, buf3, buf0, A1, B1, A0, B0);
        }
    }
    wait_arrived<0>();  // no fetch is under way when LDS is used again
    stage_barrier();

    // 32 tokens at a time; lane (hi, l32) holds channels 8j + 4hi + 0..3 of one
    // token.  A load waits for the stores before it, so finished values are kept,
    // packed, until all are done; they are turned in LDS, so that a store takes
    // whole lines.  Rows past the last token are past the residual's and the
    // output's range.
    const rsrc_t rres = make_rsrc(static_cast<const T*>(a.res) + (long)n0 * a.rs,
                                  a.res ? (unsigned)((nrows - 1) * a.rs + a.cout) * 2u : 0u);
    const rsrc_t ry = make_rsrc(static_cast<T*>(a.y) + (long)n0 * a.ys, (unsigned)((nrows - 1) * a.ys + a.cout) * 2u);
    v4 out[NB][MB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int t = (wn * NB + n) * 32 + l32;
        const float sx = X8 ? sx_lds[t] : 1.0f;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (wm * MB + m) * 32 + 8 * j + 4 * hi;
                const f32x4 sc = *reinterpret_cast<const f32x4*>(sc_lds + c);
                const f32x4 bi = *reinterpret_cast<const f32x4*>(bi_lds + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = acc[m][n][4 * j + i];
                    acc[m][n][4 * j + i] = fmaf(X8 ? z * sx : z, sc[i], bi[i]);
                }
            }

        if constexpr (LORA) {
            const int id = id_lds[t];
            unsigned long long todo = __ballot(id >= 0) & 0xffffffffull;
            // this lane's pieces of v: [eight ranks][part][token]; past the last token, its
            const long here = n0 + t < a.tokens ? n0 + t : a.tokens - 1;
            const u32x4* v = reinterpret_cast<const u32x4*>(a.joined) + (2l * hi * a.tokens + here);
            float down = 1.0f;
            u32x4 vh0, vl0;  // the first sixteen ranks' pieces
            if constexpr (D == 4) {
                if (a.joined) {
                    vh0 = v[0];
                    vl0 = v[a.tokens];
                    if (!V16<T>::BF && id >= 0) down = a.down[here];
                } else {  // up to sixteen ranks, joined here
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = 0.0f;
                    if (id >= 0 && 8 * hi < a.rank) lora_values(a, id, here, 8 * hi, f);
                    if constexpr (!V16<T>::BF) {
                        const float top = lora_top(f);
                        down = lora_factor(fmaxf(top, __shfl_xor(top, 32)));
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] *= down;
                    }
                    lora_parts<T>(f, vh0, vl0);
                }
            } else if (!V16<T>::BF && id >= 0) {
                down = a.down[here];
            }
            const float up = 1.0f / down;  // a power of two: exact
            while (todo) {  // each pass clears at least the first bit
                const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
                const bool mine = id == d;
                todo &= ~__ballot(mine);
                const rsrc_t rbm = make_rsrc(static_cast<const T*>(a.lora_b) + (long)d * a.cout * a.rank,
                                             (unsigned)a.cout * (unsigned)a.rank * 2u);
#pragma unroll
                for (int mh = 0; mh < MB; mh += 2) {
                    unsigned row[2];  // this lane's rows of the adapter's B
                    f32x16 c[2];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int ch = m0 + (wm * MB + mh + m) * 32 + l32;
                        row[m] = ch < a.cout ? (unsigned)ch * (unsigned)a.rank * 2u + 16u * hi : kOOB;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            c[m][i] = V16<T>::BF ? acc[mh + m][n][i] : 0.0f;
                    }
                    for (int r0 = 0; r0 < a.rank; r0 += 32) {
                        u32x4 b[2][2];
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                b[s][m] = bload128(
                                    rbm, r0 + 16 * s + 8 * hi < a.rank ? row[m] + 2u * (unsigned)(r0 + 16 * s) : kOOB);
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            if (r0 + 16 * s < a.rank) {
                                u32x4 vh = vh0, vl = vl0;
                                if (D != 4 || r0 + s > 0) {
                                    vh = v[(r0 / 4 + 4l * s) * a.tokens];
                                    vl = v[(r0 / 4 + 4l * s + 1) * a.tokens];
                                }
#pragma unroll
                                for (int m = 0; m < 2; ++m) c[m] = mma32<T>(b[s][m], vl, c[m]);
#pragma unroll
                                for (int m = 0; m < 2; ++m) c[m] = mma32<T>(b[s][m], vh, c[m]);
                            }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[mh + m][n][i] = !mine          ? acc[mh + m][n][i]
                                                : V16<T>::BF ? c[m][i]
                                                             : fmaf(c[m][i], up, acc[mh + m][n][i]);
                }
            }
        }

        // residual and activation, each step over all values: one branch a step
#pragma unroll
        for (int mh = 0; mh < MB; mh += 2) {
            v4 rv[2][4];
            auto add_residual = [&]() {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[mh + m][n][i] += (float)rv[m][i / 4][i % 4];
            };
            auto activate = [&](auto act) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[mh + m][n][i] = apply_act_nan(acc[mh + m][n][i], decltype(act)::value);
            };
            if (a.res) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = m0 + (wm * MB + mh + m) * 32 + 8 * j + 4 * hi;
                        const unsigned off = c < a.cout ? (unsigned)t * (unsigned)a.rs * 2u + 2u * (unsigned)c : kOOB;
                        rv[m][j] = __builtin_bit_cast(v4, bload64(rres, off));
                    }
                if (a.res_mode == CVX_RES_BEFORE_ACT) add_residual();
            }
            if (a.act == CVX_ACT_RELU) activate(std::integral_constant<int, CVX_ACT_RELU>());
            if (a.act == CVX_ACT_SILU) activate(std::integral_constant<int, CVX_ACT_SILU>());
            if (a.res_mode == CVX_RES_AFTER_ACT) add_residual();
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 16; ++i) out[n][mh + m][i / 4][i % 4] = (T)acc[mh + m][n][i];
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    unsigned char* turn = buf0 + wave * 4096;
    const int p = lane & 7;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; m += 2) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<v4*>(turn + l32 * 128 + ((k ^ (l32 & 7)) * 16) + 8 * hi) = out[n][m + k / 4][k % 4];
            wave_lds_order();
            const int c = m0 + (wm * MB + m) * 32 + 8 * p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tt = 8 * i + (lane >> 3), t = (wn * NB + n) * 32 + tt;
                const u32x4 q = *reinterpret_cast<const u32x4*>(turn + tt * 128 + ((p ^ (tt & 7)) * 16));
                const unsigned off = ((unsigned)t * (unsigned)a.ys + (unsigned)c) * 2u;
                const bool live = t < nrows;
                __builtin_amdgcn_raw_buffer_store_b128(q, ry, live && c + 8 <= a.cout ? (int)off : (int)kOOB, 0, 0);
                if (a.cout & 4)  // the last four channels of a row
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{q[0], q[1]}, ry,
                                                          live && c + 4 == a.cout ? (int)off : (int)kOOB, 0, 0);
            }
            wave_lds_order();
        }
}

template <typename T, bool X8, int WM, int WN, int MB, int NB, int D>
void launch_tile_k(const LinArgs& a, dim3 grid, hipStream_t s)
{
    if (a.rank)
        hipLaunchKernelGGL((k_linear_tile<T, X8, true, WM, WN, MB, NB, D>), grid, dim3(64 * WM * WN), 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_tile<T, X8, false, WM, WN, MB, NB, D>), grid, dim3(64 * WM * WN), 0, s, a);
}

template <typename T, bool X8>
hipError_t launch_tile_t(LinArgs a, const LinPlan& p, hipStream_t s)
{
    a.tiles_m = (a.cout + 64 * p.mb - 1) / (64 * p.mb);
    a.tiles_n = (a.tokens + 64 * p.nb - 1) / (64 * p.nb);
    const dim3 grid((unsigned)((long)a.tiles_m * a.tiles_n));  // few enough: tokens * c_out is at most 2^37
    if (p.mb == 4)
        launch_tile_k<T, X8, 2, 4, 4, 2, 2>(a, grid, s);
    else if (p.nb == 2)
        launch_tile_k<T, X8, 2, 2, 2, 2, 4>(a, grid, s);
    else
        launch_tile_k<T, X8, 2, 2, 2, 1, 4>(a, grid, s);
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
    // 4096 -> 4096 channels, bf16: 16 tokens 7.6 us (16.1 by the tile kernel), 32 8.6
    // (16.5), 64 12.3 (17.9); 64 tokens of rank 16, eight adapters in turn, 21 (40).
    // Of 8-bit operands 64 tokens to 8192 channels are 16.0 us and would be 11.8 by
    // tiles, whose instructions drop what this kernel keeps.
    // More tokens go there in blocks of 64 where that is at most a workgroup a compute
    // unit, as there would be fewer tiles still, and c_in is long enough: 128 tokens to
    // 2048 channels from 4096 12.8 us (18.1 by tiles), from 2048 8.3 (11.2), of rank 16
    // 17.0 (18.6); 256 tokens, 4096 to 1024, rank 32 23.4 (27.8), rank 64 30.7 (29.5);
    // 200 tokens, 8192 to 1024, rank 64 39 (47); 1024 tokens, 1024 to 256, rank 16 16.6
    // (13.6).
    p.few = d.tokens <= 64 ||
            (d.x_dtype == d.dtype && d.c_in >= 64 * (d.rank > 32 ? d.rank : 32) &&
             (long)((d.c_out + 15) / 16) * ((d.tokens + 63) / 64) <= 256);
    // The adapter's A is read by every workgroup: 4096 channels to 4096 9.2 us (12.2 with
    // a launch of its own), to 8192 16.4 (18.4), to 12288 27.1 (27.3), to 14336 35.7
    // (33.7); 1024 to 16384 17.6 (20.7).
    p.one = d.tokens == 1 && d.rank > 0 && d.rank <= 16 && d.x_dtype == d.dtype &&
            (long)d.c_in * d.c_out <= 3l << 24;
    p.nt = d.tokens <= 16 ? 1 : d.tokens <= 32 ? 2 : 4;
    // 32 channels a workgroup where 16 would be more than a workgroup a compute unit:
    // 64 tokens, 4096 channels to 4096 12.6 us (15.5 with 32), to 5120 21.6 (15.9), to
    // 8192 22.2 (17.3).
    p.rb = p.nt == 4 && d.c_out > 16 * 256 ? 2 : 1;
    // The tile that ends first by what a stage (128 bytes of every row) and the rest
    // of a tile measured, in 10 ns, with the tiles one a compute unit.  4096 -> 4096
    // channels, bf16: 512 tokens 22 us as 128x64 (256 tiles; 31 as 128x128), 1024
    // tokens 32 us as 128x128 (256 tiles; 44 as 128x64), 4096 tokens 105 us as
    // 256x256 (256 tiles; 130 as 128x128).
    const struct {
        int mb, nb, stage, rest;
    } tiles[] = {{4, 4, 150, 1000}, {2, 2, 45, 500}, {2, 1, 28, 400}};
    const long stages = ((long)d.c_in * (d.x_dtype == CVX_DT_E4M3 ? 1 : 2) + 127) / 128;
    long best = -1;
    for (const auto& t : tiles) {
        const long n = (long)((d.c_out + 64 * t.mb - 1) / (64 * t.mb)) * ((d.tokens + 64 * t.nb - 1) / (64 * t.nb));
        const long time = (n + 255) / 256 * (stages * t.stage + t.rest);
        if (best >= 0 && time >= best) continue;
        best = time;
        p.mb = t.mb;
        p.nb = t.nb;
    }
    p.slices = p.slice_len = p.join = p.down_nb = p.down_rc = 0;
    p.ws_bytes = 0;
    if (d.rank && !p.one) {
        // Blocks of one token up to 64, of 16 up to 2047, of 64 above.  A whole projection
        // from 4096 to 4096 channels, tokens by tokens of the same adapter together:
        // 128 tokens of rank 64 32 us with 16 (38 with one; 154 and 130 if every token has
        // an adapter of its own), 1024 tokens 53 with 16 (50 with 64), 2048 98 with 16
        // (88 with 64), 4096 156 (137).  Up to 2047 tokens may be as many requests.
        // Slices of c_in until the first product's grid fills the device.
        p.down_nb = d.tokens <= 64 ? 0 : d.tokens < 2048 ? 1 : 4;
        p.down_rc = p.down_nb < 4 || d.rank <= 16 ? 1 : d.rank <= 32 ? 2 : 4;
        const int tok = p.down_nb ? 16 * p.down_nb : 1, step = p.down_nb == 4 ? kLoraMany : kLoraChunk;
        const long chunks = (d.c_in + step - 1) / step;
        const long blocks = (long)((d.tokens + tok - 1) / tok) * ((d.rank + 16 * p.down_rc - 1) / (16 * p.down_rc));
        long want = ((p.down_nb == 4 ? 768 : 512) + blocks - 1) / blocks;
        if (want > chunks) want = chunks;
        const int per = (int)((chunks + want - 1) / want);
        p.slice_len = per * step;
        p.slices = (int)((chunks + per - 1) / per);
        p.ws_bytes = (size_t)p.slices * d.tokens * d.rank * sizeof(float);
        // Tiles of one wave a SIMD have registers for the slices of up to 16 ranks: there
        // each joins its tokens' itself, which spares a launch (512 tokens 4096 -> 4096
        // channels, rank 16: 32.7 -> 30.4 us).  More ranks are as many loads at every tile's end.
        p.join = !p.few && (p.mb == 4 || d.rank > 16 || p.slices > 8);
        if (p.join) p.ws_bytes += lora_joined_bytes(d.tokens, d.rank) + (size_t)d.tokens * sizeof(float);
    }
    return p;
}

void linear_describe(const cvx_linear_desc& d, const LinPlan& p, char* buf, int len)
{
    const char* t = d.dtype == CVX_DT_F16 ? "_Float16" : "__bf16";
    const char* x8 = d.x_dtype == CVX_DT_E4M3 ? "true" : "false";
    char lora[64] = "";
    if (p.one)
        snprintf(lora, sizeof lora, " rank=%d", d.rank);
    else if (d.rank)
        snprintf(lora, sizeof lora, " rank=%d slices=%d", d.rank, p.slices);
    if (p.few)
        snprintf(buf, len, "linear few %dx%d%s kernel=cvx::k_linear_few<%s, %s, %s, %d, %d, %d, %d, %d>", 16 * p.rb,
                 16 * p.nt, lora, t, x8, p.one ? "true" : "false", p.nt == 1 ? 8 : 4, p.rb, p.nt,
                 d.tokens <= 8 ? 8 : 16 * p.nt, p.nt == 4 || p.one ? 3 : 4);
    else
        snprintf(buf, len, "linear tile %dx%d%s kernel=cvx::k_linear_tile<%s, %s, %s, 2, %d, %d, %d, %d>", 64 * p.mb, 64 * p.nb,
                 lora, t, x8, d.rank ? "true" : "false", p.mb == 4 ? 4 : 2, p.mb, p.mb == 4 ? 2 : p.nb,
                 p.mb == 4 ? 2 : 4);
}

}  // namespace cvx
