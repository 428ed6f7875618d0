// lin_tile.h -- the products of a tile of output channels x tokens on the matrix
// cores, which the projection of many tokens and the products grouped by expert share.
//
// A stage is 128 bytes of every row of both operands, loaded straight into LDS; the
// 16-byte pieces of a row are permuted by the row's index as they are fetched, so that
// the lanes of an operand read (32 rows, the same piece) fall in different banks while
// every fetch still takes whole 128-byte lines.  Stage s+1 (and, with four stage
// buffers, up to s+3) arrives while s is multiplied; a stage has one barrier, before
// which a wave waits for its own fetches of the next stage only, and which drains
// nothing.
#pragma once

#include "lin_common.h"

namespace cvx {

// Orders this wave's LDS accesses (which the hardware keeps in order) for the compiler.
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// The operands of a tile: rows of `cb` bytes; lane's byte offsets of its fetches
// (eight rows each; a row that is not there at kOOB or past the range) from bases that
// move with the stage, and the bytes from a base to its operand's end.
struct TileRows {
    const char *w, *x;
    unsigned wend, xend;
    unsigned wo[8], xo[8];
};

// A tile's stage buffers, an array each, so that waits are for the stage read and not for
// every fetch.
struct Stages {
    unsigned char* at[4];
};

// T: 16-bit type; X: what the operands are held in (kX16: T).  WM x WN waves, each
// MB x NB blocks of 32 x 32; D stage buffers; a stage is RB bytes of every row.  WIDE:
// e4m3 values are widened to 16 bits, exactly, and multiplied as such.
template <typename T, int X, int WM, int WN, int MB, int NB, int D, int RB = 128, bool WIDE = false>
struct Tile {
    static constexpr bool X8 = X == kXE4m3;
    static constexpr bool I8 = X == kXI8;
    static constexpr unsigned XB = X == kX16 ? 2 : 1;  // bytes of an operand's value
    static constexpr int W = WM * WN, NT = 64 * W;
    static constexpr int BM = 32 * WM * MB, BN = 32 * WN * NB;
    static constexpr int RF = 1024 / RB;                          // rows of a fetch
    static constexpr int FM = BM / (RF * W), FN = BN / (RF * W);  // fetches a wave, per stage and operand
    static constexpr int STEPS = RB / (X8 ? 64 : 32);
    static constexpr int SB = (BM + BN) * RB;  // bytes of a stage
    static_assert(W == 8 ? D == 2 && STEPS % 2 == 0 : W == 4 && D == 4, "stage buffers");
    static_assert(MB % 2 == 0, "values are stored 64 channels at a time");
    static_assert(W % 2 == 0, "a wave's fetches begin at rows 8 * wave + 16 * i");
    static_assert(FM <= 8 && FN <= 8, "fetches a wave");
    static_assert(!WIDE || (X8 && W == 4), "values to widen");
    typedef typename V16<T>::v4 v4;
    typedef typename std::conditional<X8, i32x8, u32x4>::type op_t;
    // sums: of 8-bit integers exact ones
    typedef typename std::conditional<I8, i32x16, f32x16>::type sum_t;

    // The 16-byte piece this lane fetches of its row of a fetch: the pieces of row r lie
    // permuted, piece p at p ^ (r/2 % 8), of 64-byte rows at p ^ (r/4 % 4); the sixteen lanes
    // of an operand read that go together (0-3, 12-15, 20-27 of 32, or the others) then
    // fall in all of the banks.
    static __device__ __forceinline__ unsigned piece(int wave, int lane)
    {
        if (RB == 64) return (unsigned)((lane & 3) ^ (lane >> 4)) * 16;
        return (unsigned)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
    }
    // The row of the tile that this lane's part of fetch i is of.
    static __device__ __forceinline__ int fetch_row(int wave, int lane, int i)
    {
        return RF * (wave + W * i) + lane / (RB / 16);
    }

    // The fetches of stage `st` of a tile into a stage buffer.
    static __device__ __forceinline__ void issue(const TileRows& o, unsigned cb, int st, unsigned char* buf, int wave,
                                                 int lane)
    {
        const unsigned pc = piece(wave, lane);
        const unsigned kb = (unsigned)st * RB < cb ? (unsigned)st * RB : 0u;  // past the end: nothing is live
        const unsigned dead = (unsigned)st * RB + pc < cb ? 0u : kOOB;
        const char *wk = o.w + kb, *xk = o.x + kb;
        const unsigned wleft = o.wend - kb, xleft = o.xend - kb;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(wk, wleft), (lds_void*)(buf + 1024 * (wave + W * i)), 16,
                                                     o.wo[i] | dead, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < FN; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(xk, xleft),
                                                     (lds_void*)(buf + BM * RB + 1024 * (wave + W * i)), 16,
                                                     o.xo[i] | dead, 0, 0, 0);
    }
    // The first D stages.
    static __device__ __forceinline__ void begin(const TileRows& o, unsigned cb, int wave, int lane, const Stages& bufs)
    {
#pragma unroll
        for (int i = 0; i < D; ++i) issue(o, cb, i, bufs.at[i], wave, lane);
    }

    // The sums over all stages of rows of cb bytes, of the first 32*WN*NL rows of the
    // tile (wave wn takes NL blocks of them).  All waves of the workgroup call it.
    // BEGUN: the tile's first D stages are under way.  Else nothing is under way in LDS
    // before it, and after it nothing in either case.
    template <bool BEGUN, int NL>
    static __device__ __forceinline__ void sums(const TileRows& o, unsigned cb, int wave, int lane, const Stages& bufs,
                                                sum_t (&acc)[MB][NL])
    {
        const int wm = wave % WM, wn = wave / WM;
        const int hi = lane >> 5, l32 = lane & 31;
        const int nst = (int)((cb + RB - 1) / RB);
        auto issue = [&](int st, unsigned char* buf) { Tile::issue(o, cb, st, buf, wave, lane); };
        unsigned slot[RB / 32];
#pragma unroll
        for (int s = 0; s < RB / 32; ++s)
            slot[s] = (unsigned)(l32 * RB + (((2 * s + hi) ^ (RB == 64 ? (l32 >> 2) & 3 : (l32 >> 1) & 7)) * 16));
        auto read = [&](const unsigned char* buf, int st, op_t(&A)[MB], op_t(&B)[NL]) {
            const unsigned char* pa = buf + wm * MB * 32 * RB;
            const unsigned char* pb = buf + BM * RB + wn * NL * 32 * RB;
            auto one = [&](const unsigned char* p) {
                if constexpr (X8) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(p + slot[2 * st]);
                    const u32x4 y = *reinterpret_cast<const u32x4*>(p + slot[2 * st + 1]);
                    i32x8 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = (int)x[e];
                        v[4 + e] = (int)y[e];
                    }
                    return v;
                } else {
                    return *reinterpret_cast<const u32x4*>(p + slot[st]);
                }
            };
#pragma unroll
            for (int n = 0; n < NL; ++n) B[n] = one(pb + 32 * RB * n);
#pragma unroll
            for (int m = 0; m < MB; ++m) A[m] = one(pa + 32 * RB * m);
        };

#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NL; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[m][n][e] = 0;
        auto mul = [&](const op_t(&A)[MB], const op_t(&B)[NL]) {
            if constexpr (WIDE) {  // eight values of k a lane at a time
#pragma unroll
                for (int q = 0; q < 8; q += 2) {
                    u32x4 b[NL];
#pragma unroll
                    for (int n = 0; n < NL; ++n) b[n] = widen8<T, X>(u32x2{(unsigned)B[n][q], (unsigned)B[n][q + 1]});
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        const u32x4 a = widen8<T, X>(u32x2{(unsigned)A[m][q], (unsigned)A[m][q + 1]});
#pragma unroll
                        for (int n = 0; n < NL; ++n) acc[m][n] = mma32<T>(a, b[n], acc[m][n]);
                    }
                }
                return;
            }
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int n = 0; n < NL; ++n) {
                    if constexpr (X8)
                        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A[m], B[n], acc[m][n], 0, 0, 0,
                                                                                    0x7f7f7f7f, 0, 0x7f7f7f7f);
                    else if constexpr (I8)
                        acc[m][n] = mma32_i8(A[m], B[n], acc[m][n]);
                    else
                        acc[m][n] = mma32<T>(A[m], B[n], acc[m][n]);
                }
        };
        // Orders a step's instructions: the reads of the next operands and the fetches
        // of a later stage between the matrix instructions.
        auto mix = [&](auto fetches) {
            constexpr int READS = (X8 ? 2 : 1) * (MB + NL), MUL = MB * NL, F = decltype(fetches)::value;
            constexpr int OTHER = READS + F;
#pragma unroll
            for (int i = 0; i < MUL; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
#pragma unroll
                for (int q = i * OTHER / MUL; q < (i + 1) * OTHER / MUL; ++q) {
                    if (q < READS)
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    else
                        __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
                }
            }
        };
        auto mix_all = [&]() {  // the same for a whole stage
            constexpr int READS = (X8 ? 2 : 1) * (MB + NL) * STEPS, MUL = (WIDE ? 4 : 1) * MB * NL * STEPS;
            constexpr int OTHER = READS + FM + FN;
#pragma unroll
            for (int i = 0; i < MUL; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
#pragma unroll
                for (int q = i * OTHER / MUL; q < (i + 1) * OTHER / MUL; ++q) {
                    if (q % (OTHER / (FM + FN)) == 0)
                        __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
                    else
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
            }
        };
        typedef std::integral_constant<int, FM + FN> fetch;
        if constexpr (W == 8) {
            // A step's operands are read under the step before.  Both loops take D stages;
            // those past the last are zeros, and so are the fetches past it.
            typedef std::integral_constant<int, 0> no_fetch;
            op_t A0[MB], B0[NL], A1[MB], B1[NL];
            // A0, B0 hold the first step's operands, and those of the next stage's after it
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
                wait_arrived<(D - 2) * (FM + FN)>();  // the next stage has arrived, this wave has read the current one
                stage_barrier();
                issue(st + D, cur);
                read(nxt, 0, A0, B0);
                mul(A1, B1);
                mix(fetch());
            };
            if constexpr (!BEGUN) begin(o, cb, wave, lane, bufs);
            wait_arrived<(D - 1) * (FM + FN)>();
            stage_barrier();
            read(bufs.at[0], 0, A0, B0);
            for (int st = 0; st < nst; st += D)
#pragma unroll
                for (int i = 0; i < D; ++i) stage(st + i, bufs.at[i], bufs.at[(i + 1) % D]);
        } else {
            // One wave a SIMD: a stage's operands are all read under the stage before, as
            // a step's products (four instructions) are shorter than a read takes.
            op_t A0[STEPS][MB], B0[STEPS][NL], A1[STEPS][MB], B1[STEPS][NL];
            auto read_all = [&](const unsigned char* buf, op_t(&A)[STEPS][MB], op_t(&B)[STEPS][NL]) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) read(buf, s, A[s], B[s]);
            };
            auto stage = [&](int st, unsigned char* cur, unsigned char* nxt, op_t(&A)[STEPS][MB], op_t(&B)[STEPS][NL],
                             op_t(&An)[STEPS][MB], op_t(&Bn)[STEPS][NL]) {
                wait_arrived<(D - 2) * (FM + FN)>();  // the next stage has arrived, this wave has read the current one
                stage_barrier();
                issue(st + D, cur);
                read_all(nxt, An, Bn);
#pragma unroll
                for (int s = 0; s < STEPS; ++s) mul(A[s], B[s]);
                mix_all();
            };
            if constexpr (!BEGUN) begin(o, cb, wave, lane, bufs);
            wait_arrived<(D - 1) * (FM + FN)>();
            stage_barrier();
            read_all(bufs.at[0], A0, B0);
            for (int st = 0; st < nst; st += D)
#pragma unroll
                for (int i = 0; i < D; i += 2) {
                    stage(st + i, bufs.at[i], bufs.at[i + 1], A0, B0, A1, B1);
                    stage(st + i + 1, bufs.at[i + 1], bufs.at[(i + 2) % D], A1, B1, A0, B0);
                }
        }
        wait_arrived<0>();  // no fetch is under way when LDS is used again
        stage_barrier();
    }

    // Writes finished values, `out`[n][m] a lane's sixteen channels of a token, four at a
    // time: they are turned in LDS, TOK tokens (32 or 16) and 128*TOK bytes of `room` a
    // wave at a time, so that a store takes whole lines.  ry: the rows from the tile's
    // first token; m0: its first channel.
    template <int NL, int TOK>
    static __device__ __forceinline__ void store(const v4 (&out)[NL][MB][4], unsigned char* room, int wave, int lane,
                                                 rsrc_t ry, int nrows, unsigned ys, int m0, int cout)
    {
        const int wm = wave % WM, wn = wave / WM;
        const int hi = lane >> 5, l32 = lane & 31;
        unsigned char* turn = room + wave * 128 * TOK;
        const int p = lane & 7;
#pragma unroll
        for (int n = 0; n < NL; ++n)
#pragma unroll
            for (int m = 0; m < MB; m += 2)
#pragma unroll
                for (int part = 0; part < 32 / TOK; ++part) {
                    if (TOK == 32 || l32 / TOK == part) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<v4*>(turn + l32 % TOK * 128 + ((k ^ (l32 & 7)) * 16) + 8 * hi) =
                                out[n][m + k / 4][k % 4];
                    }
                    wave_lds_order();
                    const int c = m0 + (wm * MB + m) * 32 + 8 * p;
#pragma unroll
                    for (int i = 0; i < TOK / 8; ++i) {
                        const int tt = 8 * i + (lane >> 3), t = (wn * NL + n) * 32 + TOK * part + tt;
                        const u32x4 q = *reinterpret_cast<const u32x4*>(turn + tt * 128 + ((p ^ (tt & 7)) * 16));
                        const unsigned off = ((unsigned)t * ys + (unsigned)c) * 2u;
                        const bool live = t < nrows;
                        __builtin_amdgcn_raw_buffer_store_b128(q, ry, live && c + 8 <= cout ? (int)off : (int)kOOB, 0, 0);
                        if (cout & 4)  // the last four channels of a row
                            __builtin_amdgcn_raw_buffer_store_b64(u32x2{q[0], q[1]}, ry,
                                                                  live && c + 4 == cout ? (int)off : (int)kOOB, 0, 0);
                    }
                    wave_lds_order();
                }
    }
};

}  // namespace cvx
