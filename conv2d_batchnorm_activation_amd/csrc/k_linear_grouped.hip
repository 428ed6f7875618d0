// k_linear_grouped.hip -- projection of rows grouped by expert: every row by its
// group's weights, groups of any size.
//
// The products are those of k_linear_tile.hip (weights the A operand, rows the B
// operand, lin_tile.h has the loop).  How many rows a group has stands in device
// memory, so the tiles are counted there: a workgroup stays for several tiles, begins
// with a scan of the groups' ends, and finds a tile's group by its number.  Rows are
// read where they lie (row_id), so that tokens need no copy in the groups' order.
#include <stdio.h>

#include "cvx_internal.h"
#include "lin_tile.h"

namespace cvx {

namespace {

// The groups' tiles of BN rows, counted from the first group's.
struct Groups {
    int first[kMaxGroups + 1];  // of a group
    int start[kMaxGroups + 1];  // a group's first row; the next one's is its end
};

// One wave: ends that decrease are taken as the largest before them, so groups are
// disjoint and within the rows whatever stands in `offset`.
template <int BN>
__device__ __forceinline__ void count_tiles(const GroupArgs& a, int lane, Groups& s)
{
    auto row = [&](int v) { return v < 0 ? 0 : v > a.rows ? a.rows : v; };
    int end0 = row(a.offset[0]), tiles0 = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        const int g = g0 + lane;
        int end = g < a.groups ? row(a.offset[g + 1]) : 0;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(end, d);
            if (lane >= d && o > end) end = o;
        }
        if (end0 > end) end = end0;
        int begin = __shfl_up(end, 1);
        if (lane == 0) begin = end0;
        const int tiles = (end - begin + BN - 1) / BN;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (g < a.groups) {
            s.first[g] = tiles0 + sum - tiles;
            s.start[g] = begin;
        }
        end0 = __builtin_amdgcn_readlane(end, 63);
        tiles0 += __builtin_amdgcn_readlane(sum, 63);
    }
    if (lane == 0) {
        s.first[a.groups] = tiles0;
        s.start[a.groups] = end0;
    }
}

// The group of a tile, `times` tiles for each counted: the last whose first is not past it.
__device__ __forceinline__ int group_of(const GroupArgs& a, int lane, const Groups& s, int times, int tile)
{
    int n = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64)
        n += __builtin_popcountll(__ballot(g0 + lane < a.groups && s.first[g0 + lane] * times <= tile));
    return n - 1;
}

// WM x WN waves, each MB x NB blocks of 32 x 32; D stage buffers.
template <typename T, int X, int WM, int WN, int MB, int NB, int D>
__global__ void __launch_bounds__(64 * WM * WN, D == 2 ? 2 : 1) k_linear_grouped(GroupArgs a)
{
    typedef Tile<T, X, WM, WN, MB, NB, D> tile;
    typedef typename tile::v4 v4;
    constexpr bool Q = X != kX16;  // 8-bit operands, tokens' scales
    constexpr unsigned XB = tile::XB;
    constexpr int NT = tile::NT, BM = tile::BM, BN = tile::BN, SB = tile::SB;
    // an array a stage, so that waits are for the stage read, not for every fetch
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[SB], buf1[SB], buf2[D == 4 ? SB : 16],
        buf3[D == 4 ? SB : 16];
    __shared__ __attribute__((aligned(16))) float sc_lds[BM], bi_lds[BM];
    __shared__ float sx_lds[Q ? BN : 1], rw_lds[BN];
    __shared__ Groups groups;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int hi = lane >> 5, l32 = lane & 31;
    const unsigned cb = (unsigned)a.cin * XB, pitch = (unsigned)a.xs * XB;

    if (wave == 0) count_tiles<BN>(a, lane, groups);
    __syncthreads();
    // Workgroups go to the XCDs in turn: each XCD has a run of the tiles, which its
    // workgroups take in turn.
    const int n = a.tiles_m * groups.first[a.groups];
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int per = n >> 3, rest = n & 7;
    const int lo = xcd * per + (xcd < rest ? xcd : rest), up = lo + per + (xcd < rest ? 1 : 0);
    for (int at = lo + (int)(blockIdx.x >> 3); at < up; at += step) {
        // of a group, eight tiles of channels go before the next tile of rows
        const int g = __builtin_amdgcn_readfirstlane(group_of(a, lane, groups, a.tiles_m, at));
        const int tn = groups.first[g + 1] - groups.first[g], in = at - groups.first[g] * a.tiles_m;
        const int wide = 8 * tn, run = in / wide, ir = in - run * wide;
        const int gm = a.tiles_m - 8 * run < 8 ? a.tiles_m - 8 * run : 8;
        const int tr = ir / gm;
        const int m0 = (8 * run + ir - tr * gm) * BM;
        const int n0 = __builtin_amdgcn_readfirstlane(groups.start[g] + tr * BN);
        const int left = __builtin_amdgcn_readfirstlane(groups.start[g + 1]) - n0;
        const int nrows = left < BN ? left : BN;
        const int mrows = a.cout - m0 < BM ? a.cout - m0 : BM;
        TileRows op;
        op.w = static_cast<const char*>(a.w) + ((long)g * a.cout + m0) * cb;
        op.wend = (unsigned)mrows * cb;
#pragma unroll
        for (int i = 0; i < tile::FM; ++i)
            op.wo[i] = (unsigned)tile::fetch_row(wave, lane, i) * cb + tile::piece(wave, lane);
        // the row of x that a row of the tile is, or -1
        auto source = [&](int r) {
            if (r >= nrows) return -1;
            const int j = a.row_id ? a.row_id[n0 + r] : n0 + r;
            return j < a.tokens ? j : -1;
        };
        op.x = static_cast<const char*>(a.x) + (a.row_id ? 0l : (long)n0 * pitch);
        op.xend = (unsigned)((a.row_id ? a.tokens : nrows) - 1) * pitch + cb;
#pragma unroll
        for (int i = 0; i < tile::FN; ++i) {
            const int r = tile::fetch_row(wave, lane, i), j = source(r);
            op.xo[i] = j < 0 ? kOOB : (unsigned)(a.row_id ? j : r) * pitch + tile::piece(wave, lane);
        }
        for (int i = tid; i < BM; i += NT) {
            const bool ok = m0 + i < a.cout;
            sc_lds[i] = !a.scale ? 1.0f : ok ? a.scale[(long)g * a.cout + m0 + i] : 0.0f;
            bi_lds[i] = a.bias && ok ? a.bias[(long)g * a.cout + m0 + i] : 0.0f;
        }
        for (int i = tid; i < BN; i += NT) {
            if constexpr (Q) {
                const int j = source(i);
                sx_lds[i] = j < 0 ? 0.0f : a.x_scale[j];
            }
            rw_lds[i] = a.weight && i < nrows ? a.weight[n0 + i] : 1.0f;
        }
        typename tile::sum_t total[MB][NB];
        tile::sums(op, cb, wave, lane, buf0, buf1, buf2, buf3, total);

        // as in k_linear_tile.hip: lane (hi, l32) holds channels 8j + 4hi + 0..3 of one row
        v4 out[NB][MB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int t = (wn * NB + n) * 32 + l32;
            const float sx = Q ? sx_lds[t] : 1.0f, rw = rw_lds[t];
            f32x16 acc[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = (wm * MB + m) * 32 + 8 * j + 4 * hi;
                    const f32x4 sc = *reinterpret_cast<const f32x4*>(sc_lds + c);
                    const f32x4 bi = *reinterpret_cast<const f32x4*>(bi_lds + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float z = (float)total[m][n][4 * j + i];  // of integers: rounded once from 2^24 up
                        acc[m][4 * j + i] = fmaf(Q ? z * sx : z, sc[i], bi[i]);
                    }
                }
            auto activate = [&](auto act) {
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[m][i] = apply_act_nan(acc[m][i], decltype(act)::value);
            };
            if (a.act == CVX_ACT_RELU) activate(std::integral_constant<int, CVX_ACT_RELU>());
            if (a.act == CVX_ACT_SILU) activate(std::integral_constant<int, CVX_ACT_SILU>());
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 16; ++i) out[n][m][i / 4][i % 4] = (T)(acc[m][i] * rw);
            __builtin_amdgcn_sched_barrier(0);
        }
        const rsrc_t ry =
            make_rsrc(static_cast<T*>(a.y) + (long)n0 * a.ys, (unsigned)((nrows - 1) * a.ys + a.cout) * 2u);
        tile::store(out, buf0, wave, lane, ry, nrows, (unsigned)a.ys, m0, a.cout);
        lds_barrier();  // LDS is free for the next tile
    }
}

template <typename T, int X>
hipError_t launch_grouped_t(GroupArgs a, const GroupPlan& p, hipStream_t s)
{
    a.tiles_m = (a.cout + 64 * p.mb - 1) / (64 * p.mb);
    const dim3 grid((unsigned)p.grid);
    if (p.mb == 4)
        hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 4, 4, 2, 2>), grid, dim3(512), 0, s, a);
    else if (p.nb == 2)
        hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 2, 2, 2, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 2, 2, 1, 4>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_grouped(const GroupArgs& a, const GroupPlan& p, int dtype, int held, hipStream_t s)
{
    return by_types(dtype, held,
                    [&](auto t, auto x) { return launch_grouped_t<typename decltype(t)::type, x.value>(a, p, s); });
}

GroupPlan grouped_plan(const cvx_grouped_desc& d)
{
    GroupPlan p;
    const struct {
        int mb, nb, stage, rest;
    } tiles[] = {{4, 4, 150, 1000}, {2, 2, 45, 500}, {2, 1, 28, 400}};
    const long stages = ((long)d.c_in * (d.x_dtype == d.dtype ? 2 : 1) + 127) / 128;
    const long some = d.rows < d.n_groups ? d.rows : d.n_groups;  // groups that may have rows
    long best = -1;
    for (const auto& t : tiles) {
        const long m = (d.c_out + 64 * t.mb - 1) / (64 * t.mb);
        const long n = m * ((d.rows + 64 * t.nb - 1) / (64 * t.nb) + some / 2);
        const long time = (n + 255) / 256 * (stages * t.stage + t.rest);
        if (best >= 0 && time >= best) continue;
        best = time;
        p.mb = t.mb;
        p.nb = t.nb;
        // a workgroup a compute unit, as many as there may be tiles
        const long most = m * (d.rows / (64 * t.nb) + some);
        p.grid = (int)(most < 256 ? (most + 7) / 8 * 8 : 256);
    }
    return p;
}

void grouped_describe(const cvx_grouped_desc& d, const GroupPlan& p, char* buf, int len)
{
    const char* t = d.dtype == CVX_DT_F16 ? "_Float16" : "__bf16";
    snprintf(buf, len, "grouped tile %dx%d workgroups=%d kernel=cvx::k_linear_grouped<%s, %d, 2, %d, %d, %d, %d>", 64 * p.mb,
             64 * p.nb, p.grid, t, held_of(d.dtype, d.x_dtype), p.mb == 4 ? 4 : 2, p.mb, p.mb == 4 ? 2 : p.nb,
             p.mb == 4 ? 2 : 4);
}

}  // namespace cvx
