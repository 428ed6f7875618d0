// k_linear_grouped.hip -- projection of rows grouped by expert: every row by its
// group's weights, groups of any size.
//
// The products are those of k_linear_tile.hip (weights the A operand, rows the B
// operand, lin_tile.h has the loop). How many rows a group has stands in device memory,
// so the tiles are counted there: a workgroup stays for several tiles, begins with a
// scan of the groups' ends, and finds a tile's group by its number. The first stages of
// its next tile are fetched as a tile's products end; in tiles of 256x256 of 16-bit
// operands they arrive under the arithmetic of its end, in the others the compiler waits
// for them before the end's operands are read from LDS. A group's last tile, where it
// has half of the rows or fewer, takes half of the products; tiles that share weights
// are neighbours (the three together: 64 ragged groups, 32768 rows, 2048 -> 2816 bf16
// 434 -> 412 us). Rows are read where they lie (row_id), so that tokens need no copy in
// the groups' order.
//
// Few rows a group are bound by the weights' stream: 512 rows in 64 groups, 2048 -> 2816
// e4m3 74 us, 5.0 TB/s of weights, a copy's rate; eight rows in eight groups, of
// integers 11.4, 4.1 TB/s. Many rows are bound by the first touch of every group's
// weights: 64 groups of 512 rows, 2048 -> 2816 bf16 387 to 389 us (980 TFLOP/s), 318 to
// 340 as one group of as many rows (1110 to 1190), whose weights stay in the caches;
// e4m3 242 to 255, integers 233 to 239; 64 ragged groups of 512 on average 416 to 431,
// the tiles not filled being some 8%. Of these the profiler has 577 cycles a read past a
// compute unit's cache and 1149 MB past the XCDs', 403 and 781 of the one group, the
// matrix pipes busy 0.38 and 0.41 of 2.4 GHz's cycles. Eight groups of 1024 rows, 4096
// -> 14336 e4m3 470 to 483 (1990 to 2040).
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

// A tile: its group, its first channel, its first row and how many rows; of none, 0.
struct Where {
    int g, m0, n0, nrows;
};

// 64 values of four bytes into LDS, lane l's from byte `off` of the operand.
__device__ __forceinline__ void fetch64(rsrc_t r, unsigned off, void* to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, (int)off, 0, 0, 0);
}

// WM x WN waves, each MB x NB blocks of 32 x 32; D stage buffers; WIDE: e4m3 in 16 bits (lin_tile.h).
template <typename T, int X, int WM, int WN, int MB, int NB, int D, int RB, bool WIDE>
__global__ void __launch_bounds__(64 * WM * WN, WM * WN == 8 || RB == 64 ? 2 : 1) k_linear_grouped(GroupArgs a)
{
    typedef Tile<T, X, WM, WN, MB, NB, D, RB, WIDE> tile;
    typedef typename tile::v4 v4;
    constexpr bool Q = X != kX16;  // 8-bit operands, tokens' scales
    constexpr unsigned XB = tile::XB;
    constexpr int W = tile::W, NT = tile::NT, BM = tile::BM, BN = tile::BN, SB = tile::SB;
    constexpr int TOK = 16;  // rows that are turned at a time
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[SB], buf1[SB], buf2[D == 4 ? SB : 16],
        buf3[D == 4 ? SB : 16];
    const Stages bufs = {{buf0, buf1, buf2, buf3}};
    __shared__ __attribute__((aligned(16))) unsigned char turn[W * 128 * TOK];
    __shared__ __attribute__((aligned(16))) float sc_lds[BM], bi_lds[BM];
    __shared__ float sx_lds[2][Q ? BN : 64], rw_lds[BN];  // (x's scales of this tile and the next)
    __shared__ Groups groups;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int hi = lane >> 5, l32 = lane & 31;
    const unsigned cb = (unsigned)a.cin * XB, pitch = (unsigned)a.xs * XB;

    if (wave == 0) count_tiles<BN>(a, lane, groups);
    // what is not given stays as it is set here
    for (int i = tid; i < BM; i += NT) {
        sc_lds[i] = 1.0f;
        bi_lds[i] = 0.0f;
    }
    for (int i = tid; i < BN; i += NT) rw_lds[i] = 1.0f;
    __syncthreads();
    // Workgroups go to the XCDs in turn: each XCD has a run of the tiles, which its
    // workgroups take in turn.
    const int n = a.tiles_m * __builtin_amdgcn_readfirstlane(groups.first[a.groups]);
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int per = n >> 3, rest = n & 7;
    const int lo = xcd * per + (xcd < rest ? xcd : rest), up = lo + per + (xcd < rest ? 1 : 0);
    auto find = [&](int at) {
        Where t = {0, 0, 0, 0};
        if (at >= up) return t;
        // Of a group, four tiles of rows go with a tile of channels before the next of these,
        // so that tiles which share weights are taken at the same time.  (The numbers are the
        // same in all lanes, which the compiler is told where it does not see it.)
        auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        t.g = same(group_of(a, lane, groups, a.tiles_m, at));
        const int first = same(groups.first[t.g]), start = same(groups.start[t.g]);
        const int tn = same(groups.first[t.g + 1]) - first, in = at - first * a.tiles_m;
        const int run = same(in / (4 * a.tiles_m)), ir = in - run * 4 * a.tiles_m;
        const int gn = tn - 4 * run < 4 ? tn - 4 * run : 4;
        const int tm = same(ir / gn);
        t.m0 = tm * BM;
        t.n0 = start + (4 * run + ir - tm * gn) * BN;
        const int left = same(groups.start[t.g + 1]) - t.n0;
        t.nrows = left < BN ? left : BN;
        return t;
    };
    // the row of x that row r of a tile is (not below a.tokens where there is none)
    auto source = [&](const Where& t, int r) {
        if (r >= t.nrows) return 0x7fffffff;
        return a.row_id ? a.row_id[t.n0 + r] : t.n0 + r;
    };
    // this lane's fetches of x, and where it fetches x's scales, the rows these are of
    constexpr int FN = tile::FN, FS = Q ? (BN / 64 + W - 1) / W : 1;
    struct Sources {
        int x[FN], sx[FS];
    };
    auto sources = [&](const Where& t) {
        Sources s;
#pragma unroll
        for (int i = 0; i < FN; ++i) s.x[i] = source(t, tile::fetch_row(wave, lane, i));
#pragma unroll
        for (int i = 0; i < FS; ++i) s.sx[i] = Q ? source(t, 64 * (wave + W * i) + lane) : 0;
        return s;
    };
    // a tile's operands, with the fetch of x's scales begun
    auto operands = [&](const Where& t, const Sources& s, float* sx) {
        TileRows op;
        op.w = static_cast<const char*>(a.w) + ((long)t.g * a.cout + t.m0) * cb;
        op.wend = (unsigned)(a.cout - t.m0 < BM ? a.cout - t.m0 : BM) * cb;
        op.x = static_cast<const char*>(a.x) + (a.row_id ? 0l : (long)t.n0 * pitch);
        op.xend = (unsigned)((a.row_id ? a.tokens : t.nrows) - 1) * pitch + cb;
#pragma unroll
        for (int i = 0; i < tile::FM; ++i)
            op.wo[i] = (unsigned)tile::fetch_row(wave, lane, i) * cb + tile::piece(wave, lane);
#pragma unroll
        for (int i = 0; i < FN; ++i)
            op.xo[i] = (unsigned)s.x[i] >= (unsigned)a.tokens
                           ? kOOB
                           : (unsigned)(s.x[i] - (a.row_id ? 0 : t.n0)) * pitch + tile::piece(wave, lane);
        if constexpr (Q)
#pragma unroll
            for (int i = 0; i < FS; ++i)
                if (64 * (wave + W * i) < BN)
                    fetch64(make_rsrc(a.x_scale, 4u * (unsigned)a.tokens),
                            (unsigned)s.sx[i] >= (unsigned)a.tokens ? kOOB : 4u * (unsigned)s.sx[i],
                            sx + 64 * (wave + W * i));
        return op;
    };

    int at = lo + (int)(blockIdx.x >> 3);
    if (at >= up) return;
    Where cur = find(at);
    float *sx0 = sx_lds[0], *sx1 = sx_lds[1];
    TileRows op = operands(cur, sources(cur), sx0);
    tile::begin(op, cb, wave, lane, bufs);
    for (;;) {
        // What the end needs comes into LDS under the products: no wave reads the tile
        // before any more.  (It is there when the first stages' barriers are passed.)
        const int mrows = a.cout - cur.m0 < BM ? a.cout - cur.m0 : BM;
        for (int i = wave; i < BM / 64; i += W) {
            const unsigned off = 4u * (unsigned)(64 * i + lane), end = 4u * (unsigned)mrows;
            const long from = (long)cur.g * a.cout + cur.m0;
            if (a.scale) fetch64(make_rsrc(a.scale + from, end), off, sc_lds + 64 * i);
            if (a.bias) fetch64(make_rsrc(a.bias + from, end), off, bi_lds + 64 * i);
        }
        if (a.weight)
            for (int i = wave; i < BN / 64; i += W)
                fetch64(make_rsrc(a.weight + cur.n0, 4u * (unsigned)cur.nrows), 4u * (unsigned)(64 * i + lane),
                        rw_lds + 64 * i);
        at += step;
        const Where nxt = find(at);
        const Sources far = sources(nxt);  // (arrives under the products)

        // NL blocks of 32 rows a wave: half of them where they hold the tile's rows
        auto work = [&](auto blocks) {
            constexpr int NL = decltype(blocks)::value;
            typename tile::sum_t total[MB][NL];
            tile::template sums<true, NL>(op, cb, wave, lane, bufs, total);
            if (nxt.nrows) {
                op = operands(nxt, far, sx1);
                tile::begin(op, cb, wave, lane, bufs);
            }

            // as in k_linear_tile.hip: lane (hi, l32) holds channels 8j + 4hi + 0..3 of one row
            v4 out[NL][MB][4];
#pragma unroll
            for (int n = 0; n < NL; ++n) {
                const int t = (wn * NL + n) * 32 + l32;
                const float sx = Q ? sx0[t] : 1.0f, rw = rw_lds[t];
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
                make_rsrc(static_cast<T*>(a.y) + (long)cur.n0 * a.ys, (unsigned)((cur.nrows - 1) * a.ys + a.cout) * 2u);
            tile::template store<NL, TOK>(out, turn, wave, lane, ry, cur.nrows, (unsigned)a.ys, cur.m0, a.cout);
        };
        if (NB == 1 || cur.nrows > BN / 2)
            work(std::integral_constant<int, NB>());
        else if constexpr (NB > 1)
            work(std::integral_constant<int, NB / 2>());
        if (nxt.nrows == 0) break;
        lds_barrier();  // no wave reads this tile's operands of the end any more
        cur = nxt;
        float* const used = sx0;
        sx0 = sx1;
        sx1 = used;
    }
}

template <typename T, int X>
hipError_t launch_grouped_t(GroupArgs a, const GroupPlan& p, hipStream_t s)
{
    a.tiles_m = (a.cout + 64 * p.mb - 1) / (64 * p.mb);
    const dim3 grid((unsigned)p.grid);
    auto small = [&](auto wide) {
        constexpr bool WIDE = decltype(wide)::value;
        if (p.rb == 128)
            hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 2, 2, 1, 4, 128, WIDE>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 2, 2, 1, 4, 64, WIDE>), grid, dim3(256), 0, s, a);
    };
    if (p.mb == 4)
        hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 4, 4, 2, 2, 128, false>), grid, dim3(512), 0, s, a);
    else if (p.nb == 2)
        hipLaunchKernelGGL((k_linear_grouped<T, X, 2, 2, 2, 2, 4, 128, false>), grid, dim3(256), 0, s, a);
    else if (X == kXE4m3 && p.wide)
        small(std::integral_constant<bool, X == kXE4m3>());
    else
        small(std::false_type());
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_grouped(const GroupArgs& a, const GroupPlan& p, int dtype, int held, hipStream_t s)
{
    if (p.few) return launch_grouped_few(a, p, dtype, held, s);
    return by_types(dtype, held,
                    [&](auto t, auto x) { return launch_grouped_t<typename decltype(t)::type, x.value>(a, p, s); });
}

GroupPlan grouped_plan(const cvx_grouped_desc& d)
{
    GroupPlan p;
    // The tile that ends first by what a stage (128 bytes of every row) and the rest of a
    // tile measured, in 10 ns, with the tiles one a compute unit (the last kind two, of
    // half stages: one's end beside the other's products).  How the rows are spread is not
    // known here: a group is taken to have a tile at least and to leave half a one empty.
    // 351 cases, us as 256x256, 128x128, 128x64 and the last kind: 64 groups, 2048 ->
    // 2816 bf16, 8 rows each 175, 151, 144, 145; 64 184, 163, 170, 191; 128 203, 209, 234,
    // 252; 512 421, 533, 671, 773.  128 groups of e4m3, 512 -> 768, 8 rows each 25, 21, 19,
    // 14.  Five of integers, 1008 -> 1284, 128 rows each 20, 10, 8.7, 9.4.  Over all, the kind
    // taken needs 1.3% more time than the best, 54% at most (one group of 512 rows).
    const struct {
        int mb, nb, rb, at_once, stage, rest;
    } tiles[] = {{4, 4, 128, 256, 130, 900}, {2, 2, 128, 256, 45, 400}, {2, 1, 128, 256, 36, 500}, {2, 1, 64, 512, 80, 100}};
    const long stages = ((long)d.c_in * (d.x_dtype == d.dtype ? 2 : 1) + 127) / 128;
    const long some = d.rows < d.n_groups ? d.rows : d.n_groups;  // groups that may have rows
    // At most a workgroup a compute unit of the kernel for few rows, or two of long rows:
    // one row, 4096 -> 4096 channels bf16 9.3 us (17.9 by tiles), 8192 -> 1024 7.8 (28);
    // eight rows in as many groups, 2048 -> 512 7.7 (11.8); two of 4096 -> 4096 15.3 (18.2);
    // 16 of 1024 -> 512 11.0 (9.2), eight of 2048 -> 1408 14.8 (12.9).
    const long blocks = (d.rows + 15 * some) / 16;  // of up to 16 rows, at most
    const long few = (long)((d.c_out + 15) / 16) * blocks;
    // Up to 64 rows a group on average are bound by the weights' stream where tiles are many:
    // there e4m3 values are widened to 16 bits, whose sums are fp32.  64 groups, 2048 -> 2816,
    // 8 rows each 73.9 us (72.6 by the 8-bit instructions), 33 81.0 (80.1), 64 90 (93); 128
    // groups, 512 -> 768, 8 each 14.6 (13.8).  Where tiles are few, a stage's conversions stand
    // beside its products: five groups of 30 rows, 1008 -> 1284, 9.0 us (7.1), 16 of 4, 2048 ->
    // 1024, 12.2 (10.2).  Of long rows three and a half workgroups a compute unit of the kernel
    // for few rows are faster then: two groups of 32 rows, 8192 -> 2048, 14.4 us (29.9 by
    // widened tiles, 18.5 by the 8-bit instructions), three of 64, 8192 -> 1024, 19.6 (29.6,
    // 19.6), ten of 8, 4096 -> 1024, 15.9 (17.9, 12.3); four a unit: one of 64, 4096 -> 4096,
    // 20.3 (17.6, 12.5).  Tiles of 128 rows never are: 64 groups of 64 rows 98 us, of 64 rows 90.
    p.wide = d.x_dtype == CVX_DT_E4M3 && d.rows <= 64l * d.n_groups;
    p.few = few <= 256 || (few <= (p.wide ? 896 : 512) && stages >= 32);
    if (p.few) {
        p.mb = p.nb = p.rb = 0;
        p.grid = (int)blocks;
        return p;
    }
    long best = -1;
    for (const auto& t : tiles) {
        if (p.wide && t.nb > 1) continue;
        const long m = (d.c_out + 64 * t.mb - 1) / (64 * t.mb);
        const long tall = (d.rows + 64 * t.nb - 1) / (64 * t.nb) + some / 2, n = m * (tall < some ? some : tall);
        const long time = (n + t.at_once - 1) / t.at_once * (stages * t.stage + t.rest);
        if (best >= 0 && time >= best) continue;
        best = time;
        p.mb = t.mb;
        p.nb = t.nb;
        p.rb = t.rb;
        // as many workgroups as run at once, or as there may be tiles
        const long most = m * ((d.rows + (64 * t.nb - 1) * some) / (64 * t.nb));
        p.grid = (int)(most < t.at_once ? (most + 7) / 8 * 8 : t.at_once);
    }
    return p;
}

void grouped_describe(const cvx_grouped_desc& d, const GroupPlan& p, char* buf, int len)
{
    const char* t = d.dtype == CVX_DT_F16 ? "_Float16" : "__bf16";
    if (p.few)
        snprintf(buf, len, "grouped few 16x16 workgroups=%d kernel=cvx::k_grouped_few<%s, %d, %d>",
                 (d.c_out + 15) / 16 * p.grid, t, held_of(d.dtype, d.x_dtype), d.rows <= 8 ? 8 : 16);
    else
        snprintf(buf, len, "grouped tile %dx%d workgroups=%d kernel=cvx::k_linear_grouped<%s, %d, 2, %d, %d, %d, %d, %d>",
             64 * p.mb, 64 * p.nb, p.grid, t, held_of(d.dtype, d.x_dtype), p.mb == 4 ? 4 : 2, p.mb,
             p.mb == 4 ? 2 : p.nb, p.mb == 4 ? 2 : 4, p.rb);
}

}  // namespace cvx
