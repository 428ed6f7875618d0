// k_grouped_few.hip -- projection of rows grouped by expert where the groups' weights
// make few tiles: a token or a few in a few experts.
//
// A workgroup takes 16 output channels and up to 16 rows of one group; as in
// k_linear_few.hip its eight waves take 128-byte pieces of the weight rows in turn, by
// way of LDS, each with four stages under way, so a row of 8 KB is eight stages long
// where a tile of k_linear_grouped.hip goes through 64 one after another.  The workgroups of a
// launch are as many as the groups may need; each finds its rows by a scan of the
// groups' ends and ends at once where there are none.  e4m3 values are widened to 16
// bits, integers summed as such.
//
// Measured with the call, 6 us at least: one row, 4096 -> 4096 channels bf16 9.3 us
// (tiles 17.9), of integers 8.1 (12.0); 8192 -> 8192 bf16 27.8, 4.8 TB/s of weights
// (49.3); eight rows in as many groups, 2048 -> 512 bf16 7.7 (11.8).
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

// Rows a workgroup takes: group, first row, how many (0: none).
struct Block {
    int g, n0, nrows;
};

// Block `want` of the groups' blocks of 16 rows.  Ends that decrease are taken as the
// largest before them.
__device__ __forceinline__ Block find_block(const GroupArgs& a, int lane, int want)
{
    auto row = [&](int v) { return v < 0 ? 0 : v > a.rows ? a.rows : v; };
    int end0 = row(a.offset[0]), blocks0 = 0;
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
        const int blocks = (end - begin + 15) / 16;
        int sum = blocks;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const int in = want - blocks0 - (sum - blocks);  // of the group's blocks
        const unsigned long long hit = __ballot(in >= 0 && in < blocks);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int n0 = __builtin_amdgcn_readlane(begin + 16 * in, l), left = __builtin_amdgcn_readlane(end, l) - n0;
            return {g0 + l, n0, left < 16 ? left : 16};
        }
        end0 = __builtin_amdgcn_readlane(end, 63);
        blocks0 += __builtin_amdgcn_readlane(sum, 63);
    }
    return {0, 0, 0};
}

// Rows XR at most (8 or 16) of which are fetched.
template <typename T, int X, int XR>
__global__ void __launch_bounds__(512) k_grouped_few(GroupArgs a)
{
    typedef typename std::conditional<X == kXI8, i32x4, f32x4>::type sum_t;
    typedef typename std::conditional<X == kXI8, int, float>::type sum1_t;
    constexpr bool Q = X != kX16;  // 8-bit operands, tokens' scales
    constexpr unsigned XB = Q ? 1 : 2;
    constexpr int W = 8, D = 4;
    constexpr int PER = 2 + XR / 8;  // fetches of eight rows a stage
    constexpr int SB = 1024 * PER;   // a wave's stage
    // an array a stage, so that waits are for the stage read, not for every fetch
    __shared__ __attribute__((aligned(1024))) unsigned char st0[W * SB], st1[W * SB], st2[W * SB], st3[W * SB];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, l16 = lane & 15;
    const Block b = find_block(a, lane, (int)blockIdx.y);
    if (b.nrows == 0) return;
    const int c0 = blockIdx.x * 16;
    const unsigned cb = (unsigned)a.cin * XB, pitch = (unsigned)a.xs * XB;
    const int channels = a.cout - c0 < 16 ? a.cout - c0 : 16;
    const rsrc_t rw = make_rsrc(static_cast<const char*>(a.w) + ((long)b.g * a.cout + c0) * cb, (unsigned)channels * cb);
    const rsrc_t rx = make_rsrc(static_cast<const char*>(a.x) + (a.row_id ? 0l : (long)b.n0 * pitch),
                                (unsigned)((a.row_id ? a.tokens : b.nrows) - 1) * pitch + cb);
    // the row of x that a row of the block is (not below a.tokens where there is none)
    auto source = [&](int r) {
        if (r >= b.nrows) return 0x7fffffff;
        return a.row_id ? a.row_id[b.n0 + r] : b.n0 + r;
    };
    // The 16-byte pieces of row r lie permuted, piece p at p ^ (r/2 % 8), as in k_linear_few.hip.
    const unsigned piece[2] = {(unsigned)((lane & 7) ^ (lane >> 4)) * 16, (unsigned)((lane & 7) ^ (4 + (lane >> 4))) * 16};
    const unsigned wo = (unsigned)(lane >> 3) * cb;
    unsigned xo[XR / 8];
#pragma unroll
    for (int r = 0; r < XR / 8; ++r) {
        const int j = source(8 * r + (lane >> 3));
        xo[r] = (unsigned)j >= (unsigned)a.tokens ? kOOB : (unsigned)(j - (a.row_id ? 0 : b.n0)) * pitch;
    }
    // every workgroup begins at another one of a wave's stages
    const int nst = (int)((cb + 127) / 128);
    const int steps = (nst + W - 1) / W;
    const int turn = (int)((blockIdx.x >> 3) % (unsigned)steps);
    auto issue = [&](int i, unsigned char* st) {
        const int j = i + turn < steps ? i + turn : i + turn - steps;
        const unsigned kb = (unsigned)(wave + W * j) * 128;
        const bool live[2] = {i < steps && kb + piece[0] < cb, i < steps && kb + piece[1] < cb};
        unsigned char* p = st + wave * SB;
#pragma unroll
        for (int r = 0; r < 2; ++r) fetch16(rw, live[r] ? wo + 8 * r * cb + kb + piece[r] : kOOB, p + 1024 * r);
#pragma unroll
        for (int r = 0; r < XR / 8; ++r)
            fetch16(rx, live[r & 1] && xo[r] != kOOB ? xo[r] + kb + piece[r & 1] : kOOB, p + 2048 + 1024 * r);
    };
    sum_t acc = {0, 0, 0, 0};
    auto stage = [&](int i, unsigned char* st) {
        wait_vm<(D - 1) * PER>();
        const unsigned char* p = st + wave * SB;
        u32x4 wv[2], xv[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            wv[s] = *reinterpret_cast<const u32x4*>(p + l16 * 128 + ((4 * s + q) ^ (l16 >> 1)) * 16);
            const int row = XR == 8 ? lane & 7 : l16;  // eight rows: columns 8 to 15 are of none
            xv[s] = *reinterpret_cast<const u32x4*>(p + 2048 + row * 128 + ((4 * s + q) ^ (row >> 1 & 7)) * 16);
        }
        wait_lds();
        issue(i + D, st);
#pragma unroll
        for (int s = 0; s < 2; ++s) acc = mma_piece<T, X>(wv[s], xv[s], acc);
    };
    issue(0, st0);
    issue(1, st1);
    issue(2, st2);
    issue(3, st3);
    // what the end needs is loaded under the products: a thread finishes one value
    const int ch = tid & 15, r = tid >> 4, c = c0 + ch;
    const bool mine = r < b.nrows && c < a.cout;
    const long from = (long)b.g * a.cout + c;
    const float sc = a.scale && mine ? a.scale[from] : 1.0f, bi = a.bias && mine ? a.bias[from] : 0.0f;
    const float rw1 = a.weight && mine ? a.weight[b.n0 + r] : 1.0f;
    float sx = 1.0f;
    if constexpr (Q) {
        const int j = mine ? source(r) : 0x7fffffff;
        sx = (unsigned)j < (unsigned)a.tokens ? a.x_scale[j] : 0.0f;
    }
    for (int i = 0; i < steps; i += D) {
        stage(i, st0);
        stage(i + 1, st1);
        stage(i + 2, st2);
        stage(i + 3, st3);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no fetch is under way when the stages are used again
    __syncthreads();
    sum_t* red = reinterpret_cast<sum_t*>(st0);  // [wave][lane]
    static_assert(1024 <= SB, "the sums fit a wave's stage");
    red[wave * 64 + lane] = acc;
    __syncthreads();
    if (!mine) return;
    const sum1_t* red1 = reinterpret_cast<const sum1_t*>(st0);
    sum1_t sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red1[(w * 64 + (ch >> 2) * 16 + r) * 4 + (ch & 3)];
    float z = (float)sum;  // of integers: rounded once from 2^24 up
    z = fmaf(Q ? z * sx : z, sc, bi);
    static_cast<T*>(a.y)[(long)(b.n0 + r) * a.ys + c] = (T)(finish(z, 0.0f, a.act, CVX_RES_NONE) * rw1);
}

template <typename T, int X>
hipError_t launch_few_t(const GroupArgs& a, const GroupPlan& p, hipStream_t s)
{
    const dim3 grid((unsigned)((a.cout + 15) / 16), (unsigned)p.grid);
    if (a.rows <= 8)
        hipLaunchKernelGGL((k_grouped_few<T, X, 8>), grid, dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((k_grouped_few<T, X, 16>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_few(const GroupArgs& a, const GroupPlan& p, int dtype, int held, hipStream_t s)
{
    return by_types(dtype, held, [&](auto t, auto x) { return launch_few_t<typename decltype(t)::type, x.value>(a, p, s); });
}

}  // namespace cvx
