// k_linear_few.hip -- projection of few tokens, the form for generated tokens:
// bound by the stream of the weights.
//
// A workgroup takes 16*RB output channels and all tokens (of more than 64, a block
// of 64); its W waves take
// 128-byte pieces of the weight rows in turn.  A wave loads its pieces straight
// into LDS of its own, four lines of 1 KB ahead and more (D stages, no barrier:
// a wave waits for its own loads only), with whole 128-byte lines a fetch: loaded
// into registers in the matrix instruction's order, 16 rows a load, the address
// unit takes 64 cycles for a load of 1 KB, a quarter of the cache's rate.  The
// tokens' values of the same channels go the same way.  The 16-byte pieces of a
// row are permuted by the row's index, so that operand reads spread over the
// banks.  Rows that are not there (tokens, channels) cost no traffic.  The waves'
// sums meet in LDS and are added in a fixed order.  The low-rank term is a few
// thousand multiply-adds a workgroup and is taken in fp32 on the vector units: v
// from LDS, the adapters' rows of these channels from memory.
//
// Measured, the rate that of the weights: one token, 4096 -> 4096 channels bf16 7.5
// us (4.5 TB/s), with an adapter of rank 16 8.7; 16 tokens of e4m3, 8192 -> 8192
// 15.0 (4.5), with 16 adapters of rank 16 21.3; 48 tokens bf16, 4096 -> 8192 16.6
// (4.0), with 32 adapters of rank 32 34.  A copy of such weights runs at 5.4 TB/s;
// what is missing is a workgroup's first fetch and its end, as each compute unit
// has one or two workgroups in all.  With a residual or adapters what the end needs
// is loaded ahead of the first products (below), and only the stages fetched before
// stand against that time: the 17 us between 34 and 16.6 are a launch for v, 5.4,
// and 12 that the start and the end take longer.
#include "lin_common.h"

#include "cvx_internal.h"

namespace cvx {

namespace {

// The value of another lane of the same row of 16 (a DPP control).
template <int CTRL>
__device__ __forceinline__ float lane_move(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

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

// Waits until at most N of this wave's vector-memory operations are under way;
// no memory access moves across it.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Waits until this wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// NT blocks of 16 tokens, of which XR rows (a multiple of eight) are loaded.  ONE:
// a single token with an adapter of up to 16 ranks; the adapter's A goes along as
// 16 more rows, in every workgroup, which for one token is less than a launch.
template <typename T, bool X8, bool ONE, int W, int RB, int NT, int XR, int D>
__global__ void __launch_bounds__(64 * W) k_linear_few(LinArgs a)
{
    typedef typename V16<T>::v8 v8;
    constexpr unsigned XB = X8 ? 1 : 2;
    constexpr int PER = 2 * RB + XR / 8 + (ONE ? 2 : 0);  // fetches of eight rows a stage
    constexpr int WB = 2048 * RB, AB = WB + 128 * XR, SB = 1024 * PER;  // a wave's stage: weights, x, A; bytes
    static_assert(D == 3 || D == 4, "stages under way");
    // an array a stage, so that waits are for the stage read, not for every fetch
    __shared__ __attribute__((aligned(1024))) unsigned char st0[W * SB], st1[W * SB], st2[W * SB],
        st3[D == 4 ? W * SB : 16];
    // the tokens' low-rank values, [tokens][rank]: beside the stages, or where they do not fit, in one
    constexpr int ROOM = (158 * 1024 - D * W * SB) / 4, MOST = XR * kLoraMaxRank;
    constexpr int BESIDE = ROOM < MOST ? ROOM : MOST;
    static_assert(BESIDE > 0 && 4 * MOST <= W * SB && 4 * 256 * RB * NT <= W * SB, "they fit a stage");
    __shared__ __attribute__((aligned(16))) float vbeside[BESIDE];
    __shared__ int id_lds[16 * NT];
    // a block of tokens: its rows of every operand
    const long slice = (long)a.tokens * a.rank;  // of v's partial sums
    const int t0 = blockIdx.y * 16 * NT;
    a.tokens = a.tokens - t0 < 16 * NT ? a.tokens - t0 : 16 * NT;
    a.x = static_cast<const char*>(a.x) + t0 * a.xs * XB;
    a.y = static_cast<T*>(a.y) + t0 * a.ys;
    if (X8) a.x_scale += t0;
    if (a.res) a.res = static_cast<const T*>(a.res) + t0 * a.rs;
    if (a.rank) {
        a.lora_id += t0;
        a.part += (long)t0 * a.rank;
    }
    const bool beside = a.tokens * a.rank <= BESIDE;
    float* vlds = ONE || beside ? vbeside : reinterpret_cast<float*>(st1);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c0 = blockIdx.x * 16 * RB;
    const int q = lane >> 4, l16 = lane & 15;
    const unsigned cb = (unsigned)a.cin * XB;  // bytes of a weight row
    const unsigned pitch = (unsigned)a.xs * XB;
    const int rows = a.cout - c0 < 16 * RB ? a.cout - c0 : 16 * RB;
    const rsrc_t rw = make_rsrc(static_cast<const char*>(a.w) + (long)c0 * cb, (unsigned)rows * cb);
    const rsrc_t rx = make_rsrc(a.x, (unsigned)(a.tokens - 1) * pitch + cb);
    // The 16-byte pieces of row r lie permuted, piece p at p ^ (r/2 % 8): the sixteen
    // lanes of an operand read that go together then fall in all of the banks.
    const unsigned piece[2] = {(unsigned)((lane & 7) ^ (lane >> 4)) * 16, (unsigned)((lane & 7) ^ (4 + (lane >> 4))) * 16};
    const unsigned wo = (unsigned)(lane >> 3) * cb, xo = (unsigned)(lane >> 3) * pitch;

    // ONE: the token's adapter, whose rows end with its ranks (with none, at once)
    const int one = ONE ? adapter_of(a, 0) : -1;
    const rsrc_t ra = make_rsrc(static_cast<const T*>(a.lora_a) + (long)(one < 0 ? 0 : one) * a.rank * a.cin,
                                one < 0 ? 0u : (unsigned)a.rank * cb);

    // A wave's stages are wave, wave + W, ...; every workgroup begins at another one
    // of them, as rows a power of two apart keep a piece's lines in few channels
    // of the cache (48 tokens, 4096 channels: 22.5 us begun together).
    const int nst = (int)((cb + 127) / 128);
    const int steps = (nst + W - 1) / W;
    const int turn = (int)((blockIdx.x >> 3) % (unsigned)steps);  // (consecutive workgroups are on eight XCDs)
    // rows past an operand are past its descriptor's range, pieces past a row are sent there
    auto issue = [&](int i, unsigned char* st) {
        const int j = i + turn < steps ? i + turn : i + turn - steps;
        const unsigned kb = (unsigned)(wave + W * j) * 128;
        const bool live[2] = {i < steps && kb + piece[0] < cb, i < steps && kb + piece[1] < cb};
        unsigned char* p = st + wave * SB;
#pragma unroll
        for (int r = 0; r < 2 * RB; ++r)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(p + 1024 * r), 16,
                                                     live[r & 1] ? wo + 8 * r * cb + kb + piece[r & 1] : kOOB, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < XR / 8; ++r)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(p + WB + 1024 * r), 16,
                                                     live[r & 1] ? xo + 8 * r * pitch + kb + piece[r & 1] : kOOB, 0, 0, 0);
        if constexpr (ONE)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(p + AB + 1024 * r), 16,
                                                         live[r & 1] ? wo + 8 * r * cb + kb + piece[r & 1] : kOOB, 0, 0,
                                                         0);
    };
    f32x4 acc[RB][NT];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 low = {0.0f, 0.0f, 0.0f, 0.0f};
    // One stage: its operands to registers, its buffer to the stage D on, the products.
    auto stage = [&](int i, unsigned char* st) {
        wait_vm<(D - 1) * PER>();
        const unsigned char* p = st + wave * SB;
        u32x4 wv[2][RB], xv[2][NT], av[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const unsigned slot = (unsigned)((4 * s + q) ^ (l16 >> 1)) * 16;
#pragma unroll
            for (int r = 0; r < RB; ++r) wv[s][r] = *reinterpret_cast<const u32x4*>(p + 2048 * r + l16 * 128 + slot);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = XR == 8 ? lane & 7 : 16 * n + l16;  // eight rows: columns 8 to 15 are of no token
                xv[s][n] = *reinterpret_cast<const u32x4*>(p + WB + row * 128 + ((4 * s + q) ^ (row >> 1 & 7)) * 16);
            }
            if constexpr (ONE) av[s] = *reinterpret_cast<const u32x4*>(p + AB + l16 * 128 + slot);
        }
        wait_lds();
        issue(i + D, st);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[r][n] = mma_piece<T, X8>(wv[s][r], xv[s][n], acc[r][n]);
        if constexpr (ONE)
#pragma unroll
            for (int s = 0; s < 2; ++s) low = mma16<T>(av[s], xv[s][0], low);
    };
    auto low_rank = [&]() {  // slices added in order, times the adapter's factor; four ranks a step
        const int total = a.tokens * a.rank;
        for (int i = 4 * tid; i < total; i += 256 * W) {
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int s = 0; s < a.slices; s += 4) {
                f32x4 p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = s + k < a.slices ? *reinterpret_cast<const f32x4*>(a.part + (s + k) * slice + i)
                                            : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += p[k][e];
            }
            const int d = id_lds[i / a.rank];
            const float al = d >= 0 && a.lora_alpha ? a.lora_alpha[d] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= al;
            *reinterpret_cast<f32x4*>(vlds + i) = v;
        }
    };
    // Loads return in their order: what the loads of the end need goes first, those loads
    // behind the first stages' fetches.  Stages past the last are zeros.
    const int id = a.rank && tid < 16 * NT ? adapter_of(a, tid) : -1;
    issue(0, st0);
    issue(1, st1);
    issue(2, st2);
    if constexpr (D == 4) issue(3, st3);
    // What the end needs is loaded here, behind the first stages' fetches and ahead of
    // the first products.  Loads return in their order; each of the residual's, a 16-bit
    // load behind a condition of its own, is waited for before the next, and v is joined
    // from the newest.  So with these a workgroup's products begin once all of it is
    // there.  A thread finishes one channel (c) of every TSTEP-th token.
    constexpr int CH = 16 * RB, TSTEP = 64 * W / CH, ITEMS = (16 * NT + TSTEP - 1) / TSTEP;
    const int ch = tid % CH, tfirst = tid / CH, c = c0 + ch;
    const float sc = a.scale && c < a.cout ? a.scale[c] : 1.0f, bi = a.bias && c < a.cout ? a.bias[c] : 0.0f;
    float sx[ITEMS];
    T res[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int t = tfirst + TSTEP * k;
        const bool ok = t < a.tokens && c < a.cout;
        sx[k] = X8 && ok ? a.x_scale[t] : 1.0f;
        res[k] = a.res && ok ? static_cast<const T*>(a.res)[(long)t * a.rs + c] : (T)0.0f;
    }
    if (a.rank) {
        if (tid < 16 * NT) id_lds[tid] = id;
        wait_lds();
        stage_barrier();  // (which waits for no fetch)
    }
    // The low-rank term.  Lanes take the adapters' rows as they lie in memory, eight
    // ranks each, the first EARLY of a lane's pieces now; the `lanes` of a channel
    // (a power of two) add theirs.
    constexpr int NTH = 64 * W, EARLY = W == 4 ? 8 * RB * (NT / 2) : 4;
    float* us = reinterpret_cast<float*>(st2);  // [token][channel]
    int shift = 0;
    while ((8 << shift) < a.rank) ++shift;
    const int lanes = 1 << shift, r8 = 8 * (tid & (lanes - 1));
    const int all = a.rank ? (a.tokens * CH) << shift : 0;
    auto load_b = [&](int e) {
        v8 b = v8{};
        const int o = c0 + (e >> shift) % CH;
        if (e < all && r8 < a.rank && o < a.cout) {
            const int d = id_lds[(e >> shift) / CH];
            if (d >= 0)
                b = *reinterpret_cast<const v8*>(static_cast<const T*>(a.lora_b) + ((long)d * a.cout + o) * a.rank + r8);
        }
        return b;
    };
    auto add_b = [&](v8 b, int e) {
        if (e - (tid & (lanes - 1)) >= all) return;  // all lanes of a channel together
        const int t = (e >> shift) / CH;
        float u = 0.0f;
        if (r8 < a.rank && id_lds[t] >= 0) {
            const float* v = vlds + t * a.rank + r8;
#pragma unroll
            for (int i = 0; i < 8; ++i) u = fmaf((float)b[i], v[i], u);
        }
        if (lanes > 1) u += lane_move<0xb1>(u);   // the neighbour's
        if (lanes > 2) u += lane_move<0x4e>(u);   // the other pair's, of four
        if (lanes > 4) u += lane_move<0x141>(u);  // the other four's, of eight
        if (lanes > 8) u += lane_move<0x140>(u);  // the other eight's, of sixteen
        if (r8 == 0) us[e >> shift] = u;
    };
    v8 early[EARLY];
#pragma unroll
    for (int k = 0; k < EARLY; ++k) early[k] = load_b(tid + NTH * k);
    if (!ONE && a.rank && beside) low_rank();
    for (int i = 0; i < steps; i += D) {
        stage(i, st0);
        stage(i + 1, st1);
        stage(i + 2, st2);
        if constexpr (D == 4) stage(i + 3, st3);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no fetch is under way when the stages are used again
    __syncthreads();
    if (!ONE && a.rank && !beside) low_rank();
    f32x4* red = reinterpret_cast<f32x4*>(st0);  // [wave][RB][NT][lane]
    static_assert(RB * NT * 1024 <= SB, "the sums fit a wave's stage");
    const float* redf = reinterpret_cast<const float*>(st0);
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) red[((wave * RB + r) * NT + n) * 64 + lane] = acc[r][n];
    if constexpr (ONE) {
        // rank r of the token: row r, column 0
        float* lows = reinterpret_cast<float*>(st1);
        if (l16 == 0) *reinterpret_cast<f32x4*>(lows + 16 * wave + 4 * q) = low;
        __syncthreads();
        if (tid < 16) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) v += lows[16 * w + tid];
            vlds[tid] = v * (one >= 0 && a.lora_alpha ? a.lora_alpha[one] : 1.0f);
        }
    }
    __syncthreads();
    if (a.rank) {
#pragma unroll
        for (int k = 0; k < EARLY; ++k) add_b(early[k], tid + NTH * k);
        for (int e0 = tid + NTH * EARLY; e0 < all; e0 += 8 * NTH) {
            v8 late[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) late[k] = load_b(e0 + NTH * k);
#pragma unroll
            for (int k = 0; k < 8; ++k) add_b(late[k], e0 + NTH * k);
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int t = tfirst + TSTEP * k;
        if (t >= a.tokens || c >= a.cout) continue;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            z += redf[(((w * RB + (ch >> 4)) * NT + (t >> 4)) * 64 + ((ch & 15) >> 2) * 16 + (t & 15)) * 4 + (ch & 3)];
        z = fmaf(X8 ? z * sx[k] : z, sc, bi);
        if (a.rank) z += us[t * CH + ch];
        static_cast<T*>(a.y)[(long)t * a.ys + c] = (T)finish(z, (float)res[k], a.act, a.res_mode);
    }
}

template <typename T, bool X8, int W, int RB, int NT, int XR, int D, bool ONE = false>
void launch_few_k(const LinArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.cout + 16 * RB - 1) / (16 * RB)), (unsigned)((a.tokens + 16 * NT - 1) / (16 * NT)));
    hipLaunchKernelGGL((k_linear_few<T, X8, ONE, W, RB, NT, XR, D>), grid, dim3(64 * W), 0, s, a);
}

template <typename T, bool X8>
hipError_t launch_few_t(const LinArgs& a, const LinPlan& p, hipStream_t s)
{
    if constexpr (!X8) {
        if (p.one) {
            launch_few_k<T, X8, 8, 1, 1, 8, 3, true>(a, s);
            return hipGetLastError();
        }
    }
    if (a.tokens <= 8)
        launch_few_k<T, X8, 8, 1, 1, 8, 4>(a, s);
    else if (p.nt == 1)
        launch_few_k<T, X8, 8, 1, 1, 16, 4>(a, s);
    else if (p.nt == 2)
        launch_few_k<T, X8, 4, 1, 2, 32, 4>(a, s);
    else if (p.rb == 1)
        launch_few_k<T, X8, 4, 1, 4, 64, 3>(a, s);
    else
        launch_few_k<T, X8, 4, 2, 4, 64, 3>(a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_few(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s)
{
    if (dtype == CVX_DT_F16) return x8 ? launch_few_t<half_t, true>(a, p, s) : launch_few_t<half_t, false>(a, p, s);
    return x8 ? launch_few_t<bf16_t, true>(a, p, s) : launch_few_t<bf16_t, false>(a, p, s);
}

}  // namespace cvx
