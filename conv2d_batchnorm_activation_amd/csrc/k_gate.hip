// k_gate.hip -- the gated activation between two projections, and rows of any
// origin brought to 8 bits:
//
//     u = act(g) * up   (act(g) alone without `up`),   y = u rounded
//     8 bits: t = max|u|, code = nearest(u*(M*(1/t))), scale = t/M, M = 448 or 127
//     (M*(1/t) infinite: zeros)
//
// Bound by memory: every value is read once and written once.  With 8-bit output a row's
// largest magnitude is one reduction between the TPR threads that hold it, as NV 16-byte
// vectors an operand each; rows too long to be held (NV = 0) are read three times, for the
// largest fp32 value, for t and for the codes (3000 rows of 40000 bf16 channels 233 us,
// 6.7 TB/s of what is loaded and stored; 32768 channels, held, 114).  t and the codes are those of
// 64-bit values, by the formula's own steps: where u/t is a ratio of small integers,
// u*(M*(1/t)) can be a border between two codes but for the last bit of either, and then
// only the same roundings give the same code.  Few values need 64 bits: those that may be
// the largest, and those that fp32 leaves at a border.  With 64 bits for all (some 35
// instructions a value) 8192 rows of 14336 bf16 channels took 236 us; they take 106 to
// 110, 5.3 to 5.5 TB/s.  Still the vector units are busy most of that time (31
// instructions a value).  Output of the inputs' type is u in fp32, and there is no row: a
// thread takes a vector.
#include <type_traits>

#include "cvx_internal.h"
#include "rows.h"

namespace cvx {

namespace {

// The activations: SiLU, or ReLU (a NaN stays one) or none by `relu`.
template <bool SILU>
__device__ __forceinline__ double act64(double g, bool relu)
{
    if constexpr (SILU) return g / (1.0 + exp(-g));
    return relu && g < 0.0 ? 0.0 : g;
}

// In fp32.  FAST: by the hardware's exponential and reciprocal (an ulp each), with what
// rounding the exponential's argument, x = -g*log2(e), left as a factor: off by less than
// 2*2^-23 + 7*2^-24 of the value where g is at least kDeep (below, 1/exp leaves fp32; ln 2
// in fp32 is off by 2^-28.4 of itself, |x| times 1.9e-9 in `left`, up to 4*2^-24 there).
constexpr float kDeep = -80.0f;
template <bool SILU, bool FAST>
__device__ __forceinline__ float act32(float g, bool relu)
{
    if constexpr (SILU && FAST) {
        const float x = g * -1.442695041f;
        const float left = fmaf(x, -0.6931471806f, -g);
        const float e = __builtin_amdgcn_exp2f(x);
        return g * __builtin_amdgcn_rcpf(1.0f + fmaf(e, left, e));
    }
    if constexpr (SILU) {  // by the exponential that does not overflow: the value down to where fp32 ends
        const float e = expf(-fabsf(g));
        return (g < 0.0f ? g * e : g) / (1.0f + e);
    }
    return relu && g < 0.0f ? 0.0f : g;
}

// VEC values of an operand from channel i0, zero past c.
template <typename T, int VEC>
__device__ __forceinline__ typename Vec<T, VEC>::type load_vec(const T* p, int i0, int c)
{
    typedef typename Vec<T, VEC>::type V;
    if (i0 + VEC <= c) return *reinterpret_cast<const V*>(p + i0);
    V v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = i0 + e < c ? p[i0 + e] : (T)0.0f;
    return v;
}

// More than an fp32 u*f is off by, of itself: u 2*2^-23 + 8*2^-24 with its second factor,
// f half an ulp; 1.8 times the sum.
constexpr float kOff = 1.5f * 0x1p-20f;

// How far u*f is off the integer next to it.
__device__ __forceinline__ float off_ones(float u, float f, float& ones)
{
    ones = fmaf(u, f, 0x1.8p23f);  // a sum that leaves none below one
    return fabsf(fmaf(u, f, 0x1.8p23f - ones));
}

// The codes of VEC values u*f, from fp32; true if one of them may be another, none
// being larger than `most`.
template <int OUT, int VEC>
__device__ __forceinline__ bool codes32(const float (&u)[VEC], float most, float f, unsigned (&w)[VEC / 4])
{
    if constexpr (OUT == kXE4m3) {  // the same codes from a little less and a little more
        const float less = f * (1.0f - kOff), more = f * (1.0f + kOff);
        bool any = false;
#pragma unroll
        for (int q = 0; q < VEC; q += 4) {
            w[q / 4] = pack_e4m3(u[q] * less, u[q + 1] * less, u[q + 2] * less, u[q + 3] * less);
            any |= w[q / 4] != pack_e4m3(u[q] * more, u[q + 1] * more, u[q + 2] * more, u[q + 3] * more);
        }
        return any;
    }
    unsigned ones[VEC];
    float off = 0.0f;  // the most that a value is off its integer
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float s;
        off = fmaxf(off, off_ones(u[e], f, s));
        ones[e] = __builtin_bit_cast(unsigned, s);
    }
#pragma unroll
    for (int q = 0; q < VEC; q += 4)
        w[q / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(ones[q + 3], ones[q + 2], 0x0c0c0400u),
                                         __builtin_amdgcn_perm(ones[q + 1], ones[q], 0x0c0c0400u), 0x05040100u);
    return off > 0.5f - (most * f + 1.0f) * kOff;
}

// Waves a SIMD that the registers are to leave room for: eight of up to two vectors (64 registers),
// but of rows read again, with all there is to do, which would keep 21 of its registers in
// memory (3000 rows of 40000 bf16 channels to integers 313 us, 234 so; to e4m3 219 and 237).
constexpr int waves_of(int nv, bool all) { return nv > 2 || (nv == 0 && all) ? 4 : 8; }

// 8-bit output: TPR threads a row.
template <typename T, int TPR, int NV, bool SILU, bool UP, int OUT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, waves_of(NV, SILU && UP && OUT == kXI8)) k_gate(GateArgs a)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int HOLD = NV > 0 ? NV : 1;
    typedef typename Vec<T, VEC>::type V;
    const int lane = threadIdx.x % TPR;
    const long row = TPR < 256 ? (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR : (long)blockIdx.x;
    if (row >= a.rows) return;  // all threads of a row
    const T* g = static_cast<const T*>(a.gate) + row * a.gs;
    const T* p = UP ? static_cast<const T*>(a.up) + row * a.us : nullptr;
    unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.ys;
    const int c = a.c, nvec = (c + VEC - 1) / VEC;
    const bool relu = a.act == CVX_ACT_RELU;

    V gv[HOLD], uv[UP ? HOLD : 1];
    auto load = [&](int v, int j) {
        gv[j] = load_vec<T, VEC>(g, v * VEC, c);
        if constexpr (UP) uv[UP ? j : 0] = load_vec<T, VEC>(p, v * VEC, c);
    };
    auto exact = [&](int j, int e) {
        const double x = act64<SILU>((double)(float)gv[j][e], relu);
        return UP ? x * (double)(float)uv[UP ? j : 0][e] : x;
    };
    // calls f(vector's index, its slot) for every vector of this thread, loaded before
    auto each = [&](auto f) {
        if constexpr (NV > 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (lane + j * TPR < nvec) f(lane + j * TPR, j);
        } else {
            for (int v = lane; v < nvec; v += TPR) {
                load(v, 0);
                f(v, 0);
            }
        }
    };
    // a vector's u in fp32 and the largest of them: infinite where fp32 does not tell
    float u[HOLD][VEC], most[HOLD];
    auto near = [&](int j) {
        float m = 0.0f, low = 0.0f, odd = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float gf = (float)gv[j][e];
            u[j][e] = act32<SILU, true>(gf, relu);
            if constexpr (UP) u[j][e] *= (float)uv[UP ? j : 0][e];
            low = fminf(low, gf);
            m = fmaxf(m, fabsf(u[j][e]));
            if (e % 2) odd = fmaf(u[j][e], u[j][e - 1], odd);  // a NaN or an infinity from either on
        }
        const bool told = fabsf(odd) < __builtin_inff() && (!SILU || low >= kDeep);
        most[j] = told ? m : __builtin_inff();
    };
    float top = 0.0f;
    if constexpr (NV > 0) each([&](int v, int j) { load(v, j); });
    each([&](int, int j) {
        near(j);
        top = fmaxf(top, most[j] < __builtin_inff() ? most[j] : 0.0f);
    });
    top = row_top<TPR, 0>(top);

    // t, in 64 bits: the largest of the vectors that may hold it, those that fp32 does
    // not tell among them
    const bool wide = !(top > 0x1p-60f && top < 0x1p100f);  // all may
    const float least = top * (1.0f - kOff);
    double t = 0.0, bad = 0.0;
    each([&](int, int j) {
        if constexpr (NV == 0) near(j);
        const bool all = wide || most[j] == __builtin_inff();
        if (!all && most[j] < least) return;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (all || fabsf(u[j][e]) >= least) {
                const double x = exact(j, e);
                t = fmax(t, fabs(x));
                bad = fma(x, 0.0, bad);
            }
    });
    if (bad != 0.0) t = __builtin_inf();
    t = row_top<TPR, 1>(t);
    const bool lost = t > 1.7e308;
    // t = 0, or so small that M*(1/t) is infinite, which times a zero would be a NaN: zeros, and so is the scale
    const double m = kTop<OUT> * (1.0 / t), f = lost || m == __builtin_inf() ? 0.0 : m;
    if (lane == 0) a.y_scale[row] = lost ? __builtin_nanf("") : (float)(t * (1.0 / kTop<OUT>));

    // codes from fp32 where it tells them, else from 64 bits
    each([&](int v, int j) {
        unsigned w[VEC / 4];
        if constexpr (NV == 0) near(j);
        bool any = codes32<OUT, VEC>(u[j], most[j], (float)f, w);
        const bool all = wide || most[j] == __builtin_inff();
        if (any || all) {
            unsigned x[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float s;
                const float off = off_ones(u[j][e], (float)f, s);
                x[e] = __builtin_bit_cast(unsigned, s);
                if (OUT != kXI8 || all || off > 0.5f - (fabsf(u[j][e]) * (float)f + 1.0f) * kOff)
                    x[e] = code_part<OUT>(exact(j, e) * f);
            }
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) w[q] = pack_codes<OUT>(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        }
        store_codes<VEC>(y, v * VEC, c, w);
    });
}

// Output of the inputs' type: a thread a vector.
template <typename T, bool SILU, bool UP>
__global__ void __launch_bounds__(256) k_gate_wide(GateArgs a)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    typedef typename Vec<T, VEC>::type V;
    const unsigned nvec = (unsigned)(a.c + VEC - 1) / VEC;
    const long at = (long)blockIdx.x * 256 + threadIdx.x;
    const long row = at / nvec;
    const int i0 = (int)(at - row * nvec) * VEC, c = a.c;
    if (row >= a.rows) return;
    const V gv = load_vec<T, VEC>(static_cast<const T*>(a.gate) + row * a.gs, i0, c);
    V uv;
    if constexpr (UP) uv = load_vec<T, VEC>(static_cast<const T*>(a.up) + row * a.us, i0, c);
    float g[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        g[e] = act32<SILU, false>((float)gv[e], a.act == CVX_ACT_RELU);
        if constexpr (UP) g[e] *= (float)uv[e];
    }
    T* y = static_cast<T*>(a.y) + row * a.ys;
    if (i0 + VEC <= c) {
        V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = (T)g[e];
        *reinterpret_cast<V*>(y + i0) = o;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (i0 + e < c) y[i0 + e] = (T)g[e];
    }
}

// f(whether the activation is SiLU, whether there is an `up`), as values that carry them
template <typename F>
void by_act(const GateArgs& a, F f)
{
    auto of = [&](auto silu) {
        if (a.up)
            f(silu, std::true_type());
        else
            f(silu, std::false_type());
    };
    if (a.act == CVX_ACT_SILU)
        of(std::true_type());
    else
        of(std::false_type());
}

template <typename T, int TPR, int NV>
void launch_rows(const GateArgs& a, hipStream_t s)
{
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)(((long)a.rows + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
    by_act(a, [&](auto silu, auto up) {
        if (a.held == kXE4m3)
            hipLaunchKernelGGL((k_gate<T, TPR, NV, silu.value, up.value, kXE4m3>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_gate<T, TPR, NV, silu.value, up.value, kXI8>), grid, block, 0, s, a);
    });
}

template <typename T>
hipError_t launch_t(const GateArgs& a, hipStream_t s)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const long nvec = ((long)a.c + VEC - 1) / VEC;
    if (a.held == kX16) {
        const dim3 grid((unsigned)((a.rows * nvec + 255) / 256));
        by_act(a, [&](auto silu, auto up) {
            hipLaunchKernelGGL((k_gate_wide<T, silu.value, up.value>), grid, dim3(256), 0, s, a);
        });
    } else if (nvec <= 8) {
        // Up to 1280 vectors the fewest threads that hold a row in registers, of 8, 16, whole
        // waves or workgroups (up to a wave needs no barrier), with little of them idle: more
        // rows are then under way beside one that waits.  us, bf16 to integers, of some 10^8
        // values a case (390000 rows of 32 vectors, 3662 of 4096): 8 vectors 8x1 167, 16x1 256;
        // 16 8x2 121, 16x1 130; 32 16x2 103, 16x4 115, 64x1 186; 96 64x2 111, 64x4 126; 256 64x4
        // 109, 256x2 114; 640 256x3 108, 512x2 116, 1024x1 172; 1024 256x5 108, 512x2 107, 1024x1
        // 131; 1280 256x5 110, 512x3 119, 1024x2 122.
        // Longer rows by what measured less, 1.17*10^8 values of bf16 a case, half of fp32, to
        // integers (to e4m3 the same order): bf16 1281 vectors 1024x2 125, 512x4 129; 1792 106 and
        // 111 (64 rows 6.0 and 6.6, 1024 16.7 and 18.3); 2048 105 and 110; 2304 512x5 108, 1024x3
        // 146 (256 rows 10.1 and 9.2); 2600 1024x3 142, 1024x4 145.  fp32 1300 512x4 95, 1024x2
        // 101; 1700 94.0 and 94.9; 1792 95.6 and 94.6; 2049 1024x3 99, 512x5 101; 3000 97, 1024x4
        // 118.
        launch_rows<T, 8, 1>(a, s);
    } else if (nvec <= 16) {
        launch_rows<T, 8, 2>(a, s);
    } else if (nvec <= 32) {
        launch_rows<T, 16, 2>(a, s);
    } else if (nvec <= 64) {
        launch_rows<T, 16, 4>(a, s);
    } else if (nvec <= 128) {
        launch_rows<T, 64, 2>(a, s);
    } else if (nvec <= 256) {
        launch_rows<T, 64, 4>(a, s);
    } else if (nvec <= 512) {
        launch_rows<T, 256, 2>(a, s);
    } else if (nvec <= 768) {
        launch_rows<T, 256, 3>(a, s);
    } else if (nvec <= 1280) {
        launch_rows<T, 256, 5>(a, s);
    } else if (VEC == 4 && nvec < 1792) {
        launch_rows<T, VEC == 4 ? 512 : 1024, VEC == 4 ? 4 : 2>(a, s);
    } else if (nvec <= 2048) {
        launch_rows<T, 1024, 2>(a, s);
    } else if (VEC == 8 && nvec <= 2560) {
        launch_rows<T, VEC == 8 ? 512 : 1024, VEC == 8 ? 5 : 3>(a, s);
    } else if (nvec <= 3 * 1024) {
        launch_rows<T, 1024, 3>(a, s);
    } else if (nvec <= 4096) {
        launch_rows<T, 1024, 4>(a, s);
    } else if (VEC == 4 && nvec <= 6144) {
        launch_rows<T, 1024, VEC == 4 ? 6 : 0>(a, s);
    } else {
        launch_rows<T, 1024, 0>(a, s);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& all, int dtype, hipStream_t s)
{
    // as many rows a launch as keep a grid below 2^32 threads
    const long es = dtype == CVX_DT_F32 ? 4 : 2, eo = all.held != kX16 ? 1 : es;
    const long nvec = (all.c + 16 / es - 1) / (16 / es);
    const long most = all.held != kX16 ? 1l << 20 : (1l << 31) / nvec;
    for (long r0 = 0; r0 < all.rows; r0 += most) {
        GateArgs a = all;
        a.rows = (int)(all.rows - r0 < most ? all.rows - r0 : most);
        a.gate = static_cast<const char*>(all.gate) + r0 * all.gs * es;
        if (all.up) a.up = static_cast<const char*>(all.up) + r0 * all.us * es;
        a.y = static_cast<char*>(all.y) + r0 * all.ys * eo;
        if (all.held != kX16) a.y_scale = all.y_scale + r0;
        const hipError_t e = dtype == CVX_DT_F32   ? launch_t<float>(a, s)
                             : dtype == CVX_DT_F16 ? launch_t<half_t>(a, s)
                                                   : launch_t<bf16_t>(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace cvx
