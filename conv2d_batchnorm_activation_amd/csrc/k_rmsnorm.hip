// k_rmsnorm.hip -- residual addition, root-mean-square norm and, for 8-bit
// output, the row's scale, in one pass over the data.
//
//     h = x + r,  q = 1/sqrt(mean(h^2) + eps),  y = h*gamma*q
//     8 bits: u = h*gamma, t = max|u|, code = nearest(u*f), scale = t*q/M,
//     e4m3: M = 448, f = M/t; integers: M = 127, f = M*(1/t)
//
// t does not depend on q, so the sum of squares and the maximum are one
// reduction: a row costs one exchange between its threads.  TPR threads hold a
// row as NV 16-byte vectors each (one load instruction per vector and operand,
// all of them in flight before the first use), so every byte moves once; rows
// too long to be held (NV = 0) are read a second time for the output, by the
// thread that read them first, which is what lets `sum` be x or the residual.
//
// Vector loads and stores are declared with the element's alignment only: the
// hardware takes any, so odd widths and slices run the same code, and the last
// c % VEC channels go one at a time.
//
// The arithmetic is in 64 bits: the kernel is bound by memory, a 64-bit multiply
// issues at the rate of a 32-bit one here, rows whose squares leave fp32's range
// stay right (h itself is an fp32 sum, but for the one form below), and a code is
// the nearest value to u*f itself, not to an fp32 neighbour of it.
//
// Measured: 16384 rows of 4096 bf16 channels with residual and sum to e4m3 or integers
// 86 us, 5.4 TB/s, the rate of a copy of that size; 96 rows of 8192 fp16 channels 4.2 us
// and one row of 4096 2.7 us, latency; 2048 rows of 20480 fp32 channels 135 us, 5.0
// TB/s, 512 rows 39 us, 4.3 TB/s; 1024 rows of 16384 bf16 channels 32 us, 4.2 TB/s.
#include <type_traits>

#include "cvx_internal.h"
#include "rows.h"

namespace cvx {

namespace {

template <typename T, int TPR, int NV, bool RES, int OUT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, 1) k_rmsnorm(RmsArgs a)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int HOLD = NV > 0 ? NV : 1;
    constexpr bool OUT8 = OUT != kX16;
    // The sum of two fp32 values can take more than fp32: for codes, which are rounded
    // from h itself, both are held, and h is in 64 bits; else, and of two 16-bit
    // values, their fp32 sum is h, once for the norm and for `sum`.
    constexpr bool TWO = RES && OUT8 && sizeof(T) == 4;
    constexpr int HOLD2 = TWO ? HOLD : 1;
    typedef typename Vec<T, VEC>::type V;
    typedef typename Vec<float, 4>::type G4;
    const int lane = threadIdx.x % TPR;
    const long row = TPR < 256 ? (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR : (long)blockIdx.x;
    if (row >= a.rows) return;  // whole waves: a row has at least one
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    const T* r = RES ? static_cast<const T*>(a.res) + row * a.rs : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.ss : nullptr;
    const int c = a.c;
    const int nvec = (c + VEC - 1) / VEC;

    // vector v of h (fp32: of x and of the residual); channels past c are zero
    auto load_h = [&](int v, float (&h)[VEC], float (&h2)[VEC]) {
        const int i0 = v * VEC;
        if (i0 + VEC <= c) {
            const V xv = *reinterpret_cast<const V*>(x + i0);
            if constexpr (RES) {
                const V rv = *reinterpret_cast<const V*>(r + i0);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    h[e] = TWO ? (float)xv[e] : (float)xv[e] + (float)rv[e];
                    if (TWO) h2[e] = (float)rv[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[e] = (float)xv[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] = 0.0f;
                if (TWO) h2[e] = 0.0f;
                if (i0 + e < c) {
                    h[e] = RES && !TWO ? (float)x[i0 + e] + (float)r[i0 + e] : (float)x[i0 + e];
                    if constexpr (TWO) h2[e] = (float)r[i0 + e];
                }
            }
        }
    };
    auto value = [&](float h, float h2) { return TWO ? (double)h + (double)h2 : (double)h; };
    auto load_gamma = [&](int v, float (&g)[VEC]) {
        const int i0 = v * VEC;
        if (i0 + VEC <= c) {
#pragma unroll
            for (int q = 0; q < VEC; q += 4) {
                const G4 gv = *reinterpret_cast<const G4*>(a.gamma + i0 + q);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[q + e] = gv[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = i0 + e < c ? a.gamma[i0 + e] : 0.0f;
        }
    };
    auto store_t = [&](T* dst, int v, const float (&o)[VEC]) {
        const int i0 = v * VEC;
        if (i0 + VEC <= c) {
            V ov;
#pragma unroll
            for (int e = 0; e < VEC; ++e) ov[e] = (T)o[e];
            *reinterpret_cast<V*>(dst + i0) = ov;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (i0 + e < c) dst[i0 + e] = (T)o[e];
        }
    };

    // gamma is held too where that is a few registers: it is then there when the row's sum is
    constexpr bool KEEP = NV > 0 && NV <= 2;
    float h[HOLD][VEC], h2[HOLD2][VEC], gam[KEEP ? NV : 1][VEC];
    double ss = 0.0, top = 0.0;
    auto add = [&](const float (&hv)[VEC], const float (&hw)[VEC], int v, int j) {
        float g[VEC];
        if constexpr (OUT8 && !KEEP) load_gamma(v, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const double d = value(hv[e], hw[e]);
            ss += d * d;
            if constexpr (OUT8) top = fmax(top, fabs(d * (double)(KEEP ? gam[KEEP ? j : 0][e] : g[e])));
        }
    };
    // calls f(vector's index, its slot) for every vector of this thread; with `one`
    // the scheduler keeps them apart, so that one vector's values are live at a time
    auto each = [&](auto f, bool one = false) {
        if constexpr (NV > 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (lane + j * TPR < nvec) f(lane + j * TPR, j);
                if (one && NV > 2) __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            for (int v = lane; v < nvec; v += TPR) {
                load_h(v, h[0], h2[0]);
                f(v, 0);
            }
        }
    };
    if constexpr (NV > 0) each([&](int v, int j) { load_h(v, h[j], h2[TWO ? j : 0]); });
    if constexpr (KEEP) each([&](int v, int j) { load_gamma(v, gam[j]); });
    each([&](int v, int j) { add(h[j], h2[TWO ? j : 0], v, j); }, true);
    row_reduce<TPR, OUT8>(ss, top);
    const double q = 1.0 / sqrt(ss / (double)c + (double)a.eps);

    // The held values are fp32 again from here: kept from above in 64 bits they would
    // take twice the registers, and a workgroup of 1024 threads the whole of a unit.
    if constexpr (NV > 2) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) asm volatile("" : "+v"(h[j][e]));
    }

    double f = q;
    if constexpr (OUT8) {
        f = !(top > 0.0) ? 0.0 : OUT == kXI8 ? kTop<OUT> * (1.0 / top) : kTop<OUT> / top;
        // an infinity's row (q = 0) has a NaN scale, also where gamma hides it from `top`
        if (lane == 0) a.y_scale[row] = q > 0.0 ? (float)(top * q / kTop<OUT>) : __builtin_nanf("");
    }
    each([&](int v, int j) {
        const int i0 = v * VEC;
        float g[VEC], o[VEC];
        if constexpr (KEEP)
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = gam[j][e];
        else
            load_gamma(v, g);
        if constexpr (OUT8) {
            unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.ys;
            unsigned u[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) u[e] = code_part<OUT>(value(h[j][e], h2[TWO ? j : 0][e]) * (double)g[e] * f);
            unsigned w[VEC / 4];
#pragma unroll
            for (int p = 0; p < VEC / 4; ++p) w[p] = pack_codes<OUT>(u[4 * p], u[4 * p + 1], u[4 * p + 2], u[4 * p + 3]);
            store_codes<VEC>(y, i0, c, w);
        } else {
            T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = (float)(value(h[j][e], h2[TWO ? j : 0][e]) * (double)g[e] * f);
            store_t(y, v, o);
        }
        if (sum) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = (float)value(h[j][e], h2[TWO ? j : 0][e]);
            store_t(sum, v, o);
        }
    }, true);
}

template <typename T, int TPR, int NV>
void launch_one(const RmsArgs& a, hipStream_t s)
{
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)(((long)a.rows + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
    auto go = [&](auto res) {
        constexpr bool RES = decltype(res)::value;
        if (a.held == kX16)
            hipLaunchKernelGGL((k_rmsnorm<T, TPR, NV, RES, kX16>), grid, block, 0, s, a);
        else if (a.held == kXE4m3)
            hipLaunchKernelGGL((k_rmsnorm<T, TPR, NV, RES, kXE4m3>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_rmsnorm<T, TPR, NV, RES, kXI8>), grid, block, 0, s, a);
    };
    if (a.res)
        go(std::true_type());
    else
        go(std::false_type());
}

// The same to 8-bit integers alone.
template <typename T, int TPR, int NV>
void launch_i8(const RmsArgs& a, hipStream_t s)
{
    static_assert(TPR >= 256, "a workgroup a row");
    const dim3 grid((unsigned)a.rows), block(TPR);
    if (a.res)
        hipLaunchKernelGGL((k_rmsnorm<T, TPR, NV, true, kXI8>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_rmsnorm<T, TPR, NV, false, kXI8>), grid, block, 0, s, a);
}

template <typename T>
hipError_t launch_t(const RmsArgs& a, hipStream_t s)
{
    // A row of some hundred vectors is 256 threads' where the rows fill the device, and
    // 1024 threads' (fewer loads one after another) where they do not.  bf16 with a
    // residual: 4096 channels, 1 row 2.3 us by 1024 threads, 2.5 by 256; 64 rows 3.3 and
    // 3.6; 512 rows 5.7 and 5.3; 2048 rows 15.3 and 13.0.  8192 channels: 256 rows 4.9
    // and 5.7, 512 rows 8.2 and 8.5, 1024 rows 14.2 and 12.5.  Rows of more than 1024
    // vectors are 1024 threads' however many they are, for the sake of the many: by 512
    // threads 2048 rows of 20480 fp32 channels take 143 us instead of 135, though 300
    // take 20.7 instead of 23.9 and 517 44.5 instead of 46.5.
    constexpr int VEC = 16 / (int)sizeof(T);
    const long nvec = ((long)a.c + VEC - 1) / VEC;
    const bool few = a.rows <= (nvec <= 512 ? 256 : 512);
    if (a.held == kXI8 && !few && nvec > 1024 && nvec <= (VEC == 8 ? 2560 : 2048)) {
        // To integers by fewer threads, as k_gate.hip does; the other types' sums keep the
        // order that they have.  us without and with a residual, as here and by 1024 threads:
        // 6250 rows of 10240 bf16 channels 53 and 100, 84 and 106; 4464 of 14336 54 and 96, 70
        // and 96; 3125 of 20480 57 and 99, 69 and 104; fp32, 6250 of 5120 36 and 82, 66 and 95.
        if (nvec <= 1280)
            launch_i8<T, 256, 5>(a, s);
        else if (nvec <= 2048)
            launch_i8<T, 512, 4>(a, s);
        else if constexpr (VEC == 8)
            launch_i8<T, 512, 5>(a, s);
    } else if (nvec <= 64)
        launch_one<T, 64, 1>(a, s);
    else if (nvec <= 256)
        launch_one<T, 256, 1>(a, s);
    else if (nvec <= 512 && !few)
        launch_one<T, 256, 2>(a, s);
    else if (nvec <= 1024 && !few)
        launch_one<T, 256, 4>(a, s);
    else if (nvec <= 1024)
        launch_one<T, 1024, 1>(a, s);
    else if (nvec <= 2048)
        launch_one<T, 1024, 2>(a, s);
    else if (nvec <= 4096)
        launch_one<T, 1024, 4>(a, s);
    else if (nvec <= 6144)
        launch_one<T, 1024, 6>(a, s);
    else
        launch_one<T, 1024, 0>(a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const RmsArgs& all, int dtype, hipStream_t s)
{
    // at most 2^20 rows a launch: a grid holds fewer than 2^32 threads
    constexpr int kRows = 1 << 20;
    const long es = dtype == CVX_DT_F32 ? 4 : 2, eo = all.held != kX16 ? 1 : es;
    for (long r0 = 0; r0 < all.rows; r0 += kRows) {
        RmsArgs a = all;
        a.rows = all.rows - r0 < kRows ? (int)(all.rows - r0) : kRows;
        a.x = static_cast<const char*>(all.x) + r0 * all.xs * es;
        if (all.res) a.res = static_cast<const char*>(all.res) + r0 * all.rs * es;
        if (all.sum) a.sum = static_cast<char*>(all.sum) + r0 * all.ss * es;
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
