// api_tokens.hip -- the C ABI of the operators on tokens: host-side validation
// and the choice of kernels.  Every check runs on the host before anything is
// enqueued.
#include <float.h>
#include <stdint.h>

#include "cvx_internal.h"
#include "tokens.h"

using namespace cvx;

namespace {

constexpr long kMaxSpan = 1L << 40;    // elements from an operand's first to its last
constexpr long kMaxPitch = 1L << 21;   // row stride of a projection's operands: 256 rows stay below 2^31 bytes
constexpr int kMaxChannels = 1 << 20;  // channels of a projection
constexpr int kMaxI8 = (1 << 17) - 16; // of 8-bit integers: their sums, of up to 2^14 each, stay below 2^31
constexpr int kMaxNormed = 1 << 30;    // channels of a row that is normed: their index stays an int
constexpr int kMaxTokens = 1 << 24;    // tokens of a projection
constexpr long kMaxOut = 1L << 37;     // its outputs: 275 GB, and tiles of fewer than 2^32 threads in all

inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool dtype16(int dt) { return dt == CVX_DT_F16 || dt == CVX_DT_BF16; }
inline bool dtype8(int dt) { return dt == CVX_DT_E4M3 || dt == CVX_DT_I8; }
inline unsigned dt_bytes(int dt) { return dt == CVX_DT_F32 ? 4 : dtype8(dt) ? 1 : 2; }

// A strided operand [rows][c] in bytes: [lo, hi).
struct Span {
    uintptr_t lo, hi;
};
inline Span rows_span(const void* p, long rows, long stride, long c, unsigned es)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (uintptr_t)(((rows - 1) * stride + c) * (long)es)};
}
inline Span bytes_span(const void* p, size_t n)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + n};
}
inline bool meets(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// A row stride as the descriptor gives it -> elements; false if it is invalid.
inline bool stride_of(long given, long c, long rows, long* out)
{
    if (given != 0 && given < c) return false;
    *out = given == 0 ? c : given;
    return *out <= kMaxSpan && rows <= kMaxSpan / *out;
}

cvx_status check_linear(const cvx_linear_desc* d, long* xs, long* rs, long* ys)
{
    if (d == nullptr) return CVX_ERR_NULL;
    if (!dtype16(d->dtype) || (d->x_dtype != d->dtype && !dtype8(d->x_dtype))) return CVX_ERR_ARG;
    if (d->act < CVX_ACT_NONE || d->act > CVX_ACT_SILU) return CVX_ERR_ARG;
    if (d->res_mode < CVX_RES_NONE || d->res_mode > CVX_RES_AFTER_ACT) return CVX_ERR_ARG;
    if (d->rank < 0 || d->n_adapters < 0 || (d->rank == 0) != (d->n_adapters == 0)) return CVX_ERR_ARG;
    if (d->tokens < 1 || d->c_in < 1 || d->c_out < 1 || d->tokens > kMaxTokens || d->c_in > kMaxChannels ||
        d->c_out > kMaxChannels || (long)d->tokens * d->c_out > kMaxOut)
        return CVX_ERR_SHAPE;
    if (!stride_of(d->x_stride, d->c_in, d->tokens, xs) || *xs > kMaxPitch) return CVX_ERR_SHAPE;
    if (!stride_of(d->y_stride, d->c_out, d->tokens, ys) || *ys > kMaxPitch) return CVX_ERR_SHAPE;
    *rs = d->c_out;
    if (d->res_mode != CVX_RES_NONE &&
        (!stride_of(d->res_stride, d->c_out, d->tokens, rs) || *rs > kMaxPitch))
        return CVX_ERR_SHAPE;
    if (d->x_dtype == CVX_DT_I8 && d->c_in > kMaxI8) return CVX_ERR_SHAPE;
    const int per = dtype8(d->x_dtype) ? 16 : 8;
    if (d->c_in % per != 0 || *xs % per != 0) return CVX_ERR_UNSUPPORTED;
    if (d->c_out % 4 != 0 || *ys % 4 != 0 || *rs % 4 != 0) return CVX_ERR_UNSUPPORTED;
    if (d->rank % 8 != 0 || d->rank > kLoraMaxRank) return CVX_ERR_UNSUPPORTED;
    return CVX_OK;
}

cvx_status check_grouped(const cvx_grouped_desc* d, long* xs, long* ys)
{
    if (d == nullptr) return CVX_ERR_NULL;
    if (!dtype16(d->dtype) || (d->x_dtype != d->dtype && !dtype8(d->x_dtype))) return CVX_ERR_ARG;
    if (d->act < CVX_ACT_NONE || d->act > CVX_ACT_SILU) return CVX_ERR_ARG;
    if (d->rows < 1 || d->tokens < 1 || d->c_in < 1 || d->c_out < 1 || d->rows > kMaxTokens || d->tokens > kMaxTokens ||
        d->c_in > kMaxChannels || d->c_out > kMaxChannels || (long)d->rows * d->c_out > kMaxOut)
        return CVX_ERR_SHAPE;
    if (d->n_groups < 1 || d->n_groups > kMaxGroups || (long)d->n_groups * d->c_out > kMaxSpan / d->c_in)
        return CVX_ERR_SHAPE;
    if (!stride_of(d->x_stride, d->c_in, d->tokens, xs) || *xs > kMaxPitch) return CVX_ERR_SHAPE;
    if (!stride_of(d->y_stride, d->c_out, d->rows, ys) || *ys > kMaxPitch) return CVX_ERR_SHAPE;
    if (d->x_dtype == CVX_DT_I8 && d->c_in > kMaxI8) return CVX_ERR_SHAPE;
    const int per = dtype8(d->x_dtype) ? 16 : 8;
    if (d->c_in % per != 0 || *xs % per != 0 || d->c_out % 4 != 0 || *ys % 4 != 0) return CVX_ERR_UNSUPPORTED;
    return CVX_OK;
}

}  // namespace

extern "C" {

cvx_status cvx_rmsnorm(const cvx_rmsnorm_desc* d, const void* x, const void* residual, const float* gamma, void* sum,
                       void* y, float* y_scale, void* stream)
{
    if (d == nullptr) return CVX_ERR_NULL;
    if (d->dtype != CVX_DT_F32 && !dtype16(d->dtype)) return CVX_ERR_ARG;
    if (d->out_dtype != d->dtype && !dtype8(d->out_dtype)) return CVX_ERR_ARG;
    if (!(d->eps > 0.0f) || d->eps > FLT_MAX) return CVX_ERR_ARG;
    if (d->rows < 1 || d->c < 1 || d->c > kMaxNormed) return CVX_ERR_SHAPE;
    const bool out8 = dtype8(d->out_dtype);
    RmsArgs a;
    a.rs = a.ss = d->c;
    if (!stride_of(d->x_stride, d->c, d->rows, &a.xs) || !stride_of(d->y_stride, d->c, d->rows, &a.ys) ||
        (residual && !stride_of(d->res_stride, d->c, d->rows, &a.rs)) ||
        (sum && !stride_of(d->sum_stride, d->c, d->rows, &a.ss)))
        return CVX_ERR_SHAPE;
    if (!x || !gamma || !y || (out8 && !y_scale)) return CVX_ERR_NULL;
    const unsigned es = dt_bytes(d->dtype), eo = dt_bytes(d->out_dtype);
    if (!aligned_to(x, es) || !aligned_to(residual, es) || !aligned_to(sum, es) || !aligned_to(y, eo) ||
        !aligned_to(gamma, 4) || (out8 && !aligned_to(y_scale, 4)))
        return CVX_ERR_ALIGN;
    const Span in[3] = {rows_span(x, d->rows, a.xs, d->c, es), bytes_span(gamma, 4ul * d->c),
                        residual ? rows_span(residual, d->rows, a.rs, d->c, es) : Span{0, 0}};
    const Span out[3] = {rows_span(y, d->rows, a.ys, d->c, eo), out8 ? bytes_span(y_scale, 4ul * d->rows) : Span{0, 0},
                         sum ? rows_span(sum, d->rows, a.ss, d->c, es) : Span{0, 0}};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            if (j < i && meets(out[i], out[j])) return CVX_ERR_ALIAS;
            const bool same = i == 2 && ((j == 0 && sum == x && a.ss == a.xs) ||
                                         (j == 2 && sum == residual && a.ss == a.rs));
            if (!same && meets(out[i], in[j])) return CVX_ERR_ALIAS;
        }
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.sum = sum;
    a.y = y;
    a.y_scale = y_scale;
    a.rows = d->rows;
    a.c = d->c;
    a.eps = d->eps;
    a.held = held_of(d->dtype, d->out_dtype);
    return launch_rmsnorm(a, d->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? CVX_OK : CVX_ERR_HIP;
}

cvx_status cvx_gate(const cvx_gate_desc* d, const void* gate, const void* up, void* y, float* y_scale, void* stream)
{
    if (d == nullptr) return CVX_ERR_NULL;
    if (d->dtype != CVX_DT_F32 && !dtype16(d->dtype)) return CVX_ERR_ARG;
    if (d->out_dtype != d->dtype && !dtype8(d->out_dtype)) return CVX_ERR_ARG;
    if (d->act < CVX_ACT_NONE || d->act > CVX_ACT_SILU) return CVX_ERR_ARG;
    if (d->rows < 1 || d->c < 1 || d->c > kMaxNormed) return CVX_ERR_SHAPE;
    const bool out8 = dtype8(d->out_dtype);
    GateArgs a;
    a.us = d->c;
    if (!stride_of(d->gate_stride, d->c, d->rows, &a.gs) || !stride_of(d->y_stride, d->c, d->rows, &a.ys) ||
        (up && !stride_of(d->up_stride, d->c, d->rows, &a.us)))
        return CVX_ERR_SHAPE;
    if (!gate || !y || (out8 && !y_scale)) return CVX_ERR_NULL;
    const unsigned es = dt_bytes(d->dtype), eo = dt_bytes(d->out_dtype);
    if (!aligned_to(gate, es) || !aligned_to(up, es) || !aligned_to(y, eo) || (out8 && !aligned_to(y_scale, 4)))
        return CVX_ERR_ALIGN;
    const Span in[2] = {rows_span(gate, d->rows, a.gs, d->c, es),
                        up ? rows_span(up, d->rows, a.us, d->c, es) : Span{0, 0}};
    const Span out[2] = {rows_span(y, d->rows, a.ys, d->c, eo), out8 ? bytes_span(y_scale, 4ul * d->rows) : Span{0, 0}};
    if (meets(out[0], out[1])) return CVX_ERR_ALIAS;
    for (const Span& o : out)
        for (const Span& i : in)
            if (meets(o, i)) return CVX_ERR_ALIAS;
    a.gate = gate;
    a.up = up;
    a.y = y;
    a.y_scale = y_scale;
    a.rows = d->rows;
    a.c = d->c;
    a.act = d->act;
    a.held = held_of(d->dtype, d->out_dtype);
    return launch_gate(a, d->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? CVX_OK : CVX_ERR_HIP;
}

size_t cvx_linear_workspace_bytes(const cvx_linear_desc* d)
{
    long xs, rs, ys;
    if (check_linear(d, &xs, &rs, &ys) != CVX_OK) return 0;
    return linear_plan(*d).ws_bytes;
}

cvx_status cvx_linear_plan(const cvx_linear_desc* d, char* buf, int buf_len)
{
    if (buf == nullptr || buf_len < 1) return CVX_ERR_NULL;
    long xs, rs, ys;
    const cvx_status st = check_linear(d, &xs, &rs, &ys);
    if (st != CVX_OK) return st;
    linear_describe(*d, linear_plan(*d), buf, buf_len);
    return CVX_OK;
}

cvx_status cvx_linear(const cvx_linear_desc* d, const void* x, const float* x_scale, const void* w,
                      const float* scale, const float* bias, const void* residual, const void* lora_a,
                      const void* lora_b, const float* lora_alpha, const int* lora_id, void* y, void* workspace,
                      size_t ws_bytes, void* stream)
{
    LinArgs a;
    const cvx_status st = check_linear(d, &a.xs, &a.rs, &a.ys);
    if (st != CVX_OK) return st;
    const bool x8 = dtype8(d->x_dtype), lora = d->rank > 0;
    if (!x || !w || !y || (x8 && !x_scale)) return CVX_ERR_NULL;
    if (d->res_mode != CVX_RES_NONE && !residual) return CVX_ERR_NULL;
    if (lora && (!lora_a || !lora_b || !lora_id)) return CVX_ERR_NULL;
    a.x = x;
    a.x_scale = x8 ? x_scale : nullptr;
    a.w = w;
    a.scale = scale;
    a.bias = bias;
    a.res = d->res_mode != CVX_RES_NONE ? residual : nullptr;
    a.lora_a = lora ? lora_a : nullptr;
    a.lora_b = lora ? lora_b : nullptr;
    a.lora_alpha = lora ? lora_alpha : nullptr;
    a.lora_id = lora ? lora_id : nullptr;
    a.y = y;
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(a.scale, 16) || !aligned_to(a.bias, 16) ||
        !aligned_to(a.lora_a, 16) || !aligned_to(a.lora_b, 16) || !aligned_to(a.lora_alpha, 4) ||
        !aligned_to(a.lora_id, 4) || !aligned_to(a.x_scale, 4) || !aligned_to(a.res, 8) || !aligned_to(y, 8))
        return CVX_ERR_ALIGN;
    const LinPlan p = linear_plan(*d);
    const long t = d->tokens;
    const unsigned ex = dt_bytes(d->x_dtype);
    const Span ysp = rows_span(y, t, a.ys, d->c_out, 2);
    const Span wsp = p.ws_bytes ? bytes_span(workspace, p.ws_bytes) : Span{0, 0};
    const struct {
        const void* p;
        Span s;
    } in[] = {{x, rows_span(x, t, a.xs, d->c_in, ex)},
              {a.x_scale, bytes_span(a.x_scale, 4ul * t)},
              {w, bytes_span(w, (size_t)d->c_out * d->c_in * ex)},
              {a.scale, bytes_span(a.scale, 4ul * d->c_out)},
              {a.bias, bytes_span(a.bias, 4ul * d->c_out)},
              {a.res, rows_span(a.res, t, a.rs, d->c_out, 2)},
              {a.lora_a, bytes_span(a.lora_a, (size_t)d->n_adapters * d->rank * d->c_in * 2)},
              {a.lora_b, bytes_span(a.lora_b, (size_t)d->n_adapters * d->rank * d->c_out * 2)},
              {a.lora_alpha, bytes_span(a.lora_alpha, 4ul * d->n_adapters)},
              {a.lora_id, bytes_span(a.lora_id, 4ul * t)}};
    for (const auto& i : in)
        if (i.p && meets(ysp, i.s)) return CVX_ERR_ALIAS;
    if (p.ws_bytes) {
        if (workspace == nullptr || ws_bytes < p.ws_bytes) return CVX_ERR_WORKSPACE;
        if (!aligned_to(workspace, 16)) return CVX_ERR_ALIGN;
        if (meets(wsp, ysp)) return CVX_ERR_ALIAS;
        for (const auto& i : in)
            if (i.p && meets(wsp, i.s)) return CVX_ERR_ALIAS;
    }
    a.part = static_cast<float*>(workspace);
    a.joined = nullptr;
    a.down = nullptr;
    if (p.join) {
        a.joined = static_cast<char*>(workspace) + (size_t)p.slices * d->tokens * d->rank * sizeof(float);
        a.down = reinterpret_cast<float*>(static_cast<char*>(a.joined) + lora_joined_bytes(d->tokens, d->rank));
    }
    a.tokens = d->tokens;
    a.cin = d->c_in;
    a.cout = d->c_out;
    a.act = d->act;
    a.res_mode = d->res_mode;
    a.rank = d->rank;
    a.n_adapters = d->n_adapters;
    a.slices = p.slices;
    a.slice_len = p.slice_len;
    a.tiles_m = a.tiles_n = 0;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int held = held_of(d->dtype, d->x_dtype);
    if (lora && !p.one && launch_lora_down(a, p, d->dtype, held, s) != hipSuccess) return CVX_ERR_HIP;
    if (p.join && launch_lora_join(a, d->dtype, s) != hipSuccess) return CVX_ERR_HIP;
    const hipError_t e = p.few ? launch_linear_few(a, p, d->dtype, held, s) : launch_linear_tile(a, p, d->dtype, held, s);
    return e == hipSuccess ? CVX_OK : CVX_ERR_HIP;
}

cvx_status cvx_linear_grouped_plan(const cvx_grouped_desc* d, char* buf, int buf_len)
{
    if (buf == nullptr || buf_len < 1) return CVX_ERR_NULL;
    long xs, ys;
    const cvx_status st = check_grouped(d, &xs, &ys);
    if (st != CVX_OK) return st;
    grouped_describe(*d, grouped_plan(*d), buf, buf_len);
    return CVX_OK;
}

cvx_status cvx_linear_grouped(const cvx_grouped_desc* d, const void* x, const float* x_scale, const void* w,
                              const float* scale, const float* bias, const int* offset, const int* row_id,
                              const float* row_weight, void* y, void* stream)
{
    GroupArgs a;
    const cvx_status st = check_grouped(d, &a.xs, &a.ys);
    if (st != CVX_OK) return st;
    const bool x8 = dtype8(d->x_dtype);
    const long ex = dt_bytes(d->x_dtype);
    // rows found by their number lie at 32-bit offsets, as many as stay below kOOB
    if (row_id ? ((d->tokens - 1) * a.xs + d->c_in) * ex > (1l << 31) : d->tokens < d->rows) return CVX_ERR_SHAPE;
    if (!x || !w || !y || !offset || (x8 && !x_scale)) return CVX_ERR_NULL;
    a.x = x;
    a.x_scale = x8 ? x_scale : nullptr;
    a.w = w;
    a.scale = scale;
    a.bias = bias;
    a.offset = offset;
    a.row_id = row_id;
    a.weight = row_weight;
    a.y = y;
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(y, 8) || !aligned_to(a.x_scale, 4) ||
        !aligned_to(scale, 4) || !aligned_to(bias, 4) || !aligned_to(offset, 4) || !aligned_to(row_id, 4) ||
        !aligned_to(row_weight, 4))
        return CVX_ERR_ALIGN;
    const Span ysp = rows_span(y, d->rows, a.ys, d->c_out, 2);
    const size_t outs = (size_t)d->n_groups * d->c_out;
    const struct {
        const void* p;
        Span s;
    } in[] = {{x, rows_span(x, d->tokens, a.xs, d->c_in, (unsigned)ex)},
              {a.x_scale, bytes_span(a.x_scale, 4ul * d->tokens)},
              {w, bytes_span(w, outs * d->c_in * ex)},
              {scale, bytes_span(scale, 4 * outs)},
              {bias, bytes_span(bias, 4 * outs)},
              {offset, bytes_span(offset, 4ul * d->n_groups + 4)},
              {row_id, bytes_span(row_id, 4ul * d->rows)},
              {row_weight, bytes_span(row_weight, 4ul * d->rows)}};
    for (const auto& i : in)
        if (i.p && meets(ysp, i.s)) return CVX_ERR_ALIAS;
    a.rows = d->rows;
    a.tokens = d->tokens;
    a.groups = d->n_groups;
    a.cin = d->c_in;
    a.cout = d->c_out;
    a.act = d->act;
    a.tiles_m = 0;
    const hipError_t e = launch_linear_grouped(a, grouped_plan(*d), d->dtype, held_of(d->dtype, d->x_dtype),
                                               static_cast<hipStream_t>(stream));
    return e == hipSuccess ? CVX_OK : CVX_ERR_HIP;
}

}  // extern "C"
