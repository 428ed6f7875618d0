// tokens.h -- declarations of the operators on tokens (rows of channels): the
// root-mean-square norm and the projection with low-rank adapters.  Not part of
// the public ABI (include/cvx.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cvx.h"

namespace cvx {

// ------------------------------------------------------------------ the norm
struct RmsArgs {
    const void* x;
    const void* res;      // or null
    const float* gamma;
    void* sum;            // or null
    void* y;
    float* y_scale;       // 8-bit output only
    long xs, rs, ss, ys;  // row strides, elements
    int rows, c;
    float eps;
    int out8;
};
hipError_t launch_rmsnorm(const RmsArgs& a, int dtype, hipStream_t s);

// ------------------------------------------------------------ the projection
struct LinArgs {
    const void* x;
    const float* x_scale;  // 8-bit x only
    const void* w;
    const float* scale;    // or null
    const float* bias;     // or null
    const void* res;       // or null
    const void* lora_a;
    const void* lora_b;
    const float* lora_alpha;  // or null
    const int* lora_id;
    void* y;
    float* part;           // low-rank values [slices][tokens][rank], fp32
    void* joined;          // tile kernel: the same, joined, as high and low 16-bit parts:
                           // [rank/8, to a multiple of two][part][token] pieces of eight; or
                           // null, where the tiles join them
    float* down;           // tile kernel, fp16: per token, the power of two they are multiplied by
    long xs, rs, ys;       // row strides, elements
    int tokens, cin, cout;
    int act, res_mode;
    int rank, n_adapters;
    int slices;            // slices of c_in that v's products are split into
    int slice_len;         // channels a slice
    int tiles_m, tiles_n;  // tile kernel: output channel and token tiles
};

// What runs a projection.
struct LinPlan {
    int few;             // 1: the kernel for few tokens; 0: the tile kernel
    int one;             // few: a single token, the adapter's first product in the same kernel
    int nt, rb;          // few: 16-token blocks and 16-channel blocks a workgroup holds; a grid
                         // row is 16*nt tokens
    int mb, nb;          // tile: 64*mb channels x 64*nb tokens
    int slices, slice_len;
    int join;              // tile: the first product's slices are joined by a kernel of their own
    int down_nb, down_rc;  // first product: 16-token blocks (0: one token) and 16-rank blocks a workgroup
    size_t ws_bytes;
};

constexpr int kLoraChunk = 1024;  // channels a workgroup of k_lora_down takes per step: slices are of whole ones
constexpr int kLoraMany = 512;    // channels in the shortest slice of k_lora_down_many
constexpr int kLoraMaxRank = 128;

inline size_t lora_joined_bytes(long tokens, int rank) { return (size_t)(rank + 15) / 16 * 64 * tokens; }

LinPlan linear_plan(const cvx_linear_desc& d);
void linear_describe(const cvx_linear_desc& d, const LinPlan& p, char* buf, int len);
hipError_t launch_lora_down(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s);
hipError_t launch_lora_join(const LinArgs& a, int dtype, hipStream_t s);
hipError_t launch_linear_few(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s);
hipError_t launch_linear_tile(const LinArgs& a, const LinPlan& p, int dtype, int x8, hipStream_t s);

}  // namespace cvx
