// ops.cuh -- the operators around int8 experts (scored routing, int8 products,
// the int8-activation FFN, the block norms): what abi.cu hands to their
// launchers.
#pragma once

#include "common.cuh"

namespace moe {

// Scored routing (route_scored.cu).
struct ScoredArgs {
    const float *logits, *bias;  // [T][E]; [E] or null
    int T, E, k;
    int sigmoid, n_group, group_size, topk_group, group_top, renorm;
    float scale;
    int32_t *ids;
    float *w;
};
cudaError_t launch_route_scored(const ScoredArgs &a, cudaStream_t s);

// Block norms (norm.cu).
struct NormArgs {
    const float *rows;  // combine source: rows, route_pos, w (k routes per token), or null
    const int32_t *route_pos;
    const float *w;
    int k;
    const uint16_t *z;         // dense source, or null
    const uint16_t *residual;  // with a block source; without one the row to normalise
    const uint16_t *post_w, *next_w;
    const float *gate_h, *gate_t;
    float eps, offset, residual_scale, block_scale;
    int T, H;
    uint16_t *y, *xn;
    int8_t *xq;
    float *sx;
    float inv_h;  // 1 / H
};
cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s);

// int8 x int8 products (i8_gemv.cu: few tokens; i8_tc.cu: tensor cores).
struct LinearArgs {
    const int8_t *xq, *wq;  // [T][K], [N][K]
    const float *sx, *sw;   // [T], [N]
    int T, N, K;
    void *y;                // [T][N] bf16 or fp32
    int fp32;
};
cudaError_t launch_linear_i8(const LinearArgs &a, cudaStream_t s);
cudaError_t launch_linear_i8_tc(const LinearArgs &a, cudaStream_t s);

// Grouped FFN with int8 activations over int8 experts (same files).
struct FfnI8Args {
    LayerView L;
    const int8_t *xq;  // [T][H]
    const float *sx;   // [T]
    int T, k;
    const int32_t *counts, *offsets, *sorted_route;
    float *rows;       // [T k][H], sorted order
    void *ws;
};
size_t ffn_i8_workspace(int E, int H, int I, int T, int k);  // of whichever kernels take the call
cudaError_t launch_ffn_i8(const FfnI8Args &a, cudaStream_t s);
size_t ffn_i8_tc_workspace(int H, int I, int T, int k);
cudaError_t launch_ffn_i8_tc(const FfnI8Args &a, cudaStream_t s);
cudaError_t i8_take_error(unsigned *code, unsigned *info);
cudaError_t i8tc_take_error(unsigned *code, unsigned *info);

}  // namespace moe
