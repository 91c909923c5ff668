// Internal interface of the kernels around the grouped GEMM (qg_experts.cu):
// router, row quantiser and combination.
#pragma once

#include "qg_internal.h"

namespace qg {

struct RouteArgs {
    const void* logits;    // [M, ld] of type
    int type;
    int64_t ld;
    const float* bias;     // [E] or null
    int score;             // QG_SCORE_SOFTMAX or QG_SCORE_SIGMOID
    int renormalize;
    float scale;
    int top_k;
    int32_t* experts;      // [M, top_k]
    float* weights;        // [M, top_k]
    int32_t* offsets;      // [E + 1]
    int32_t* rows;         // [M, top_k]
    int M, E;
    void* ws;
};
size_t route_workspace_bytes(int M, int E, int sms);
cudaError_t launch_route(const RouteArgs& a, const LaunchCtl& c, cudaStream_t st);

struct QuantizeRowsArgs {
    const void* X;            // [M, ldx] of x_type; gated: 2 K columns, gate then up
    int x_type;
    int64_t ldx;
    int gated;
    const int32_t* rows;      // [M, top_k] or null (row m to row m)
    int top_k;
    const int32_t* num_rows;  // device, or null (M)
    uint8_t* Xq;              // [out_rows, ldxq]
    int64_t ldxq;
    float* Sx;                // [ceil(K/128), ldsx]
    int64_t ldsx;
    int M, out_rows, K;
};
cudaError_t launch_quantize_rows(const QuantizeRowsArgs& a, const LaunchCtl& c, cudaStream_t st);

struct CombineArgs {
    const void* Y;            // [R, ldy] of type
    int type;
    int64_t ldy;
    const int32_t* rows;      // [M, top_k]
    const float* weights;     // [M, top_k]
    int top_k;
    const void* residual;     // [M, ldr] or null
    int64_t ldr;
    void* out;                // [M, ldo]
    int64_t ldo;
    int M, R, K;
};
cudaError_t launch_combine(const CombineArgs& a, const LaunchCtl& c, cudaStream_t st);

}  // namespace qg
