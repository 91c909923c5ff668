// Internal interface of the grouped W8A8 GEMM (qg_grouped.cu) for the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

struct GroupedArgs {
    const float* Sx;          // [ceil(K/128), ldsx]
    int64_t ldsx;
    const float* S;           // [E, ceil(N/128), ceil(K/128)]
    const int32_t* offsets;   // device [E + 1]
    void* Y;                  // [R, ldy] of y_type
    int64_t ldy;
    int y_type;
    int R, E, N, K;
};

// The rows of a tile (more than 64: on a CTA pair, with 256 weight rows).
int grouped_tile_rows(int R, int E, int N, int K, int sms);

// Activation rows of a copy (a pair's CTAs hold half of a tile's rows each).
inline int grouped_box_rows(int tile_rows) { return tile_rows > 64 ? tile_rows / 2 : tile_rows; }

// tmW: the weights as one [E * N, K] matrix of bytes, 128 x 128 boxes, 128-byte
// swizzle; tmX: the activations ([R, K] bytes, boxes of 128 K x
// grouped_box_rows).
cudaError_t launch_grouped(const GroupedArgs& a, const CUtensorMap& tmW, const CUtensorMap& tmX, const LaunchCtl& c,
                           cudaStream_t st);
// Zeros in the rows of the groups: the K = 0 product.
cudaError_t launch_grouped_zero(const GroupedArgs& a, cudaStream_t st);

}  // namespace qg
