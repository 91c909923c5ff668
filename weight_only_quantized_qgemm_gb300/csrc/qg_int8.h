// Internal interface of the 8-bit integer kernels (qg_int8.cu) for the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

struct Int8Args {
    const int8_t* Xq;    // [M, ldxq]
    int64_t ldxq;
    const float* Sx;     // [M]
    const float* Sw;     // [N]
    const float* bias;   // [N] or null
    void* Y;             // [M, ldy] of y_type
    int64_t ldy;
    int y_type;          // QG_BF16, QG_FP16 or QG_FP32
    int M, N, K;
    void* ws;
};

// The CTAs that work on a tile together, for a schedule's activation rows per
// tile (nmma, the MMA's N side): 2 is a CTA pair with a tile of 256 weight
// rows, and the schedule's G then counts pairs.
inline int int8_ctas(int tile_rows) { return tile_rows > 64 ? 2 : 1; }

// The work of a shape: G workers (CTAs or CTA pairs) run nfull whole tiles
// each, then tail_g of them share the units of the other T - nfull G tiles;
// split: a tile is cut.  (The other kinds' schedules leave these at 0.)
struct Int8Schedule : Schedule {
    int nfull = 0;
    int tail_g = 0;
    bool split = false;
    // > 1: a cluster of this many workers runs equal pieces of each tile (nfull
    // is 0, tail_g = G = T * pieces)
    int pieces = 0;
};

// CTAs of a cluster that share a tile, at most (five pairs; single CTAs: 8).
constexpr int kMostClusterCtas = 10;
// The clusters of c CTAs that run at once on the current device, for each c.
void int8_cluster_capacity(int (&clusters)[kMostClusterCtas + 1]);
// The same on a GB300 with 152 SMs, for questions without a device.
inline const int* int8_nominal_clusters(int sms) {
    static constexpr int kNone[kMostClusterCtas + 1] = {};
    static constexpr int kFull[kMostClusterCtas + 1] = {0, 0, 76, 46, 36, 28, 23, 15, 15, 0, 13};
    return sms == 152 ? kFull : kNone;
}

// The schedule of a shape on `sms` SMs (forced > 0: with that many CTAs, the
// tail cut evenly over all of them); clusters: the device's capacity by CTAs a cluster.
Int8Schedule int8_schedule(int M, int N, int K, int sms, int forced, const int* clusters);

// Workspace of a schedule (s.nmma = the tile's activation rows): the arrival
// counters (kInt8CounterBytes, zero between calls, at offset 0 for every
// shape), the activations as FP16 [M, K] (nothing where the GEMM expands them
// itself, int8_inline_x), then the split-K partial sums of a schedule that
// splits tiles (two slots of 128 x s.nmma FP32 per CTA); 0 when it holds neither.
constexpr size_t kInt8CounterBytes = 32768;
constexpr int kInt8Slices = 2;   // counters of an epilogue warp of a split tile
inline bool int8_inline_x(const Schedule& s) { return s.nmma <= 16; }
size_t int8_expanded_bytes(const Schedule& s, int M, int K);
size_t int8_workspace_bytes(const Int8Schedule& s, int M, int K);

// tmW: the weight map ([N, K] bytes, 128 x 128 boxes, 128-byte swizzle);
// tmX: the expanded activations ([M, K] FP16, boxes of 64 K x the rows of a
// tile that one CTA holds, s.nmma / int8_ctas), not used where the GEMM expands
// them itself.
cudaError_t launch_int8(const Int8Args& a, const Int8Schedule& s, const CUtensorMap& tmW, const CUtensorMap& tmX,
                        const LaunchCtl& c, cudaStream_t st);
cudaError_t launch_quantize_int8(const void* X, int x_type, int64_t ldx, int8_t* Xq, int64_t ldxq, float* Sx, int M,
                                 int K, const LaunchCtl& c, cudaStream_t st);
// Y = bias (or zeros) in every row: the K = 0 product.
cudaError_t launch_int8_bias_rows(const Int8Args& a, cudaStream_t st);

}  // namespace qg
