// Log probabilities of given tokens, entropy and top alternatives over rows of
// logits (e.g. the output of an lm_head GEMM), for sm_103a.
//
//   m = max_v x[v],  s = sum_v exp(x[v] - m),  logp[v] = x[v] - m - ln s
//   H = ln s - (1/s) sum_v exp(x[v] - m) (x[v] - m)
//
// all sums in FP32.  The alternatives are ordered by value, ties by the lower
// index, on 32-bit keys that order like the values (NaN above +inf, -0 = +0).
//
// One CTA per row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_device.cuh"
#include "qg_logprobs.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int kType>
__device__ __forceinline__ float load_logit(const void* row, int64_t v) {
    if constexpr (kType == QG_FP32) return static_cast<const float*>(row)[v];
    if constexpr (kType == QG_BF16)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[v]) << 16);
    return __half2float(static_cast<const __half*>(row)[v]);
}

// Keys that order like the values they stand for: -inf lowest, NaN highest.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));   // -0 becomes +0
    return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = 0.0f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) r += buf[j];
    return r;
}

__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* buf) {
    x = __reduce_max_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t r = 0u;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) r = max(r, buf[j]);
    return r;
}

// The top alternatives of a row, one distinct value at a time: the largest key
// below the previous one, then its occurrences in index order.
template <int kType>
__device__ void top_by_value(const void* row, int V, int k, uint32_t* buf, uint32_t* keys, int* ids) {
    int have = 0;
    uint64_t below = 1ull << 32;   // keys under this are left
    while (have < k) {
        uint32_t best = 0u;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const uint32_t key = order_key(load_logit<kType>(row, v));
            if (key < below) best = max(best, key);
        }
        best = block_max(best, buf);
        for (int v0 = 0; v0 < V && have < k; v0 += kThreads) {
            const int v = v0 + threadIdx.x;
            const bool hit = v < V && order_key(load_logit<kType>(row, v)) == best;
            const uint32_t mask = __ballot_sync(0xffffffffu, hit);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = __popc(mask);
            __syncthreads();
            int before = 0, total = 0;
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                if (j < static_cast<int>(threadIdx.x >> 5)) before += buf[j];
                total += buf[j];
            }
            const int at = have + before + __popc(mask & ((1u << (threadIdx.x & 31)) - 1u));
            if (hit && at < k) {
                keys[at] = best;
                ids[at] = v;
            }
            have += total;
        }
        below = best;
    }
    __syncthreads();
}

template <int kType>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
    __shared__ float fbuf[kWarps];
    __shared__ uint32_t ubuf[kWarps];
    __shared__ uint32_t top_keys[kMaxTopK];
    __shared__ int top_ids[kMaxTopK];
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t m = blockIdx.x;
    constexpr int kSize = kType == QG_FP32 ? 4 : 2;
    const void* row = static_cast<const uint8_t*>(a.logits) + m * a.ld * kSize;
    uint32_t best = 0u;
    for (int v = threadIdx.x; v < a.V; v += kThreads) best = max(best, order_key(load_logit<kType>(row, v)));
    const float mx = key_value(block_max(best, ubuf));
    const bool none = mx == -INFINITY;   // a row with nothing left
    float s = 0.0f, w = 0.0f;
    if (!none)
        for (int v = threadIdx.x; v < a.V; v += kThreads) {
            const float d = load_logit<kType>(row, v) - mx;
            const float e = __expf(d);
            s += e;
            if (e != 0.0f) w += e * d;
        }
    s = block_sum(s, fbuf);
    w = block_sum(w, fbuf);
    const float ls = logf(s);
    for (int t = threadIdx.x; t < a.T; t += kThreads) {
        const int64_t id = a.tokens[m * a.ldt + t];
        const bool in = id >= 0 && id < a.V;
        a.token_lp[m * a.T + t] = !in || none ? -INFINITY : load_logit<kType>(row, id) - mx - ls;
    }
    if (a.entropy && threadIdx.x == 0) a.entropy[m] = none ? 0.0f : ls - w / s;
    if (a.top_k > 0) {
        top_by_value<kType>(row, a.V, a.top_k, ubuf, top_keys, top_ids);
        if (threadIdx.x < a.top_k) {
            a.top_ids[m * a.top_k + threadIdx.x] = top_ids[threadIdx.x];
            a.top_lp[m * a.top_k + threadIdx.x] = none ? -INFINITY : key_value(top_keys[threadIdx.x]) - mx - ls;
        }
    }
}

template <int kType>
cudaError_t launch(const LogprobArgs& a, const LaunchCtl& c, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    if (c.overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<kType>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, const LaunchCtl& c, cudaStream_t st) {
    switch (a.type) {
        case QG_BF16: return launch<QG_BF16>(a, c, st);
        case QG_FP16: return launch<QG_FP16>(a, c, st);
        case QG_FP32: return launch<QG_FP32>(a, c, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace qg
