// What a layer of experts needs around its grouped products, for sm_103a: the
// router, the quantiser that copies a token's activations to its experts' rows
// (or applies the gate between an expert's two products), and the weighted sum
// of the experts' results.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_device.cuh"
#include "qg_experts.h"
#include "qg_launch.h"

namespace qg {
namespace {

template <int kType>
__device__ __forceinline__ float to_f32(const void* p, int64_t i) {
    if (kType == QG_FP32) return static_cast<const float*>(p)[i];
    if (kType == QG_BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    return __half2float(static_cast<const __half*>(p)[i]);
}

// Launched ahead of the preceding grid's end: every kernel here waits for it
// before it touches memory.
cudaLaunchConfig_t config(unsigned grid, unsigned block, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// ----------------------------------------------------------------- router
// A warp takes a token: lane l holds experts l, l + 32, ...  Of the choices'
// order by expert, then by token, each CTA knows its own part: a warp counts its
// tokens' choices by expert, the counts of a CTA's warps add up in order, and
// with more than one CTA a second kernel adds the counts of the CTAs in front.
// (Counting, not atomics, so that the order is that of the tokens on every call.)
// Bound by instructions and latency, not by bytes: 8192 x 256, top 8 with biases, 20
// us (17 of them the first kernel: 1012 instructions a token, half the issue slots)
// for 5 MB; 16 x 128 4 us.
//
// Without a bias the order of the scores is that of the logits, which are
// compared as they are.  With one the scores decide that are next to another,
// and 32 bits are not enough for those: where the chosen ones, or the last one
// and the next, lie closer than the scores' error, the token is done again in 64.
// Warps of a CTA, one CTA on an SM: as many as the registers for PL experts a lane
// allow (a token is a chain of reductions, of which 16 warps hide too little).
template <int PL>
constexpr int kRouteWarps = PL <= 16 ? 32 : 16;
inline int route_warps(int E) { return E <= 512 ? 32 : 16; }
// How near, relative to max(1, |sum|).  The quick sigmoid's e^-x is good to 2^-22 +
// |x| 2^-24, of which s (1 - s) shows in s, its sum with 1 and its reciprocal to 2^-24
// and 2^-23, the sum with the bias to another 2^-24: less than 4e-7 for each of two.
// Softmax: the common total of up to 37 roundings comes on top.
constexpr float kNearSigmoid = 1e-6f, kNearSoftmax = 6e-6f;

// A value's bits as a whole number that orders like it (never 0).
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 as 0
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        v = w > v ? w : v;
    }
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The largest keys above 0, the j0-th to the one in front of the j1-th, in order
// (ties to the lower expert), taken out of `key`: lane j receives the j-th one's
// expert and its key, and keeps what it had where none is left.
template <class Key, int PL>
__device__ __forceinline__ void choose(Key (&key)[PL], int j0, int j1, int lane, int& expert, Key& at) {
    for (int j = j0; j < j1; ++j) {
        Key best = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        const Key top = warp_max(best);
        if (top == 0) return;
        const int e = static_cast<int>(
            __reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(bi * 32 + lane) : 0xffffffffu));
        if (lane == (e & 31)) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (i == e >> 5) key[i] = 0;
        }
        if (lane == j) {
            expert = e;
            at = top;
        }
    }
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The `want` largest keys above 0 and whatever else reaches the want-th largest of
// the lanes' maxima (which at least that many do), in order: lane j receives the
// j-th one's expert (-1: none) and key.  Returns how many they are; more than 32: too
// many for this, nothing was done.  A few more than `want` in general, which are
// ranked by counting: half the instructions of taking them out one by one.
template <int PL>
__device__ __forceinline__ int sorted_largest(const uint32_t (&key)[PL], int want, int lane, uint2* held, int& expert,
                                              uint32_t& at, uint32_t& bound) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = best > key[i] ? best : key[i];
    bound = 1u;
    for (int seen = 0; seen < want;) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0u) {   // fewer lanes than that hold any
            bound = 1u;
            break;
        }
        bound = top;
        seen += __popc(__ballot_sync(0xffffffffu, best == top));
        if (best == top) best = 0u;
    }
    const uint32_t before = (1u << lane) - 1u;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t all = __ballot_sync(0xffffffffu, in);
        const int place = n + __popc(all & before);
        if (in && place < 32) held[place] = make_uint2(key[i], static_cast<uint32_t>(i * 32 + lane));
        n += __popc(all);
    }
    if (n > 32) return n;
    __syncwarp();
    const uint2 mine = lane < n ? held[lane] : make_uint2(0u, 0xffffffffu);
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const uint2 o = held[i];
        rank += o.x > mine.x || (o.x == mine.x && o.y < mine.y) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) held[rank] = mine;
    __syncwarp();
    const uint2 now = lane < n ? held[lane] : make_uint2(0u, 0xffffffffu);
    __syncwarp();   // `held` serves the next token
    expert = static_cast<int>(now.y);
    at = now.x;
    return n;
}

// Whether two sums, x's not below y's, may be in another order in 64 bits.
__device__ __forceinline__ bool nearly(uint32_t x, uint32_t y, float near) {
    const float a = key_value(x);
    return !(a - key_value(y) > near * fmaxf(1.0f, fabsf(a)));
}

__device__ __forceinline__ float quick_exp(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}
__device__ __forceinline__ float quick_reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One token: lane j < k receives its j-th expert (-1: none) and the weight.  held: 32
// pairs of the warp's own.
template <int kType, int PL>
__device__ __forceinline__ void route_token(const RouteArgs& a, const void* row, int lane, uint2* held, int& expert,
                                            float& weight) {
    float v[PL];
    float top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < a.E ? to_f32<kType>(row, e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        top = fmaxf(top, v[i]);
        bad |= !(v[i] < INFINITY);   // NaN or +inf
    }
    if (__any_sync(0xffffffffu, bad)) {   // routed nowhere, and the weights say so
        expert = -1;
        weight = __uint_as_float(0x7FC00000u);
        return;
    }
    const int k = a.top_k;
    const bool soft = a.score == QG_SCORE_SOFTMAX;
    if (soft) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    uint32_t key[PL], at = 0u, bound;
    float total = 0.0f;   // of the softmax, where it is needed
    if (soft && (a.bias != nullptr || !a.renormalize)) {
#pragma unroll
        for (int i = 0; i < PL; ++i) total += expf(v[i] - top);
        total = warp_sum(total);
    }
    if (a.bias == nullptr) {
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = v[i] > -INFINITY ? order_key(v[i]) : 0u;
        if (sorted_largest(key, k, lane, held, expert, at, bound) > 32) {
            expert = -1;
            choose(key, 0, k, lane, expert, at);
        }
    } else {
        const float unit = soft ? 1.0f / total : 1.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = i * 32 + lane;
            const float s = soft ? quick_exp(v[i] - top) * unit : quick_reciprocal(1.0f + quick_exp(-v[i]));
            const float by = s + (e < a.E ? __ldg(a.bias + e) : 0.0f);
            key[i] = v[i] > -INFINITY && by > -INFINITY ? order_key(by) : 0u;   // a NaN is above nothing
        }
        // the next one behind the chosen too
        const int n = sorted_largest(key, k < 32 ? k + 1 : 32, lane, held, expert, at, bound);
        const float margin = soft ? kNearSoftmax : kNearSigmoid;
        bool wide_all = n > 32;
        if (!wide_all) {
            const uint32_t next = __shfl_down_sync(0xffffffffu, at, 1), kth = __shfl_sync(0xffffffffu, at, k - 1);
            bool near = lane < (k < 32 ? k : 31) && next != 0u && nearly(at, next, margin);
            if (k == 32) {   // no lane holds the next one
#pragma unroll
                for (int i = 0; i < PL; ++i) near |= key[i] != 0u && key[i] < bound && nearly(kth, key[i], margin);
            }
            if (__any_sync(0xffffffffu, near)) {
                // The sums that may belong among the first k in 64 bits, as far as lanes
                // hold them all.
                bool more = soft;   // whose total would have to be in 64 bits, too
#pragma unroll
                for (int i = 0; i < PL; ++i) more |= key[i] != 0u && key[i] < bound && nearly(kth, key[i], margin);
                wide_all = __any_sync(0xffffffffu, more);
                if (!wide_all) {
                    const bool in = at != 0u && (lane < k || nearly(kth, at, margin));
                    const int m = __popc(__ballot_sync(0xffffffffu, in));   // the first m lanes
                    uint64_t wide = 0;
                    if (in) {
                        const double x = to_f32<kType>(row, expert);
                        const double by = 1.0 / (1.0 + exp(-x)) + static_cast<double>(a.bias[expert]);
                        if (by > -INFINITY) wide = order_key(by);
                    }
                    int rank = 0;
                    for (int i = 0; i < m; ++i) {
                        const uint64_t w = __shfl_sync(0xffffffffu, wide, i);
                        const int e = __shfl_sync(0xffffffffu, expert, i);
                        rank += w > wide || (w == wide && e < expert) ? 1 : 0;
                    }
                    if (wide == 0) rank = 32;
                    int mine = -1;
                    for (int i = 0; i < m; ++i) {
                        const int r = __shfl_sync(0xffffffffu, rank, i);
                        const int e = __shfl_sync(0xffffffffu, expert, i);
                        if (r == lane) mine = e;
                    }
                    expert = mine;
                }
            }
        }
        if (wide_all) {
            uint64_t wide[PL], wat = 0;
            double sum = 1.0;
            if (soft) {
                sum = 0.0;
#pragma unroll 1
                for (int i = 0; i < PL; ++i) {
                    const int e = i * 32 + lane;
                    if (e < a.E) sum += exp(static_cast<double>(to_f32<kType>(row, e)) - static_cast<double>(top));
                }
                sum = warp_sum(sum);
            }
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int e = i * 32 + lane;
                wide[i] = 0;
                if (e < a.E && v[i] > -INFINITY) {
                    const double x = v[i];
                    const double s = soft ? exp(x - static_cast<double>(top)) / sum : 1.0 / (1.0 + exp(-x));
                    const double by = s + static_cast<double>(a.bias[e]);
                    if (by > -INFINITY) wide[i] = order_key(by);
                }
            }
            expert = -1;
            choose(wide, 0, k, lane, expert, wat);
        }
    }
    if (lane >= k) expert = -1;
    // The weights, from the chosen logits.  Renormalized ones are ratios: about the
    // largest of the chosen, whose scores a bias (or sigmoids of low logits) may leave
    // anywhere below 1, down to where 64 bits hold none.
    const float x = expert >= 0 ? to_f32<kType>(row, expert) : 0.0f;
    float from = top;
    bool about = soft, nothing = false;
    if (a.renormalize) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, expert >= 0 ? order_key(x) : 0u);
        from = most != 0u ? key_value(most) : 0.0f;
        nothing = (soft ? from - top : from) < -690.0f;
        about = soft || from < -60.0f;   // where sigmoids are exponentials, which 32 bits may not hold
    }
    float w = 0.0f;
    if (expert >= 0 && !nothing) w = about ? expf(x - from) : 1.0f / (1.0f + expf(-x));
    const float sum = a.renormalize ? warp_sum(w) : soft ? total : 1.0f;
    weight = sum > 0.0f ? w * (a.scale / sum) : 0.0f;
}

// The CTAs' counts by expert have 16 bits, and a token takes an expert once: so many
// tokens a CTA at most, which a device of few SMs would pass.
constexpr int kMostTokens = 0xFFFF;

inline int route_ctas(int M, int E, int sms) {
    // up to a token a warp one CTA does it all (64 tokens, 256 experts: 10.4 us; over
    // eight CTAs with the second launch 8.7)
    if (M <= route_warps(E)) return 1;
    const int most = (M + 7) / 8, least = (M + kMostTokens - 1) / kMostTokens;
    const int ctas = most < sms ? most : sms;
    return ctas < least ? least : ctas;
}

// The table of the counts: rows of whole 16 bytes.
__host__ __device__ inline int route_pitch(int E) { return (E + 7) / 8 * 8; }

// where[e] = the exclusive prefix over the experts of total[e] (each a CTA's or
// the whole call's), total in shared memory; all threads of the CTA.
__device__ __forceinline__ void prefix_experts(const int* total, int* where, int E) {
    if (threadIdx.x < 32) {
        int before = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + static_cast<int>(threadIdx.x);
            const int mine = e < E ? total[e] : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int other = __shfl_up_sync(0xffffffffu, upto, o);
                if (static_cast<int>(threadIdx.x) >= o) upto += other;
            }
            if (e < E) where[e] = before + upto - mine;
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (threadIdx.x == 0) where[E] = before;
    }
    __syncthreads();
}

constexpr int kHeldTokens = 4;   // of a warp

template <int kType, int PL>
__global__ void __launch_bounds__(kRouteWarps<PL> * 32) route_kernel(const RouteArgs a, int chunk) {
    constexpr int kWarps = kRouteWarps<PL>;
    extern __shared__ int route_smem[];
    int* count = route_smem;                        // [warps][E]
    int* total = route_smem + kWarps * a.E;    // [E]
    int* where = total + a.E;                       // [E + 1]
    // a warp's choices, where they are few: expert, and place among the warp's
    __shared__ ushort2 held[kWarps][kHeldTokens][32];
    __shared__ uint2 sorting[kWarps][32];
    grid_dependents_launch();
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kWarps * a.E; i += kWarps * 32) count[i] = 0;
    grid_dependency_wait();
    __syncthreads();
    // contiguous tokens to a CTA, and of those to a warp
    const int c0 = blockIdx.x * chunk;
    const int c1 = c0 + chunk < a.M ? c0 + chunk : a.M;
    const int each = (chunk + kWarps - 1) / kWarps;
    const int t0 = c0 + warp * each;
    const int t1 = t0 + each < c1 ? t0 + each : c1;
    int* mine = count + warp * a.E;
    const int64_t size = kType == QG_FP32 ? 4 : 2;
    for (int m = t0; m < t1; ++m) {
        int expert;
        float weight;
        route_token<kType, PL>(a, static_cast<const uint8_t*>(a.logits) + m * a.ld * size, lane, sorting[warp], expert, weight);
        if (lane < a.top_k) {
            const int64_t at = static_cast<int64_t>(m) * a.top_k + lane;
            a.experts[at] = expert;
            a.weights[at] = weight;
            // its place among the warp's choices of the expert; a token's experts differ
            const int place = expert >= 0 ? mine[expert]++ : -1;
            if (each <= kHeldTokens) held[warp][m - t0][lane] = make_ushort2(static_cast<uint16_t>(expert), static_cast<uint16_t>(place));
            else a.rows[at] = place;
        }
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kWarps * 32) {
        int sum = 0;
        constexpr int kBatch = 16;   // loads on the way at a time
#pragma unroll
        for (int w0 = 0; w0 < kWarps; w0 += kBatch) {
            int n[kBatch];
#pragma unroll
            for (int w = 0; w < kBatch; ++w) n[w] = count[(w0 + w) * a.E + e];
#pragma unroll
            for (int w = 0; w < kBatch; ++w) {
                count[(w0 + w) * a.E + e] = sum;
                sum += n[w];
            }
        }
        total[e] = sum;
        if (gridDim.x > 1)
            static_cast<uint16_t*>(a.ws)[static_cast<int64_t>(blockIdx.x) * route_pitch(a.E) + e] = static_cast<uint16_t>(sum);
    }
    __syncthreads();
    if (gridDim.x == 1) {
        prefix_experts(total, where, a.E);
        for (int e = threadIdx.x; e <= a.E; e += kWarps * 32) a.offsets[e] = where[e];
    }
    if (each <= kHeldTokens) {
        for (int m = t0; m < t1; ++m) {
            if (lane >= a.top_k) continue;
            const ushort2 h = held[warp][m - t0][lane];
            a.rows[static_cast<int64_t>(m) * a.top_k + lane] =
                h.x == 0xFFFFu ? -1 : h.y + mine[h.x] + (gridDim.x == 1 ? where[h.x] : 0);
        }
        return;
    }
    for (int64_t i = static_cast<int64_t>(t0) * a.top_k + lane; i < static_cast<int64_t>(t1) * a.top_k; i += 32) {
        const int e = a.experts[i];
        if (e >= 0) a.rows[i] += mine[e] + (gridDim.x == 1 ? where[e] : 0);
    }
}

// Behind route_kernel on several CTAs: where each expert's rows begin, and the
// rows of this CTA's choices, from all CTAs' counts.
constexpr int kPlaceThreads = 1024;
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteArgs a, int chunk) {
    extern __shared__ int route_smem[];
    int* total = route_smem;            // [E]: of all CTAs
    int* front = total + a.E;           // [E]: of the CTAs in front
    int* where = front + a.E;           // [E + 1]
    grid_dependents_launch();
    grid_dependency_wait();
    // A warp adds up eight experts at a time, a lane a share of the CTAs.
    const uint4* table = static_cast<const uint4*>(a.ws);
    const int ctas = gridDim.x;
    const int groups = route_pitch(a.E) / 8;
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kPlaceThreads / 32) {
        int all[8] = {}, before[8] = {};
        constexpr int kBatch = 5;   // loads on the way at a time: of up to 160 CTAs, all
        for (int b0 = lane; b0 < ctas; b0 += 32 * kBatch) {
            uint4 w[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int b = b0 + 32 * i;
                w[i] = b < ctas ? __ldcg(table + static_cast<int64_t>(b) * groups + g) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                const bool front_of = b0 + 32 * i < static_cast<int>(blockIdx.x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int lo = static_cast<int>(u[e] & 0xFFFFu), hi = static_cast<int>(u[e] >> 16);
                    all[2 * e] += lo;
                    all[2 * e + 1] += hi;
                    before[2 * e] += front_of ? lo : 0;
                    before[2 * e + 1] += front_of ? hi : 0;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 8 * g + i;
            const int t = __reduce_add_sync(0xffffffffu, all[i]), f = __reduce_add_sync(0xffffffffu, before[i]);
            if (lane == 0 && e < a.E) {
                total[e] = t;
                front[e] = f;
            }
        }
    }
    __syncthreads();
    prefix_experts(total, where, a.E);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += kPlaceThreads) a.offsets[e] = where[e];
    const int c0 = blockIdx.x * chunk;
    const int c1 = c0 + chunk < a.M ? c0 + chunk : a.M;
    for (int64_t i = static_cast<int64_t>(c0) * a.top_k + threadIdx.x; i < static_cast<int64_t>(c1) * a.top_k;
         i += kPlaceThreads) {
        const int e = __ldcg(a.experts + i);
        if (e >= 0) a.rows[i] = __ldcg(a.rows + i) + where[e] + front[e];
    }
}

template <int kType, int PL>
cudaError_t launch_route_pl(const RouteArgs& a, const LaunchCtl& c, cudaStream_t st) {
    const int ctas = route_ctas(a.M, a.E, c.num_sms);
    const int chunk = a.M > 0 ? (a.M + ctas - 1) / ctas : 1;
    cudaLaunchAttribute attr;
    const size_t smem = (kRouteWarps<PL> + 2) * a.E * sizeof(int) + sizeof(int);
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(configured, route_kernel<kType, PL>, (kRouteWarps<PL> + 2) * 32 * PL * 4 + 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(ctas), kRouteWarps<PL> * 32, smem, st, &attr);
    e = cudaLaunchKernelEx(&cfg, route_kernel<kType, PL>, a, chunk);
    if (e != cudaSuccess || ctas == 1) return e;
    cfg = config(static_cast<unsigned>(ctas), kPlaceThreads, (3 * a.E + 1) * sizeof(int), st, &attr);
    return cudaLaunchKernelEx(&cfg, route_place_kernel, a, chunk);
}

template <int kType>
cudaError_t launch_route_type(const RouteArgs& a, const LaunchCtl& c, cudaStream_t st) {
    if (a.E <= 64) return launch_route_pl<kType, 2>(a, c, st);
    if (a.E <= 128) return launch_route_pl<kType, 4>(a, c, st);
    if (a.E <= 256) return launch_route_pl<kType, 8>(a, c, st);
    if (a.E <= 512) return launch_route_pl<kType, 16>(a, c, st);
    return launch_route_pl<kType, 32>(a, c, st);
}

// ----------------------------------------------------------------- row quantiser
// Eight lanes take a block of 128 columns of a row: its maximum, the scale, sixteen
// codes each, which go to every one of the row's places.
template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// silu(g) u in 32 bits: g u / (1 + e^-g).  The exponential is good to
// 2^-22 + |g| 2^-24, the reciprocal to 2^-23: far below an E4M3 step (2^-4).  With
// subnormals as zeros (an e^-g below 2^-126 is nothing beside 1), each is one
// instruction; without, they took 40 % of the kernel's.  The reciprocal is that of a
// quarter of the sum, and a quarter of g is taken (exact: g has 16 bits), so that it
// stays normal up to the sum's overflow at g = -88.7; at 4 2^-126 a gate of -87.4 would
// let nothing through, however large u is.
__device__ __forceinline__ float gate(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmaf_rn(e, 0.25f, 0.25f)));
    return 0.25f * g * r * u;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// x / s, rounded to nearest, from r, the rounded 1 / s: one correction of the
// product by its remainder (Markstein's theorem; s normal, and its reciprocal, and
// x / s of at most 448).  A division of every element took most of the kernel's
// time (issue slots 83 % busy).  With these signs a -0 stays one.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(q, s, -x), -r, q);
}

constexpr int kQuantWarps = 8;
// CTAs per SM: as many as spill no registers (from 5 on they do).  Two shapes with 2 /
// 3 / 4 / 5 / 6: 41 / 45 / 40.5 / 42 / 45 us for 4096 x 5120 to eight rows each, 62 / 57 /
// 50.7 / 54 / 67 for the gate on 32763 x 2 x 2048.
constexpr int kQuantCtas = 4;

// Resident warps walk over jobs (512 columns of a row, 16 of them a lane, so that a
// lane's codes are one 16-byte store and eight lanes share a block), the next
// job's loads on their way while this one's codes are worked out.  Bound by
// memory: the gate on 32763 x 2 x 2048 51 us (6.6 TB/s, 0.97 of the copy rate); 4096 x 5120
// to eight rows each 40 us (5.4 TB/s: scattered rows of 5 KB and, 3 us of it, scales).
template <bool kBf16, bool kGated, bool kPlaces>
__global__ void __launch_bounds__(kQuantWarps * 32, kQuantCtas)
    quantize_rows_kernel(const QuantizeRowsArgs a, int steps) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    int live = a.M;
    if (a.num_rows != nullptr) {
        const int n = __ldcg(a.num_rows);
        live = n < live ? n : live;
    }
    const unsigned warps = gridDim.x * kQuantWarps;
    const unsigned first = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
    // (row, step of the row) of a job, stepped without divisions
    const int dm = static_cast<int>(warps / static_cast<unsigned>(steps));
    const int ds = static_cast<int>(warps - static_cast<unsigned>(dm) * steps);
    int m = static_cast<int>(first / static_cast<unsigned>(steps));
    int s = static_cast<int>(first - static_cast<unsigned>(m) * steps);
    const int places = kPlaces ? a.top_k : 1;
    uint4 w[2], w2[2];
    int place;   // lane j holds the row's j-th place (out of range: none)
    auto fetch = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = w2[h] = make_uint4(0u, 0u, 0u, 0u);
        place = -1;
        if (m >= live) return;
        const int k0 = s * 512 + lane * 16;
        const uint16_t* x = static_cast<const uint16_t*>(a.X) + m * a.ldx + k0;
        if (k0 < a.K) {   // K is a multiple of 16: all of them or none
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h] = reinterpret_cast<const uint4*>(x)[h];
                if (kGated) w2[h] = reinterpret_cast<const uint4*>(x + a.K)[h];
            }
        }
        if (!kPlaces) place = m;
        else if (lane < places) place = __ldcg(a.rows + static_cast<int64_t>(m) * places + lane);
    };
    fetch();
    while (m < live) {
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            widen8<kBf16>(w[h], v[h]);
            if (kGated) {
                float u[8];
                widen8<kBf16>(w2[h], u);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[h][i] = gate(v[h][i], u[i]);
            }
        }
        const int k0 = s * 512 + lane * 16;
        const int to = place < a.out_rows ? place : -1;
        m += dm;
        s += ds;
        if (s >= steps) {
            s -= steps;
            ++m;
        }
        fetch();
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(v[0][i]), fabsf(v[1][i])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float sc = quotient(amax, 448.0f, 1.0f / 448.0f);
        if (!(amax > 0.0f)) sc = 1.0f;   // blocks of zeros, and those past K
        if (sc > 1e-30f) {
            const float r = __frcp_rn(sc);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = quotient(v[i >> 3][i & 7], sc, r);
        } else {   // a reciprocal or a remainder would not be a normal number
            sc = __fdiv_rn(amax, 448.0f);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = __fdiv_rn(v[i >> 3][i & 7], sc);
        }
        const uint4 codes =
            make_uint4(codes4(v[0][0], v[0][1], v[0][2], v[0][3]), codes4(v[0][4], v[0][5], v[0][6], v[0][7]),
                       codes4(v[1][0], v[1][1], v[1][2], v[1][3]), codes4(v[1][4], v[1][5], v[1][6], v[1][7]));
        uint8_t* q = a.Xq + k0;
        float* scale = a.Sx + (k0 >> 7) * a.ldsx;
        const bool in = k0 < a.K;
        if constexpr (!kPlaces) {
            if (in && to >= 0) *reinterpret_cast<uint4*>(q + to * a.ldxq) = codes;
            if (in && to >= 0 && (lane & 7) == 0) scale[to] = sc;
        } else {
            // four places at a time; the scale of a block by its eight lanes, a place each
#pragma unroll 1
            for (int j0 = 0; j0 < places; j0 += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = __shfl_sync(0xffffffffu, to, j0 + j);   // -1 from `places` on
                    if (in && r >= 0) *reinterpret_cast<uint4*>(q + r * a.ldxq) = codes;
                }
            }
#pragma unroll 1
            for (int j0 = 0; j0 < places; j0 += 8) {
                const int r = __shfl_sync(0xffffffffu, to, j0 + (lane & 7));
                // of a block that is there (its first column decides)
                if ((k0 & ~127) < a.K && r >= 0) scale[r] = sc;
            }
        }
    }
}

template <bool kBf16>
cudaError_t launch_quantize_type(const cudaLaunchConfig_t& cfg, const QuantizeRowsArgs& a, int steps) {
    if (a.gated)
        return a.rows != nullptr ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<kBf16, true, true>, a, steps)
                                 : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<kBf16, true, false>, a, steps);
    return a.rows != nullptr ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<kBf16, false, true>, a, steps)
                             : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<kBf16, false, false>, a, steps);
}

// ----------------------------------------------------------------- combination
// A thread takes eight neighbouring columns of a token (one where the tensors
// do not allow vectors) and sums them over the token's experts in their order.
// Bound by memory.
__device__ __forceinline__ uint4 load16(const void* p, int64_t byte) {
    return *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + byte);
}
// The same where `there`, else zeros.  Volatile, so that the compiler leaves a
// batch of them in front of the first use (with branches around plain loads it
// waited for each: 374 us for 8191 x 8 x 5120).
__device__ __forceinline__ uint4 load16_if(bool there, const void* p, int64_t byte) {
    uint4 v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                 "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                 "@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
                 : "l"(static_cast<const uint8_t*>(p) + byte), "r"(static_cast<uint32_t>(there))
                 : "memory");
    return v;
}
__device__ __forceinline__ void widen8(const uint4& a, const uint4& b, float (&x)[8]) {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
}
template <int kType>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if (kType == QG_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A CTA takes a part of one token's columns.  The rows' loads are all on their way
// before the first is used: eight experts' at a time, without branches between
// them (a row that is not there is not read, and counts as zeros).  8191 x 8 x 5120:
// 111 us, the copy rate (6.8 TB/s).
constexpr int kCombineThreads = 320;

template <int kType, bool kVec>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs a, int parts) {
    constexpr int kW = kVec ? 8 : 1;
    constexpr int kLoads = kVec && kType == QG_FP32 ? 2 : 1;   // 16-byte loads of a thread's columns
    grid_dependents_launch();
    grid_dependency_wait();
    const int m = static_cast<int>(blockIdx.x / static_cast<unsigned>(parts));
    const int part = static_cast<int>(blockIdx.x - static_cast<unsigned>(m) * parts);
    const int k0 = (part * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * kW;
    if (k0 >= a.K) return;
    const int32_t* rows = a.rows + static_cast<int64_t>(m) * a.top_k;
    const float* weights = a.weights + static_cast<int64_t>(m) * a.top_k;
    float acc[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
        float w[8];
        int r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = j0 + j < a.top_k;
            r[j] = in ? rows[j0 + j] : -1;
            w[j] = in ? weights[j0 + j] : 0.0f;
        }
        uint4 raw[8][kLoads];
        float one[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool there = r[j] >= 0 && r[j] < a.R;
            const int64_t at = (there ? r[j] : 0) * a.ldy + k0;
            if constexpr (kVec) {
#pragma unroll
                for (int l = 0; l < kLoads; ++l)
                    raw[j][l] = load16_if(there, a.Y, at * (kType == QG_FP32 ? 4 : 2) + 16 * l);
            } else {
                one[j] = there ? to_f32<kType>(a.Y, at) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (kVec) {
                float x[8];
                if constexpr (kType == QG_FP32) widen8(raw[j][0], raw[j][1], x);
                else widen8<kType == QG_BF16>(raw[j][0], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(w[j], x[i], acc[i]);   // a weight of NaN shows all the same
            } else {
                acc[0] = __fmaf_rn(w[j], one[j], acc[0]);
            }
        }
    }
    if (a.residual != nullptr) {
        const int64_t at = m * a.ldr + k0;
        if constexpr (kVec) {
            float x[8];
            if constexpr (kType == QG_FP32) widen8(load16(a.residual, at * 4), load16(a.residual, at * 4 + 16), x);
            else widen8<kType == QG_BF16>(load16(a.residual, at * 2), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += x[i];
        } else {
            acc[0] += to_f32<kType>(a.residual, at);
        }
    }
    const int64_t at = m * a.ldo + k0;
    if constexpr (kVec) {
        if constexpr (kType == QG_FP32) {
            float* o = static_cast<float*>(a.out) + at;
            *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint4(narrow2<kType>(acc[0], acc[1]), narrow2<kType>(acc[2], acc[3]),
                           narrow2<kType>(acc[4], acc[5]), narrow2<kType>(acc[6], acc[7]));
        }
    } else if constexpr (kType == QG_FP32) {
        static_cast<float*>(a.out)[at] = acc[0];
    } else {
        static_cast<uint16_t*>(a.out)[at] = static_cast<uint16_t>(narrow2<kType>(acc[0], 0.0f));
    }
}

template <int kType>
cudaError_t launch_combine_type(const CombineArgs& a, cudaStream_t st) {
    const int size = kType == QG_FP32 ? 4 : 2;
    auto fits = [&](const void* p, int64_t ld) { return p == nullptr || (aligned_16(p) && ld * size % 16 == 0); };
    const bool vec = a.K % 8 == 0 && fits(a.Y, a.ldy) && fits(a.out, a.ldo) && fits(a.residual, a.ldr);
    const int pieces = vec ? a.K / 8 : a.K;
    // equal parts of a row, in whole warps
    const int parts = (pieces + kCombineThreads - 1) / kCombineThreads;
    const int threads = ((pieces + parts - 1) / parts + 31) / 32 * 32;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(static_cast<int64_t>(a.M) * parts),
                                          static_cast<unsigned>(threads), 0, st, &attr);
    if (vec) return cudaLaunchKernelEx(&cfg, combine_kernel<kType, true>, a, parts);
    return cudaLaunchKernelEx(&cfg, combine_kernel<kType, false>, a, parts);
}

}  // namespace

size_t route_workspace_bytes(int M, int E, int sms) {
    const int ctas = route_ctas(M, E, sms);
    return ctas > 1 ? static_cast<size_t>(ctas) * route_pitch(E) * sizeof(uint16_t) : 0;
}

cudaError_t launch_route(const RouteArgs& a, const LaunchCtl& c, cudaStream_t st) {
    switch (a.type) {
        case QG_BF16: return launch_route_type<QG_BF16>(a, c, st);
        case QG_FP16: return launch_route_type<QG_FP16>(a, c, st);
        case QG_FP32: return launch_route_type<QG_FP32>(a, c, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_quantize_rows(const QuantizeRowsArgs& a, const LaunchCtl& c, cudaStream_t st) {
    const int steps = (a.K + 511) / 512;   // of a row
    const int64_t jobs = static_cast<int64_t>(a.M) * steps;
    const int64_t most = static_cast<int64_t>(c.num_sms) * kQuantCtas;
    const int64_t blocks = (jobs + kQuantWarps - 1) / kQuantWarps;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        config(static_cast<unsigned>(blocks < most ? blocks : most), kQuantWarps * 32, 0, st, &attr);
    return a.x_type == QG_BF16 ? launch_quantize_type<true>(cfg, a, steps) : launch_quantize_type<false>(cfg, a, steps);
}

cudaError_t launch_combine(const CombineArgs& a, const LaunchCtl& c, cudaStream_t st) {
    switch (a.type) {
        case QG_BF16: return launch_combine_type<QG_BF16>(a, st);
        case QG_FP16: return launch_combine_type<QG_FP16>(a, st);
        case QG_FP32: return launch_combine_type<QG_FP32>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace qg
