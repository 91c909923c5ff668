// Verification of drafted tokens against the target's probabilities, for sm_103a.
//
// With p_j the softmax of the target's row j and q_j that of the draft's row
// (a certain draft: 1 at the drafted token), the drafts d_0, d_1, ... of a
// sequence are kept in order while u_j q_j(d_j) < p_j(d_j).  At the first one that
// is not kept (row n) the token is drawn from max(p_n - q_n, 0), behind the last
// one from p_n: the largest weight[v] / noise[v] with exponential random noise,
// which draws v with probability weight[v] / sum.  (A race needs no sum of the
// weights and no ordered scan over the vocabulary, and two implementations draw
// the same token unless the two largest ratios are as close as their rounding.)
// Greedy: drafts are kept while they are the target's largest logit, and the
// last token is that of row n.
//
// A cluster of CTAs takes a sequence, each CTA a slice of the vocabulary:
//   1. over all rows, one pass: the sum of exponentials of the slice about a
//      reference (greedy: the largest logit and its index), a warp at a time on a
//      stretch of a row; the CTAs' parts are read through distributed shared
//      memory by all of them, so that each knows n;
//   2. the race over the slice of row n, read again (from L2 for few sequences, from
//      HBM for many: of 64 x 6 x 131072 the 67 MB of the race, 1 % of them hits);
//   3. the first CTA compares the winners.
// With many sequences the pass over the rows is a kernel of its own, in front: the
// clusters that a sequence's rows would need leave SMs idle (of eight CTAs, 120 to
// 128 of 152 are used), and one grid of warps over all stretches does not.
//
// All sums have a fixed order.  Bound by memory: every logit is read once, and two
// rows of a sequence a second time with the noise.  64 x 6 rows of 131072 with their
// drafts: 45.7 us, of them 27 the pass over the rows (152 MB of BF16, a third of the
// sequences with fewer drafts: 5.6 TB/s under exponentials), 13 the race (67 MB), the rest the clusters'
// start and the joins; 1 x 5 x 32768: 9.7 us, latency.
//
// The sums: with L = log2 e and c a whole number that follows the largest x L from
// below (by at most 32), s = sum 2^(x L - c): a term is one fma with one rounding,
// one ex2 and one addition, and c moves only when a term would pass 2^32, so that
// no maximum is carried along.  Where c is no exact number near x L (beyond
// 2^23: logits of +-6e6, among them rows of a type's lowest value) or nothing is
// left, the row is done again about its maximum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qg_launch.h"
#include "qg_pair.cuh"
#include "qg_verify.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int kWarps = kThreads / 32;
constexpr int kMostRows = 2 * QG_MAX_DRAFTS + 1;
constexpr int kMostCtas = 16;
constexpr int kParts = 8;          // stretches of a row's slice, at most
constexpr float kLog2e = 1.4426950408889634f;

template <int kType>
struct Elem;
template <>
struct Elem<QG_BF16> {
    static constexpr int kSize = 2;
    static constexpr uint32_t kLowest = 0xFF80FF80u;   // -inf in every place
    static __device__ __forceinline__ float at(const void* p, int64_t i) {
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    }
    static __device__ __forceinline__ void wide(uint32_t w, float* x) {
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xFFFF0000u);
    }
    // eight values as they lie in memory (at a multiple of 16 bytes)
    struct Raw8 {
        uint4 a;
    };
    static __device__ __forceinline__ Raw8 load8(const void* p, int64_t i) {
        return Raw8{*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i)};
    }
    static __device__ __forceinline__ void wide8(const Raw8& r, float (&x)[8]) {
        wide(r.a.x, x), wide(r.a.y, x + 2), wide(r.a.z, x + 4), wide(r.a.w, x + 6);
    }
};
template <>
struct Elem<QG_FP16> {
    static constexpr int kSize = 2;
    static constexpr uint32_t kLowest = 0xFC00FC00u;   // -inf in every place
    static __device__ __forceinline__ float at(const void* p, int64_t i) {
        return __half2float(static_cast<const __half*>(p)[i]);
    }
    static __device__ __forceinline__ void wide(uint32_t w, float* x) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        x[0] = f.x;
        x[1] = f.y;
    }
    // eight values as they lie in memory (at a multiple of 16 bytes)
    struct Raw8 {
        uint4 a;
    };
    static __device__ __forceinline__ Raw8 load8(const void* p, int64_t i) {
        return Raw8{*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i)};
    }
    static __device__ __forceinline__ void wide8(const Raw8& r, float (&x)[8]) {
        wide(r.a.x, x), wide(r.a.y, x + 2), wide(r.a.z, x + 4), wide(r.a.w, x + 6);
    }
};
template <>
struct Elem<QG_FP32> {
    static constexpr int kSize = 4;
    static constexpr uint32_t kLowest = 0xFF800000u;   // -inf in every place
    static __device__ __forceinline__ float at(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ void wide(uint32_t w, float* x) { x[0] = __uint_as_float(w); }
    struct Raw8 {
        uint4 a, b;
    };
    static __device__ __forceinline__ Raw8 load8(const void* p, int64_t i) {
        const uint4* w = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        return Raw8{w[0], w[1]};
    }
    static __device__ __forceinline__ void wide8(const Raw8& r, float (&x)[8]) {
        const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    }
};

__device__ __forceinline__ float ex2(float t) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));   // below 2^-126: 0
    return e;
}

__device__ __forceinline__ float lg2(float t) {
    float l;
    asm("lg2.approx.f32 %0, %1;" : "=f"(l) : "f"(t));
    return l;
}

// e^d for d <= 0, with the product's rounding carried along: within 2^-22 of it
// at any distance from the maximum (a rounded d log2 e alone costs |d| 2^-24).
__device__ __forceinline__ float exp_near(float d) {
    const float t = __fmul_rn(d, kLog2e);
    const float lo = __fmaf_rn(d, kLog2e, -t) + d * 1.925963033e-8f;   // the product's rest, and log2 e's
    const float e = ex2(t);
    return d > -150.0f ? __fmaf_rn(e, lo * 0.6931471806f, e) : 0.0f;
}

// A part of a row: its maximum and sum of exponentials about it; greedy: the
// maximum and its first index (as bits).
struct Part {
    float m, s;
};

// Exact zero for s where nothing is left; NaN and +inf spread to s.
__device__ __forceinline__ Part join(Part a, Part b) {
    const float m = fmaxf(a.m, b.m);
    const float s = (a.m > -INFINITY ? a.s * ex2((a.m - m) * kLog2e) : a.s) +
                    (b.m > -INFINITY ? b.s * ex2((b.m - m) * kLog2e) : b.s);
    return Part{m, s};
}
__device__ __forceinline__ Part join_greedy(Part a, Part b) {
    const bool second = b.m > a.m || (b.m == a.m && __float_as_uint(b.s) < __float_as_uint(a.s));
    return second ? b : a;
}

// One value into a running part (greedy).
__device__ __forceinline__ void see_greedy(Part& p, float x, int v) {
    if (x > p.m) {   // indices ascend in a lane, so the first stays
        p.m = x;
        p.s = __uint_as_float(static_cast<uint32_t>(v));
    }
}

template <int kCount>
__device__ __forceinline__ void see(Part& p, const float (&x)[kCount]) {
    float m = p.m;
#pragma unroll
    for (int i = 0; i < kCount; ++i) m = fmaxf(m, x[i]);
    float s = p.m > -INFINITY ? p.s * ex2((p.m - m) * kLog2e) : p.s;
    const float c = m > -INFINITY ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < kCount; ++i) s += ex2((x[i] - c) * kLog2e);
    p.m = m;
    p.s = s;
}

// A part of a row about c: s = sum 2^(x L - c).
constexpr float kNoRef = -1e30f;      // nothing seen
constexpr float kMostRef = 8388608.0f;
struct Sum {
    float c, s;
};
__device__ __forceinline__ Sum join(Sum a, Sum b) {
    const float c = fmaxf(a.c, b.c);
    return Sum{c, a.s * ex2(a.c - c) + b.s * ex2(b.c - c)};
}
template <int kCount>
__device__ __forceinline__ void see(Sum& p, const float (&x)[kCount]) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < kCount; ++i) m = fmaxf(m, x[i]);
    if (m * kLog2e > p.c + 32.0f) {
        const float c = ceilf(m * kLog2e);
        p.s *= ex2(p.c - c);
        p.c = c;
    }
    if constexpr (kCount == 1) {
        p.s += ex2(__fmaf_rn(x[0], kLog2e, -p.c));
    } else {   // two terms an instruction: the pass is bound by what it issues
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kCount; i += 2) {
            float t0, t1;
            asm("{\n\t.reg .b64 v, l, c, t;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 l, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
                "fma.rn.f32x2 t, v, l, c;\n\tmov.b64 {%0, %1}, t;\n\t}"
                : "=f"(t0), "=f"(t1)
                : "f"(x[i]), "f"(x[i + 1]), "f"(kLog2e), "f"(-p.c));
            t0 = ex2(t0);
            t1 = ex2(t1);
            asm("{\n\t.reg .b64 a, t;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tadd.rn.f32x2 a, a, t;\n\t"
                "mov.b64 {%0, %1}, a;\n\t}"
                : "+f"(s0), "+f"(s1)
                : "f"(t0), "f"(t1));
        }
        p.s += s0 + s1;
    }
}
// The same about the maximum m' = c ln 2 (rounded): s' = s 2^(c - m' L).
__device__ __forceinline__ Part about_max(Sum a) {
    const float m = a.c * 0.6931471806f;
    return Part{m, a.s * ex2(-__fmaf_rn(m, kLog2e, -a.c))};
}

constexpr int kSum = 0, kMax = 1, kGreedyScan = 2;   // kMax: about the maximum
// Sixteen bytes of a row, the elements from v on.
template <int kType, int kHow, class State>
__device__ __forceinline__ void take(State& p, const uint4& w, int v) {
    using El = Elem<kType>;
    constexpr int kVec = 16 / El::kSize;
    float x[kVec];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) El::wide(ws[e], x + e * (kVec / 4));
    if constexpr (kHow == kGreedyScan) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) see_greedy(p, x[e], v + e);
    } else {
        see(p, x);
    }
}

// The slice [v0, v1) of a row, by one warp: scalars up to the first 16-byte
// boundary and behind the last, vectors in between, four and the scalars on their way
// at a time.
template <int kType, int kHow, class State>
__device__ __forceinline__ State scan_row(const void* row, int v0, int v1, int lane, State p) {
    using El = Elem<kType>;
    constexpr int kVec = 16 / El::kSize;
    const uint8_t* base = static_cast<const uint8_t*>(row);
    const uintptr_t first = reinterpret_cast<uintptr_t>(base) + static_cast<int64_t>(v0) * El::kSize;
    const int head = static_cast<int>(((16 - (first & 15u)) & 15u) / El::kSize);
    const int a0 = v0 + head < v1 ? v0 + head : v1;
    const int nvec = (v1 - a0) / kVec;
    const int a1 = a0 + nvec * kVec;
    float front[1] = {-INFINITY}, back[1] = {-INFINITY};   // adds nothing
    if (v0 + lane < a0) front[0] = El::at(row, v0 + lane);
    if (a1 + lane < v1) back[0] = El::at(row, a1 + lane);
    const uint4* vec = reinterpret_cast<const uint4*>(base + static_cast<int64_t>(a0) * El::kSize) + lane;
    constexpr int kU = 4;
    for (int i = 0; i < nvec || i == 0; i += 32 * kU) {
        uint4 w[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            w[u] = make_uint4(El::kLowest, El::kLowest, El::kLowest, El::kLowest);
            if (i + 32 * u + lane < nvec) w[u] = __ldcg(vec + i + 32 * u);
        }
        if (i == 0 && a0 > v0) {
            if constexpr (kHow == kGreedyScan) see_greedy(p, front[0], v0 + lane);
            else see(p, front);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) take<kType, kHow>(p, w[u], a0 + (i + 32 * u + lane) * kVec);
    }
    if (a1 < v1) {
        if constexpr (kHow == kGreedyScan) see_greedy(p, back[0], a1 + lane);
        else see(p, back);
    }
    return p;
}
// Of all lanes.
__device__ __forceinline__ Sum warp_join(Sum p) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        p = join(p, Sum{__shfl_xor_sync(0xffffffffu, p.c, o), __shfl_xor_sync(0xffffffffu, p.s, o)});
    return p;
}
template <bool kGreedy>
__device__ __forceinline__ Part warp_join(Part p) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Part q{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o)};
        p = kGreedy ? join_greedy(p, q) : join(p, q);
    }
    return p;
}
template <int kType>
__device__ __forceinline__ Sum scan_sum(const void* row, int v0, int v1, int lane) {
    return warp_join(scan_row<kType, kSum>(row, v0, v1, lane, Sum{kNoRef, 0.0f}));
}
__device__ __forceinline__ int length_of(const VerifyArgs& a, int b) {
    if (a.lengths == nullptr) return a.G;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.G ? a.G : n;
}

template <int kType, bool kGreedy>
__device__ __forceinline__ Part scan_max(const void* row, int v0, int v1, int lane) {
    return warp_join<kGreedy>(scan_row<kType, kGreedy ? kGreedyScan : kMax>(
        row, v0, v1, lane, Part{-INFINITY, kGreedy ? __uint_as_float(0x7FFFFFFFu) : 0.0f}));
}

__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(smem_u32(p), rank)) : "memory");
    return v;
}

// A candidate of the race: the larger ratio, then the lower index.
struct Best {
    float ratio;
    int v;
};
__device__ __forceinline__ Best better(Best a, Best b) {
    return b.ratio > a.ratio || (b.ratio == a.ratio && b.v < a.v) ? b : a;
}

// Stretches of this many elements are a warp's work where the rows have a kernel of
// their own.
constexpr int kStretch = 2048;
inline int verify_stretches(int V) { return (V + kStretch - 1) / kStretch; }

// The parts of all rows by stretch: parts[(b (2 G + 1) + r) stretches + i].  Warps walk
// over the stretches, the loads of the next four vectors (of the next stretch) on
// their way while four are summed, and while a stretch's lanes are joined.
template <int kType, bool kGreedy>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_rows_kernel(const VerifyArgs a, int stretches, float2* out) {
    using El = Elem<kType>;
    using State = std::conditional_t<kGreedy, Part, Sum>;
    constexpr int kHow = kGreedy ? kGreedyScan : kSum;
    constexpr int kVec = 16 / El::kSize;
    constexpr int kU = 4;
    constexpr int kTurns = kStretch / (32 * kVec * kU);
    static_assert(kTurns * 32 * kVec * kU == kStretch, "whole turns");
    grid_dependents_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const bool sampled = !kGreedy && a.draft != nullptr;
    const int most = sampled ? 2 * a.G + 1 : a.G + 1;   // rows of a sequence
    const int rows = a.B * most;
    const int warps = gridDim.x * kWarps, first = blockIdx.x * kWarps + (threadIdx.x >> 5);
    // the next stretch, stepped without divisions
    const int drow = warps / stretches, dpiece = warps - drow * stretches;
    int row = first / stretches, piece = first - row * stretches;
    auto step = [&]() {
        row += drow;
        piece += dpiece;
        if (piece >= stretches) {
            piece -= stretches;
            ++row;
        }
    };
    // an open stretch: its row, place and part
    const uint8_t* p = nullptr;
    int s0 = 0;
    float2* to = nullptr;
    bool whole = false;   // in whole vectors, all there
    uint4 w[kU];
    auto load = [&](int turn, uint4 (&x)[kU]) {
        const uint4* vec = reinterpret_cast<const uint4*>(p + static_cast<int64_t>(s0) * El::kSize) + turn * 32 * kU + lane;
#pragma unroll
        for (int u = 0; u < kU; ++u) x[u] = __ldcg(vec + 32 * u);
    };
    auto open = [&](uint4 (&x)[kU]) {   // the next one that counts, from (row, piece) on
        for (; row < rows; step()) {
            const int b = row / most, r = row - b * most;
            const int length = length_of(a, b);
            const bool of_target = r <= a.G;
            if (of_target ? r > length : r - (a.G + 1) >= length) continue;
            p = of_target ? static_cast<const uint8_t*>(a.target) + (b * a.t_seq + r * a.t_row) * El::kSize
                          : static_cast<const uint8_t*>(a.draft) + (b * a.d_seq + (r - a.G - 1) * a.d_row) * El::kSize;
            s0 = piece * kStretch;
            to = out + (static_cast<int64_t>(b) * (2 * a.G + 1) + r) * stretches + piece;
            whole = a.V - s0 >= kStretch && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
            if (whole) load(0, x);
            step();
            return true;
        }
        return false;
    };
    auto none = [] {
        if constexpr (kGreedy) return Part{-INFINITY, __uint_as_float(0x7FFFFFFFu)};
        else return Sum{kNoRef, 0.0f};
    };
    bool there = open(w);
    while (there) {
        float2* const at = to;
        State sum = none();
        if (whole) {
            const int v = s0 + lane * kVec;
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
                uint4 x[kU];
                if (t + 1 < kTurns) load(t + 1, x);
                else there = open(x);
#pragma unroll
                for (int u = 0; u < kU; ++u) take<kType, kHow>(sum, w[u], v + (t * kU + u) * 32 * kVec);
#pragma unroll
                for (int u = 0; u < kU; ++u) w[u] = x[u];
            }
        } else {
            sum = scan_row<kType, kHow>(p, s0, a.V - s0 < kStretch ? a.V : s0 + kStretch, lane, sum);
            there = open(w);
        }
        float2 part;
        if constexpr (kGreedy) {
            sum = warp_join<true>(sum);
            part = make_float2(sum.m, sum.s);
        } else {
            sum = warp_join(sum);
            part = make_float2(sum.c, sum.s);
        }
        if (lane == 0) *at = part;
    }
}

// kApart: the rows' parts come from verify_rows_kernel.
template <int kType, bool kGreedy, bool kApart>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    verify_kernel(const VerifyArgs a, int ctas, int stretches, const float2* given) {
    using El = Elem<kType>;
    __shared__ Part parts[kMostRows][kParts];
    __shared__ Part mine[kMostRows];        // this CTA's slice
    __shared__ Part all[kMostRows];         // the whole rows
    __shared__ Best best[kWarps];
    __shared__ Best winner, winner_p;       // of max(p - q, 0), or of p
    __shared__ int kept, odd_rows;
    grid_dependents_launch();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = blockIdx.x % ctas;
    const int b = blockIdx.x / ctas;
    const bool sampled = !kGreedy && a.draft != nullptr;
    const int length = length_of(a, b);
    // rows 0 .. length of the target, then 0 .. length - 1 of the draft
    const int trows = length + 1;
    const int rows = trows + (sampled ? length : 0);
    auto row_at = [&](int r) -> const void* {
        const uint8_t* p = r < trows ? static_cast<const uint8_t*>(a.target) + (b * a.t_seq + r * a.t_row) * El::kSize
                                     : static_cast<const uint8_t*>(a.draft) + (b * a.d_seq + (r - trows) * a.d_row) * El::kSize;
        return p;
    };
    // slices and stretches end at multiples of 32 elements, so that rows that
    // are aligned stay so
    auto cut = [](int64_t n, int i, int of) { return static_cast<int>((n + 31) / 32 * i / of * 32); };
    const int v0 = cut(a.V, rank, ctas);
    int v1 = cut(a.V, rank + 1, ctas);
    if (v1 > a.V) v1 = a.V;
    const int slice = v1 - v0;
    // Stretches of a row: a warp's costs one turn of loads, and one more for each 1024
    // elements; as many to a row as take the warps the least.
    int pieces = 1;
    for (int n = 2, least = (rows + kWarps - 1) / kWarps * (1 + (slice + 1023) / 1024); n <= kParts; n *= 2) {
        const int cost = (rows * n + kWarps - 1) / kWarps * (1 + (slice / n + 1023) / 1024);
        if (cost < least) {
            least = cost;
            pieces = n;
        }
    }
    auto stretch = [&](int i, int& r, int& piece, int& s0, int& s1) {
        r = i / pieces;
        piece = i - r * pieces;
        s0 = v0 + cut(slice, piece, pieces);
        s1 = v0 + cut(slice, piece + 1, pieces);
        if (s1 > v1) s1 = v1;
    };
    // the CTAs' parts of a row, in their order
    auto of_all = [&](int r, auto joined) {
        Part p = ctas > 1 ? Part{ld_cluster(&mine[r].m, 0), ld_cluster(&mine[r].s, 0)} : mine[r];
        for (int c = 1; c < ctas; ++c)
            p = joined(p, Part{ld_cluster(&mine[r].m, static_cast<uint32_t>(c)), ld_cluster(&mine[r].s, static_cast<uint32_t>(c))});
        return p;
    };
    auto join_sums = [](Part a, Part b) {
        const Sum s = join(Sum{a.m, a.s}, Sum{b.m, b.s});
        return Part{s.c, s.s};
    };
    auto join_maxima = [](Part a, Part b) { return kGreedy ? join_greedy(a, b) : join(a, b); };
    if (threadIdx.x == 0) odd_rows = 0;
    // the whole row's sums (greedy: its maximum) from all parts
    auto enter_row = [&](int r, Part p) {
        if constexpr (kGreedy) {
            all[r] = p;
        } else {
            const bool fine = fabsf(p.m) <= kMostRef && p.s < INFINITY;
            all[r] = fine ? about_max(Sum{p.m, p.s}) : Part{0.0f, -1.0f};
            if (!fine) atomicOr(&odd_rows, 1);
        }
    };
    if constexpr (kApart) {
        __syncthreads();   // odd_rows
        for (int r = warp; r < rows; r += kWarps) {
            const int at = r < trows ? r : a.G + 1 + r - trows;
            const float2* from = given + (static_cast<int64_t>(b) * (2 * a.G + 1) + at) * stretches;
            Part p{kGreedy ? -INFINITY : kNoRef, kGreedy ? __uint_as_float(0x7FFFFFFFu) : 0.0f};
            for (int i = lane; i < stretches; i += 32) {
                const float2 v = __ldcg(from + i);
                p = kGreedy ? join_greedy(p, Part{v.x, v.y}) : join_sums(p, Part{v.x, v.y});
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const Part q{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o)};
                p = kGreedy ? join_greedy(p, q) : join_sums(p, q);
            }
            if (lane == 0) enter_row(r, p);
        }
    } else {
        for (int i = warp; i < rows * pieces; i += kWarps) {
            int r, piece, s0, s1;
            stretch(i, r, piece, s0, s1);
            Part p;
            if constexpr (kGreedy) {
                p = scan_max<kType, true>(row_at(r), s0, s1, lane);
            } else {
                const Sum q = scan_sum<kType>(row_at(r), s0, s1, lane);
                p = Part{q.c, q.s};
            }
            if (lane == 0) parts[r][piece] = p;
        }
        __syncthreads();
        for (int r = threadIdx.x; r < rows; r += kThreads) {
            Part p = parts[r][0];
            for (int i = 1; i < pieces; ++i) p = kGreedy ? join_greedy(p, parts[r][i]) : join_sums(p, parts[r][i]);
            mine[r] = p;
        }
        __syncthreads();
        cluster_sync_all();
        for (int r = threadIdx.x; r < rows; r += kThreads) {
            if constexpr (kGreedy) enter_row(r, of_all(r, join_maxima));
            else enter_row(r, of_all(r, join_sums));
        }
    }
    __syncthreads();
    if constexpr (!kGreedy) {
        if (odd_rows) {   // the same in all CTAs of the cluster
            cluster_sync_all();   // every part has been read
            for (int i = warp; i < rows * pieces; i += kWarps) {
                int r, piece, s0, s1;
                stretch(i, r, piece, s0, s1);
                if (all[r].s >= 0.0f) continue;
                const Part p = scan_max<kType, false>(row_at(r), s0, s1, lane);
                if (lane == 0) parts[r][piece] = p;
            }
            __syncthreads();
            for (int r = threadIdx.x; r < rows; r += kThreads) {
                if (all[r].s >= 0.0f) continue;
                Part p = parts[r][0];
                for (int i = 1; i < pieces; ++i) p = join(p, parts[r][i]);
                mine[r] = p;
            }
            __syncthreads();
            cluster_sync_all();
            for (int r = threadIdx.x; r < rows; r += kThreads)
                if (!(all[r].s >= 0.0f)) all[r] = of_all(r, join_maxima);
            __syncthreads();
        }
    }
    // which drafts are kept: a lane a draft
    if (warp == 0) {
        bool keep = false;
        if (lane < length) {
            const int64_t d = a.tokens[b * a.ldt + lane];
            if constexpr (kGreedy) {
                keep = d == static_cast<int64_t>(__float_as_uint(all[lane].s)) && all[lane].m > -INFINITY;
            } else if (d >= 0 && d < a.V) {
                const Part t = all[lane];
                const float p = exp_near(El::at(row_at(lane), d) - t.m) / t.s;
                float q = 1.0f;
                if (sampled) {
                    const Part s = all[trows + lane];
                    q = exp_near(El::at(row_at(trows + lane), d) - s.m) / s.s;
                }
                keep = a.uniform[b * a.ldu + lane] * q < p;
            }
        }
        const uint32_t not_kept = ~__ballot_sync(0xffffffffu, keep);
        const int n = not_kept == 0u ? 32 : __ffs(static_cast<int>(not_kept)) - 1;   // the first draft that is not kept
        if (lane == 0) kept = n;
    }
    __syncthreads();
    const int n = kept;
    int64_t last = -1;   // the token that follows
    if constexpr (!kGreedy) {
        const Part t = all[n];
        const void* trow = row_at(n);
        const bool drafted = n < length;
        const Part s = drafted && sampled ? all[trows + n] : Part{0.0f, 1.0f};
        const void* drow = drafted && sampled ? row_at(trows + n) : nullptr;
        const int64_t d = drafted && !sampled ? a.tokens[b * a.ldt + n] : -1;   // the certain draft
        const float pr = 1.0f / t.s, qr = 1.0f / s.s;
        const float* noise = a.noise + b * a.ldn;
        // The race of max(p - q, 0), or of p (for a row where that is 0 everywhere).
        // Eight tokens a lane at a time: quick probabilities, good to kSlack of p, and
        // whether a token may reach the largest ratio that the warp has seen (w >= reach
        // noise, with the slack); if one of any lane may, the exact ratios of those
        // that may.  Few turns of a warp have any.  (Bounds of every ratio by a
        // reciprocal, and the largest of them every turn: 49.8 us for 64 x 6 x 131072
        // against 46.5.)
        //   kSlack: the exact probability has the same x - m.  Against it the quick one's
        // exponent t = fma(x - m, L, -log2 s), |t| <= 126, is off by its rounding (2^-18), by
        // L's (|x - m| <= 110: 2.1e-6) and by log2 s's (2^-19): with the ex2 and the exact
        // one's rest 6e-6 as a factor, of p and of a q below p.  kTiny: below 2^-126 a
        // quick probability is 0.
        constexpr float kSlack = 2e-5f, kTiny = 0x1p-120f;
        const float tl = -lg2(t.s), sl = -lg2(s.s);
        auto race = [&](bool with_q, Best& result) {
            Best top{0.0f, 0x7FFFFFFF};
            float reach = 0.0f;
            auto exact = [&](int v, float x, float y, float e) {
                const float p = exp_near(x - t.m) * pr;
                float q = 0.0f;
                if (with_q) {
                    if (drow != nullptr) q = exp_near(y - s.m) * qr;
                    else if (v == d) q = 1.0f;
                }
                const float w = p - q;
                if (w > 0.0f) {
                    const float ratio = __fdiv_rn(w, e);
                    // indices ascend in a thread, so the first of equals stays
                    if (ratio > top.ratio) top = Best{ratio, v};
                }
            };
            // tokens v, v + step, ... (one with a noise of NaN does not count)
            auto enter = [&](int v, int step, const float (&x)[8], const float (&y)[8], const float (&e)[8]) {
                float w[8], high[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = ex2(__fmaf_rn(x[j] - t.m, kLog2e, tl));
                    w[j] = p;
                    if (with_q) {
                        if (drow != nullptr) w[j] -= ex2(__fmaf_rn(y[j] - s.m, kLog2e, sl));
                        else if (v + j * step == d) w[j] -= 1.0f;
                    }
                    high[j] = __fmaf_rn(kSlack, p, w[j]);
                }
                if (reach == 0.0f) {   // at first: what some token has at least
                    float low = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float r;
                        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e[j]));
                        const float least = __fmaf_rn(2.0f, w[j], -high[j]) * r;   // w - kSlack p
                        if (r > 0.0f && r < INFINITY) low = fmaxf(low, least);
                    }
                    reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(low)));   // not negative
                }
                bool may = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) may |= high[j] >= __fmaf_rn(reach, e[j], -kTiny);
                if (__any_sync(0xffffffffu, may)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (high[j] >= __fmaf_rn(reach, e[j], -kTiny)) exact(v + j * step, x[j], y[j], e[j]);
                    reach = fmaxf(reach, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top.ratio))));
                }
            };
            constexpr int kVec = 8;
            const bool vectors = ((reinterpret_cast<uintptr_t>(trow) | reinterpret_cast<uintptr_t>(drow) |
                                   reinterpret_cast<uintptr_t>(noise)) & 15u) == 0;
            const float nan = __uint_as_float(0x7FC00000u);
            int v_done = v0;
            if (vectors) {   // slices begin at multiples of 32
                const int nvec = (v1 - v0) / kVec;
                v_done = v0 + nvec * kVec;
                for (int i0 = 32 * warp; i0 < nvec; i0 += kThreads) {
                    const bool in = i0 + lane < nvec;
                    const int v = v0 + (in ? i0 + lane : nvec - 1) * kVec;
                    float x[kVec], y[kVec], e[kVec];
                    const typename El::Raw8 xr = El::load8(trow, v);
                    const typename El::Raw8 yr = El::load8(with_q && drow != nullptr ? drow : trow, v);
                    const Elem<QG_FP32>::Raw8 er = Elem<QG_FP32>::load8(noise, v);
                    El::wide8(xr, x);
                    El::wide8(yr, y);
                    Elem<QG_FP32>::wide8(er, e);
                    if (!in) {
#pragma unroll
                        for (int j = 0; j < kVec; ++j) e[j] = nan;
                    }
                    enter(v, 1, x, y, e);
                }
            }
            for (int v = v_done + 32 * warp; v < v1; v += kThreads * kVec) {
                float x[kVec], y[kVec], e[kVec];
#pragma unroll
                for (int u = 0; u < kVec; ++u) {
                    const int at = v + lane + kThreads * u;
                    const int w = at < v1 ? at : v1 - 1;
                    x[u] = El::at(trow, w);
                    y[u] = with_q && drow != nullptr ? El::at(drow, w) : 0.0f;
                    e[u] = at < v1 ? noise[w] : nan;
                }
                enter(v + lane, kThreads, x, y, e);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = better(top, Best{__shfl_xor_sync(0xffffffffu, top.ratio, o), __shfl_xor_sync(0xffffffffu, top.v, o)});
            __syncthreads();   // `best` may still be read from the race before
            if (lane == 0) best[warp] = top;
            __syncthreads();
            if (threadIdx.x == 0) {
                Best w = best[0];
                for (int i = 1; i < kWarps; ++i) w = better(w, best[i]);
                result = w;
            }
            __syncthreads();
            cluster_sync_all();
            // of all CTAs, known to each
            Best w = result;
            if (ctas > 1 && lane < ctas) {
                w.ratio = ld_cluster(&result.ratio, static_cast<uint32_t>(lane));
                w.v = static_cast<int>(
                    __float_as_uint(ld_cluster(reinterpret_cast<const float*>(&result.v), static_cast<uint32_t>(lane))));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                w = better(w, Best{__shfl_xor_sync(0xffffffffu, w.ratio, o), __shfl_xor_sync(0xffffffffu, w.v, o)});
            return Best{__shfl_sync(0xffffffffu, w.ratio, 0), __shfl_sync(0xffffffffu, w.v, 0)};
        };
        Best w = race(drafted, winner);
        if (drafted && w.v == 0x7FFFFFFF) w = race(false, winner_p);
        if (w.v != 0x7FFFFFFF) last = w.v;
    }
    if (rank == 0) {
        if constexpr (kGreedy)
            if (all[n].m > -INFINITY) last = static_cast<int64_t>(__float_as_uint(all[n].s));
        const int j = static_cast<int>(threadIdx.x);
        if (j <= a.G) a.out[static_cast<int64_t>(b) * (a.G + 1) + j] = j < n ? a.tokens[b * a.ldt + j] : j == n ? last : -1;
        if (j == 0) a.accepted[b] = n;
    }
    cluster_sync_all();   // nobody leaves while its shared memory is read
}

template <int kType, bool kGreedy, bool kApart>
cudaError_t launch_clusters(const VerifyArgs& a, const LaunchCtl& c, cudaStream_t st) {
    static std::atomic<uint64_t> wide{0};
    cudaError_t e = set_once(wide, verify_kernel<kType, kGreedy, kApart>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    // CTAs of a sequence: as many as run at once (a power of two: clusters of 7 leave a
    // third of the SMs idle), none with less of the vocabulary than pays the larger
    // cluster: 1024, or 2048 where only the race is left.  (40 shapes, 1 to 106
    // sequences of 1182 to 159231: in the mean 10.97 us with 1024, 11.24 with 2048, 11.07
    // with 512; 29 x 20585, the race alone, 17.4 with 2048 and 20.7 with 1024.)
    constexpr int kLeast = kApart ? 2048 : 1024;
    int ctas = kMostCtas;
    while (ctas > 1 && (static_cast<int64_t>(ctas) * a.B > kCtasPerSm * c.num_sms || a.V / ctas < kLeast)) ctas /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<kType, kGreedy, kApart>, a, ctas, verify_stretches(a.V),
                              static_cast<const float2*>(a.ws));
}

template <int kType, bool kGreedy>
cudaError_t launch(const VerifyArgs& a, const LaunchCtl& c, cudaStream_t st) {
    if (verify_workspace_bytes(a.B, a.G, a.V, c.num_sms) == 0) return launch_clusters<kType, kGreedy, false>(a, c, st);
    const int stretches = verify_stretches(a.V);
    const int64_t warps = static_cast<int64_t>(a.B) * (2 * a.G + 1) * stretches;
    const int64_t most = static_cast<int64_t>(c.num_sms) * kCtasPerSm, blocks = (warps + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, verify_rows_kernel<kType, kGreedy>, a, stretches, static_cast<float2*>(a.ws));
    return e != cudaSuccess ? e : launch_clusters<kType, kGreedy, true>(a, c, st);
}

template <int kType>
cudaError_t launch_type(const VerifyArgs& a, const LaunchCtl& c, cudaStream_t st) {
    return a.uniform == nullptr ? launch<kType, true>(a, c, st) : launch<kType, false>(a, c, st);
}

}  // namespace

// 0: the clusters pass over the rows themselves (few sequences: one launch less)
size_t verify_workspace_bytes(int B, int G, int V, int sms) {
    if (static_cast<int64_t>(B) * kMostCtas <= 2 * sms || V < 4 * kStretch) return 0;
    return static_cast<size_t>(B) * (2 * G + 1) * verify_stretches(V) * sizeof(float2);
}

cudaError_t launch_verify(const VerifyArgs& a, const LaunchCtl& c, cudaStream_t st) {
    switch (a.type) {
        case QG_BF16: return launch_type<QG_BF16>(a, c, st);
        case QG_FP16: return launch_type<QG_FP16>(a, c, st);
        case QG_FP32: return launch_type<QG_FP32>(a, c, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace qg
