// Log probabilities of given tokens, entropy and top alternatives over rows of
// logits (e.g. the output of an lm_head GEMM), for sm_103a.
//
// With L = log2 e, c a whole number near (max x) L, t[v] = x[v] L - c:
//   s = sum 2^t[v],  w = sum 2^t[v] t[v]
//   ln p[v] = ln2 t[v] - ln s,   H = ln s - ln2 w / s
// all in FP32.  c is whole so that t is one fma with one rounding however far
// the row lies from zero; it moves with the running maximum, and s and w move
// with it (s' = 2^d s, w' = 2^d (w + d s) for a step d = c - c'), so one pass
// over the logits gives everything.  Logits of -inf are raised to a finite
// floor first: their 2^t is 0 and 2^t t stays 0 instead of NaN; a NaN passes
// the floor and spreads to s.
//
// The alternatives come from the same pass.  Every thread keeps the largest
// logits of up to eight stretches of its turns; the k-th largest of the maxima of
// pairs of threads is a bound that at least k logits reach, and only the
// stretches that reach it (little more than k of them) are looked at again, in
// L2.  What reaches the bound (about k (1 + k / 128) logits of a row without
// structure) is ranked by counting.  They are ordered on 64-bit keys: the value,
// then the lower index.
//
// Rows where this does not hold are worked out by the plain method at the end
// of this file's row function: a maximum beyond +-1e8 (or at the floor: a row
// of nothing but masks), a NaN or +inf, or more than kCap logits above the bound.
// (More than kCap at the bound, as where masks leave fewer tokens than are asked
// for, are filled in by index.)
//
// Five CTAs per SM walk over the rows.  One warp of a CTA streams them into a
// ring in shared memory by bulk copies, running on into the next row while the
// other four finish one (under load the end of a row takes 4 us, with nothing on
// the way from memory when each row had a CTA of its own and registers for its
// loads).  Many small CTAs, because that end is a chain of block-wide steps and
// the others' streaming hides it (three CTAs of 256 threads: 177 us for 4096 x
// 131072 BF16 and 65 for 4096 x 32768, now 158 and 53); turns of eight vectors a
// thread, because each costs a wait, a maximum and an arrival (of four, 167
// against 165 us and 57 against 53 when they were compared).  Bound by memory on
// long rows: 4096 x 131072 BF16 runs at the measured copy rate.  Rows that are too
// few for the SMs are split over a cluster of up to 16 CTAs, which store their
// sums and lists to rank 0's shared memory, where they are joined (no workspace,
// no atomics on memory, the same order of sums on every call).
#include <cstddef>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_gemm.cuh"
#include "qg_launch.h"
#include "qg_logprobs.h"
#include "qg_pair.cuh"

namespace qg {
namespace {

constexpr int kThreads = 128;      // that take logits; one more warp streams them in
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = kThreads / 2;
constexpr int kCtasPerSm = 5;
constexpr int kMostStages = 4;     // of the ring, one turn each (stages_of)
constexpr int kULg = 3;
constexpr int kU = 1 << kULg;      // 16-byte vectors a thread takes in a turn
constexpr int kTurn = kU * kThreads;
constexpr int kSegs = 8;           // stretches of a thread's turns that it keeps the maxima of
constexpr int kCap = 512;          // candidates at the bound
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = 1e8f;       // a maximum beyond this goes the plain way
constexpr float kNoRef = -3e38f;   // c before the first logit

template <int kType>
struct Fmt;   // element unpacking: kE elements in a 16-byte vector

template <>
struct Fmt<QG_FP32> {
    static constexpr int kE = 4, kSize = 4;
    static constexpr float kFloor = -1e30f;
    using Word = float;   // of one element, as loaded
    __device__ static float value(Word w) { return w; }
    __device__ static uint32_t floor_word(uint32_t w) {
        uint32_t r;
        asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(__float_as_uint(kFloor)));
        return r;
    }
    __device__ static uint32_t max_word(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ static float max_of(uint32_t w) { return __uint_as_float(w); }
    __device__ static float element(const uint32_t (&w)[4], int e) { return __uint_as_float(w[e]); }
    static constexpr uint32_t kEmpty = 0xFF800000u;   // words of -inf
};

template <>
struct Fmt<QG_BF16> {
    static constexpr int kE = 8, kSize = 2;
    static constexpr float kFloor = -0x1.94p99f;   // about -1e30: the bf16 0xF14A
    using Word = uint16_t;
    __device__ static float value(Word w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
    __device__ static uint32_t floor_word(uint32_t w) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xF14AF14Au));
        return r;
    }
    __device__ static uint32_t max_word(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ static float max_of(uint32_t w) {
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ static void unpack(uint32_t w, float& a, float& b) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xFFFF0000u);
    }
    __device__ static float element(const uint32_t (&w)[4], int e) {
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
    static constexpr uint32_t kEmpty = 0xFF80FF80u;
};

template <>
struct Fmt<QG_FP16> {
    static constexpr int kE = 8, kSize = 2;
    static constexpr float kFloor = -65504.0f;
    using Word = uint16_t;
    __device__ static float value(Word w) { return __half2float(__ushort_as_half(w)); }
    __device__ static uint32_t floor_word(uint32_t w) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xFBFFFBFFu));
        return r;
    }
    __device__ static uint32_t max_word(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ static void unpack(uint32_t w, float& a, float& b) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    }
    __device__ static float max_of(uint32_t w) {
        float a, b;
        unpack(w, a, b);
        return fmaxf(a, b);
    }
    __device__ static float element(const uint32_t (&w)[4], int e) {
        float a, b;
        unpack(w[e >> 1], a, b);
        return e & 1 ? b : a;
    }
    static constexpr uint32_t kEmpty = 0xFC00FC00u;
};

// Element v of a row, as loaded (the conversion at once would wait for the load).
template <typename F>
__device__ __forceinline__ typename F::Word word_at(const void* row, int64_t v) {
    return static_cast<const typename F::Word*>(row)[v];
}
template <typename F>
__device__ __forceinline__ float value_at(const void* row, int64_t v) {
    return F::value(word_at<F>(row, v));
}

// ----------------------------------------------------------------- small pieces
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
// (value, index) as one number: larger value first, then lower index; 0 is below every entry.
__device__ __forceinline__ uint64_t entry_of(float x, uint32_t index) {
    return static_cast<uint64_t>(order_key(x)) << 32 | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ uint32_t entry_index(uint64_t e) { return 0xFFFFFFFFu - static_cast<uint32_t>(e); }

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Stores to the shared memory of another CTA of the cluster (a mapped address).
__device__ __forceinline__ void st_peer(uint32_t to, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t to, float x, float y, float z, float w) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(x), "f"(y), "f"(z), "f"(w)
                 : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t to, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory");
}

// The reference c of logits up to `top`.  Not below that of -kFar: c is then
// within a few units of top L (its rounding is 2^-24 of it), and a thread or a
// part with nothing but masks adds 2^-huge = 0 instead of what rounding leaves.
__device__ __forceinline__ float reference_of(float top) { return ceilf(fmaxf(top, -kFar) * kLog2e); }

// Running sums of one thread (or CTA, or row): maximum, reference c, s and w.
struct Sums {
    float mx, c, s, w;
    // the same sums about a reference c2 >= c
    __device__ void move_to(float c2) {
        const float d = c - c2;
        const float f = ex2(d);
        w = f * fmaf(d, s, w);
        s = f * s;
        c = c2;
    }
};

struct alignas(16) PartSums {
    Sums sums;
    float bad;   // the part's list is not to be used
};

struct Shared {
    uint64_t full[kMostStages], empty[kMostStages];   // of the ring
    int abort;
    float warp_mx[kWarps];
    float warp_s[kWarps], warp_w[kWarps];
    uint32_t warp_u[kWarps];
    alignas(16) uint32_t pair_key[kPairs];   // read four at a time
    float bound, tie;   // the bound, and the maximum that it was taken from
    float seg_mx[kSegs][kThreads];
    uint16_t flagged[kSegs * kThreads];   // seg * kThreads + thread
    int nflagged, ncand;
    PartSums parts[kMaxCluster];          // of a split row; written by the parts' CTAs, read by rank 0
    uint64_t list[kMaxTopK];              // the CTA's best entries, in order
    uint64_t cand[kCap];
};

// The barrier of the threads that take logits.
__device__ __forceinline__ void meet() { named_bar_sync(1, kThreads); }
// The barrier of all threads of a row's cluster.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    cluster_sync_all();
}

static_assert(kMaxTopK <= kPairs, "the bound is one of the pairs' maxima");
static_assert(kMaxCluster * kMaxTopK <= kCap, "the parts' lists fit the candidates");
static_assert(offsetof(Shared, pair_key) % 16 == 0 && alignof(Shared) >= 16, "vector reads of the maxima");
static_assert(offsetof(Shared, full) % 8 == 0 && offsetof(Shared, parts) % 16 == 0 &&
                  offsetof(Shared, list) % 8 == 0 && offsetof(Shared, cand) % 8 == 0,
              "barriers, sums and entries");

__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    meet();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    meet();
    float r = 0.0f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) r += buf[j];
    return r;
}

__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* buf) {
    x = __reduce_max_sync(0xffffffffu, x);
    meet();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    meet();
    uint32_t r = 0u;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) r = max(r, buf[j]);
    return r;
}

// The part of a row that one CTA of its cluster takes: up to 15 bytes of head,
// vectors of 16 bytes, a tail; vectors [v0, v1) here, the head in the first
// part and the tail in the last.
template <int kType>
struct Part {
    const uint8_t* row;
    const uint4* vec;
    int head, tail0, v0, v1, turns;
    __device__ Part(const LogprobArgs& a, uint32_t m, uint32_t rank, uint32_t S) {
        using F = Fmt<kType>;
        row = static_cast<const uint8_t*>(a.logits) + int64_t{m} * a.ld * F::kSize;
        head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / F::kSize;
        if (head > a.V) head = a.V;
        const int nv = (a.V - head) / F::kE;
        const int lg = __ffs(S) - 1;   // S is a power of two
        v0 = static_cast<int>(static_cast<int64_t>(nv) * rank >> lg);
        v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) >> lg);
        vec = reinterpret_cast<const uint4*>(row + head * F::kSize);
        tail0 = head + nv * F::kE;
        turns = (v1 - v0 + kTurn - 1) / kTurn;
    }
};

// A part with its share of the row's head and tail, for the ways that read it
// again from memory.  They are functions of their own that work it out anew: as
// part of the one pass they cost that its registers (158 -> 173 us on 4096 x
// 131072 BF16).
template <int kType>
struct WholePart : Part<kType> {
    int heads, tails;
    __device__ WholePart(const LogprobArgs& a, uint32_t m, uint32_t rank, uint32_t S)
        : Part<kType>(a, m, rank, S), heads(rank == 0 ? this->head : 0),
          tails(rank == S - 1 ? a.V - this->tail0 : 0) {}
};

// fn(logit, its index) for this thread's share of a part, in no order.
template <int kType, typename Fn>
__device__ __forceinline__ void each_logit(const WholePart<kType>& part, Fn fn) {
    using F = Fmt<kType>;
    const int tid = threadIdx.x;
    if (tid < part.heads) fn(value_at<F>(part.row, tid), tid);
    if (tid < part.tails) fn(value_at<F>(part.row, part.tail0 + tid), part.tail0 + tid);
#pragma unroll 4
    for (int u = part.v0 + tid; u < part.v1; u += kThreads) {
        const uint4 x = part.vec[u];
        const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < F::kE; ++e) fn(F::element(raw, e), part.head + u * F::kE + e);
    }
}

// Appends the largest logits of a part, from those of key `best` down, to the
// `have` entries of sh.cand until there are k: one distinct value at a time, its
// occurrences in index order.  Returns the entries there are (fewer than k where
// the part has no more).
template <int kType>
__device__ __forceinline__ int top_from(const WholePart<kType>& part, uint32_t best, int have, int k, Shared& sh) {
    using F = Fmt<kType>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    while (have < k && best != 0u) {
        // hits: a bit per logit from `index` on; the threads' are in index order
        auto append = [&](uint32_t hits, uint32_t index) {
            int upto = __popc(hits);
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int before = __shfl_up_sync(0xffffffffu, upto, s);
                if (lane >= s) upto += before;
            }
            meet();
            if (lane == 31) sh.warp_u[warp] = upto;
            meet();
            int at = have + upto - __popc(hits);
            for (int j = 0; j < kWarps; ++j) {
                if (j < warp) at += sh.warp_u[j];
                have += sh.warp_u[j];
            }
            for (; hits != 0u && at < k; hits &= hits - 1u, ++at)
                sh.cand[at] = static_cast<uint64_t>(best) << 32 | (0xFFFFFFFFu - (index + __ffs(hits) - 1));
        };
        if (part.heads > 0) append(tid < part.heads && order_key(value_at<F>(part.row, tid)) == best, tid);
        for (int u0 = part.v0; u0 < part.v1 && have < k; u0 += kThreads) {
            const int u = u0 + tid;
            uint32_t hits = 0u;
            if (u < part.v1) {
                const uint4 x = part.vec[u];
                const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < F::kE; ++e) hits |= (order_key(F::element(raw, e)) == best ? 1u : 0u) << e;
            }
            append(hits, part.head + u * F::kE);
        }
        if (part.tails > 0 && have < k)
            append(tid < part.tails && order_key(value_at<F>(part.row, part.tail0 + tid)) == best, part.tail0 + tid);
        if (have >= k) break;
        uint32_t next = 0u;
        each_logit(part, [&](float x, int) {
            const uint32_t key = order_key(x);
            if (key < best) next = max(next, key);
        });
        best = block_max(next, sh.warp_u);
    }
    meet();
    return have < k ? have : k;
}

// The `need` largest of a part where more than kCap logits reach the bound that
// was taken from the maximum `tie`, such as masked ones where fewer than top_k
// are left: what is above the tie, then the tie and the values under it by index
// (32 x 131072 BF16 with 5 tokens left, 8 asked for: 1650 us with the plain
// method for such rows, now 22).  Returns the entries in sh.cand; more than kCap or
// fewer than needed where this fails.
template <int kType>
__device__ __noinline__ int top_of_ties(const LogprobArgs& a, uint32_t m, uint32_t rank, uint32_t S, float tie,
                                        int need, Shared& sh) {
    const WholePart<kType> part(a, m, rank, S);
    const uint32_t key = order_key(tie);
    meet();   // everyone has read the count
    if (threadIdx.x == 0) sh.ncand = 0;
    meet();
    uint32_t best = 0u;   // of the others
    each_logit(part, [&](float x, int index) {
        const uint32_t k = order_key(x);
        if (k > key) {
            const int at = atomicAdd(&sh.ncand, 1);
            if (at < kCap) sh.cand[at] = entry_of(x, index);
        } else {
            best = max(best, k);
        }
    });
    best = block_max(best, sh.warp_u);
    const int n = sh.ncand;
    return n < need ? top_from(part, best, n, need, sh) : n;
}

// ----------------------------------------------------------------- the plain way
// A whole row by its definition: maximum, then sums of differences.
template <int kType>
__device__ __noinline__ void plain_row(const LogprobArgs& a, uint32_t m, Shared& sh) {
    using F = Fmt<kType>;
    const WholePart<kType> part(a, m, 0, 1);
    uint32_t best = 0u;
    each_logit(part, [&](float x, int) { best = max(best, order_key(x)); });
    best = block_max(best, sh.warp_u);
    const float mx = key_value(best);
    const bool none = mx == -INFINITY;   // a row with nothing left
    float s = 0.0f, w = 0.0f;
    if (!none)
        each_logit(part, [&](float x, int) {
            const float d = x - mx;
            const float e = ex2(d * kLog2e);
            s += e;
            if (e != 0.0f) w += e * d;
        });
    s = block_sum(s, sh.warp_s);
    w = block_sum(w, sh.warp_w);
    const float ls = logf(s);
    for (int t = threadIdx.x; t < a.T; t += kThreads) {
        const int64_t id = a.tokens[int64_t{m} * a.ldt + t];
        const bool in = id >= 0 && id < a.V;
        a.token_lp[int64_t{m} * a.T + t] = !in || none ? -INFINITY : value_at<F>(part.row, id) - mx - ls;
    }
    if (a.entropy && threadIdx.x == 0) a.entropy[m] = none ? 0.0f : ls - w / s;
    if (a.top_k > 0) {
        top_from(part, best, 0, a.top_k, sh);
        if (threadIdx.x < a.top_k) {
            const uint64_t e = sh.cand[threadIdx.x];
            a.top_ids[int64_t{m} * a.top_k + threadIdx.x] = entry_index(e);
            a.top_lp[int64_t{m} * a.top_k + threadIdx.x] =
                none ? -INFINITY : key_value(static_cast<uint32_t>(e >> 32)) - mx - ls;
        }
        meet();   // before the next row's candidates
    }
}

// ----------------------------------------------------------------- one pass
// ln p of logit x by the row's reference and ln s.  Below -1e30 (where x L may
// leave the range) both are lost in x: it is its own log probability.  Of a token
// that holds all of the row the roundings of t, 2^t and ln s leave about +-2e-7:
// not above 0.  (Rows with a NaN do not come here.)
__device__ __forceinline__ float logp_of(float x, float c, float ls) {
    return x < -1e30f ? x : fminf(fmaf(fmaf(x, kLog2e, -c), kLn2, -ls), 0.0f);
}

// kN vectors of a thread: their maximum first, which is returned (moving c where
// it rose), then their terms, two at a time.
template <int kType, int kN>
__device__ __forceinline__ float take(const uint4 (&x)[kN], float& mx, float& c, uint64_t& s2, uint64_t& w2) {
    using F = Fmt<kType>;
    uint32_t u[kN * 4];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        u[4 * j + 0] = F::floor_word(x[j].x);
        u[4 * j + 1] = F::floor_word(x[j].y);
        u[4 * j + 2] = F::floor_word(x[j].z);
        u[4 * j + 3] = F::floor_word(x[j].w);
    }
    uint32_t mw[kN * 2];
#pragma unroll
    for (int j = 0; j < kN * 2; ++j) mw[j] = F::max_word(u[2 * j], u[2 * j + 1]);
#pragma unroll
    for (int n = kN; n > 0; n >>= 1)
#pragma unroll
        for (int j = 0; j < n; ++j) mw[j] = F::max_word(mw[j], mw[j + n]);
    const float top = F::max_of(mw[0]);
    if (top > mx) {
        mx = top;
        const float c2 = reference_of(top);
        if (c2 > c) {
            const float d = c - c2;
            const float f = ex2(d);
            const uint64_t f2 = pack2(f, f);
            w2 = fma2(fma2(pack2(d, d), s2, w2), f2, pack2(0.0f, 0.0f));
            s2 = fma2(s2, f2, pack2(0.0f, 0.0f));
            c = c2;
        }
    }
    const uint64_t l2 = pack2(kLog2e, kLog2e);
    const uint64_t c2 = pack2(-c, -c);
#pragma unroll
    for (int j = 0; j < kN * 4; j += (F::kE == 4 ? 2 : 1)) {
        float a, b;
        if constexpr (F::kE == 4) {
            a = __uint_as_float(u[j]);
            b = __uint_as_float(u[j + 1]);
        } else {
            F::unpack(u[j], a, b);
        }
        const uint64_t t2 = fma2(pack2(a, b), l2, c2);
        unpack2(t2, a, b);
        const uint64_t e2 = pack2(ex2(a), ex2(b));
        s2 = add2(s2, e2);
        w2 = fma2(e2, t2, w2);
    }
    return top;
}

template <int kType>
__device__ __forceinline__ void take_row(const LogprobArgs& a, uint32_t m, uint32_t rank, uint32_t S, Shared& sh,
                                         const uint4* ring, uint64_t* joined, int stages, bool resident,
                                         uint32_t next, int64_t& ahead, int& stage, uint32_t& phase,
                                         const WaitCtl& wc) {
    using F = Fmt<kType>;
    const int tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const Part<kType> part(a, m, rank, S);
    const uint8_t* row = part.row;
    const uint4* vec = part.vec;
    const int head = part.head, v0 = part.v0, v1 = part.v1, tail0 = part.tail0;

    // the asked token's logit, on its way while the row is read, and the token
    // of the CTA's next row (its load and the logit's in a row cost 1 us a row)
    bool known = false;   // the token lies in the vocabulary
    typename F::Word tok_w = 0;
    if (rank == 0 && tid < a.T) {
        if (ahead >= 0 && ahead < a.V) {
            known = true;
            tok_w = word_at<F>(row, ahead);
        }
        if (next < static_cast<uint32_t>(a.M)) ahead = a.tokens[int64_t{next} * a.ldt + tid];
    }
    int lone = -1;   // the index of the head or tail logit this thread takes
    if (rank == 0 && tid < head) lone = tid;
    if (rank == S - 1 && tid >= 32 && tid - 32 < a.V - tail0) lone = tail0 + tid - 32;
    typename F::Word lone_w = 0;
    if (lone >= 0) lone_w = word_at<F>(row, lone);

    Sums t{-INFINITY, kNoRef, 0.0f, 0.0f};
    uint64_t s2 = pack2(0.0f, 0.0f), w2 = pack2(0.0f, 0.0f);
    const uint4 empty = make_uint4(F::kEmpty, F::kEmpty, F::kEmpty, F::kEmpty);
    // turns of a stretch, as a power of two
    int seg_lg = 0;
    while (kSegs << seg_lg < part.turns) ++seg_lg;
    float seg = -INFINITY;
    for (int n = 0; n < part.turns; ++n) {
        // a wait that gives up raises the abort flag and the status; the row
        // goes on (with what the ring holds), so that every thread meets the others
        wait_bounded(smem_u32(&sh.full[stage]), phase, wc);
        const uint4* at = ring + stage * kTurn + tid;
        const int left = v1 - v0 - n * kTurn;   // vectors, from this turn on
        if (left >= kTurn) {
            uint4 x[kU];
#pragma unroll
            for (int j = 0; j < kU; ++j) x[j] = at[j * kThreads];
            seg = fmaxf(seg, take<kType>(x, t.mx, t.c, s2, w2));
        } else {
            // a part's last turn, two vectors a thread at a time: nothing is
            // worked out for what is not there
#pragma unroll 1
            for (int j = 0; j * kThreads < left; j += 2) {
                const int here = left - j * kThreads - tid;
                const uint4 x[2] = {here > 0 ? at[j * kThreads] : empty,
                                    here > kThreads ? at[(j + 1) * kThreads] : empty};
                seg = fmaxf(seg, take<kType>(x, t.mx, t.c, s2, w2));
            }
        }
        if (((n + 1) & ((1 << seg_lg) - 1)) == 0 || n + 1 == part.turns) {   // read by this thread only
            sh.seg_mx[n >> seg_lg][tid] = seg;
            seg = -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    {
        float s_hi, w_hi;
        unpack2(s2, t.s, s_hi);
        unpack2(w2, t.w, w_hi);
        t.s += s_hi;
        t.w += w_hi;
    }
    const float lone_x = F::value(lone_w);
    if (lone >= 0) {
        const float x = lone_x < F::kFloor ? F::kFloor : lone_x;   // a NaN passes
        t.mx = fmaxf(t.mx, x);
        const float c2 = reference_of(x);
        if (c2 > t.c) t.move_to(c2);
        const float tt = fmaf(x, kLog2e, -t.c);
        const float e = ex2(tt);
        t.s += e;
        t.w = fmaf(e, tt, t.w);
    }

    // the CTA's maximum and sums, and (for alternatives) the pairs' maxima
    const float own = t.mx;
    const float pair = fmaxf(own, __shfl_xor_sync(0xffffffffu, own, 1));
    float mx = pair;
    const uint32_t key = (order_key(mx) & ~(kPairs - 1u)) | (kPairs - 1u - (tid >> 1));
    if ((tid & 1) == 0) sh.pair_key[tid >> 1] = key;
#pragma unroll
    for (int s = 16; s > 1; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    if (lane == 0) sh.warp_mx[warp] = mx;
    if (tid == 0) sh.nflagged = sh.ncand = 0;
    if (tid < kMaxTopK) sh.list[tid] = 0ull;
    meet();
    mx = sh.warp_mx[0];
#pragma unroll
    for (int j = 1; j < kWarps; ++j) mx = fmaxf(mx, sh.warp_mx[j]);
    const float c = reference_of(mx);
    t.move_to(c);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        t.s += __shfl_xor_sync(0xffffffffu, t.s, s);
        t.w += __shfl_xor_sync(0xffffffffu, t.w, s);
    }
    if (lane == 0) {
        sh.warp_s[warp] = t.s;
        sh.warp_w[warp] = t.w;
    }

    bool bad = false;   // this CTA's list is not to be used
    if (a.top_k > 0) {
        // The bound: the top_k-th largest of the maxima of pairs of threads, by
        // counting, on their keys with the pair's number in the low bits (which
        // makes them distinct, and the bound at most that much lower than the
        // maximum).  Each thread counts for its pair against half of them (against
        // the threads' own 128 maxima it took 0.7 us more a row under load, for 22
        // logits instead of 24 at the bound of 20 alternatives).
        float bound = mx;
        if (a.top_k > 1) {
            const uint4* k4 = reinterpret_cast<const uint4*>(sh.pair_key) + (tid & 1) * (kPairs / 8);
            int above = 0;
#pragma unroll
            for (int j = 0; j < kPairs / 8; ++j) {
                const uint4 o = k4[j];
                above += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
            }
            above += __shfl_xor_sync(0xffffffffu, above, 1);
            if (above == a.top_k - 1) {   // both threads of the pair
                sh.bound = key_value(max(key & ~(kPairs - 1u), order_key(-INFINITY)));
                sh.tie = pair;
            }
            meet();
            bound = sh.bound;
        }
        if (own >= bound) {
            float seg_of[kSegs];
            int hits = 0;
#pragma unroll
            for (int j = 0; j < kSegs; ++j) {
                seg_of[j] = j << seg_lg < part.turns ? sh.seg_mx[j][tid] : NAN;
                hits += seg_of[j] >= bound;
            }
            int at = hits > 0 ? atomicAdd(&sh.nflagged, hits) : 0;
#pragma unroll
            for (int j = 0; j < kSegs; ++j)
                if (seg_of[j] >= bound) sh.flagged[at++] = static_cast<uint16_t>(j * kThreads + tid);
        }
        if (lone >= 0 && (lone_x < F::kFloor ? F::kFloor : lone_x) >= bound)
            sh.cand[atomicAdd(&sh.ncand, 1)] = entry_of(lone_x, lone);   // 14 at most
        meet();
        // a part that went into the ring without a second turn round it is still there
        const uint4* from = resident && part.turns <= stages ? ring - v0 : vec;
        const int nflagged = sh.nflagged;
        auto look = [&](const uint4& x, int u) {
            const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = F::floor_word(raw[j]);
            if (F::max_of(F::max_word(F::max_word(w[0], w[1]), F::max_word(w[2], w[3]))) < bound) return;
            const uint32_t index = head + u * F::kE;
            float y[F::kE];
            int hits = 0;
#pragma unroll
            for (int e = 0; e < F::kE; ++e) {
                y[e] = F::element(raw, e);
                hits += (y[e] < F::kFloor ? F::kFloor : y[e]) >= bound;
            }
            if (*static_cast<volatile int*>(&sh.ncand) > kCap) return;   // too many already
            int at = atomicAdd(&sh.ncand, hits);
#pragma unroll
            for (int e = 0; e < F::kE; ++e)
                if ((y[e] < F::kFloor ? F::kFloor : y[e]) >= bound) {
                    if (at < kCap) sh.cand[at] = entry_of(y[e], index + e);
                    ++at;
                }
        };
        // all vectors of the flagged stretches, spread over the threads
        const int per_lg = seg_lg + kULg;
        auto vector_of = [&](int q) {
            const int f = sh.flagged[q >> per_lg];
            const int round = ((f / kThreads) << per_lg) + (q & ((1 << per_lg) - 1));
            return v0 + round * kThreads + f % kThreads;
        };
        // (a marked stretch holds a logit at the bound or more: more than kCap of
        // them need no count)
        const int all = nflagged > kCap ? 0 : nflagged << per_lg;
        for (int q = tid; q < all; q += 4 * kThreads) {   // four loads in flight
            uint4 x[4];
            int u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u[j] = q + j * kThreads < all ? vector_of(q + j * kThreads) : v1;
                x[j] = u[j] < v1 ? from[u[j]] : empty;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (u[j] < v1) look(x[j], u[j]);
        }
        meet();
        int n = sh.nflagged > kCap ? kCap + 1 : sh.ncand;
        const int size = (v1 - v0) * F::kE + (rank == 0 ? head : 0) + (rank == S - 1 ? a.V - tail0 : 0);
        const int need = a.top_k < size ? a.top_k : size;
        if (n > kCap) n = top_of_ties<kType>(a, m, rank, S, a.top_k > 1 ? sh.tie : mx, need, sh);
        // (fewer than asked for: NaNs, which no bound sees)
        bad = n > kCap || n < need;
        if (!bad)
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t mine = sh.cand[i];
                int above = 0;
#pragma unroll 8
                for (int j = 0; j < n; ++j) above += sh.cand[j] > mine;
                if (above < a.top_k) sh.list[above] = mine;
            }
    }
    meet();
    Sums r{mx, c, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        r.s += sh.warp_s[j];
        r.w += sh.warp_w[j];
    }

    if (S > 1) {
        // every part's sums and list to rank 0, which has started by then
        cluster_wait_all();
        const uint32_t to = map_to_cta(smem_u32(&sh.parts[rank]), 0);
        if (tid == 0) {
            st_peer(to, r.mx, r.c, r.s, r.w);
            st_peer(to + 16, bad ? 1.0f : 0.0f);
        }
        if (tid < a.top_k) st_peer(map_to_cta(smem_u32(joined + rank * a.top_k + tid), 0), sh.list[tid]);
        cluster_meet();
        if (rank != 0) return;
        // every warp adds the parts up for itself, lane l holding part l
        const bool has = lane < static_cast<int>(S);
        Sums p{-INFINITY, kNoRef, 0.0f, 0.0f};
        if (has) p = sh.parts[lane].sums;
        bad = __any_sync(0xffffffffu, has && sh.parts[lane].bad != 0.0f);
        float top = p.mx;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        r.mx = top;
        r.c = reference_of(top);
        p.move_to(r.c);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            p.s += __shfl_xor_sync(0xffffffffu, p.s, s);
            p.w += __shfl_xor_sync(0xffffffffu, p.w, s);
        }
        r.s = p.s;
        r.w = p.w;
        if (a.top_k > 0) {
            // At least top_k entries reach the q-th largest of the lists' j-th
            // entries, j q >= top_k, with the smallest j that S lists allow (with
            // j = top_k, the largest of the last entries, 20 alternatives of 32
            // rows in 16 parts left 230 entries to rank and took 18.6 us).
            const int j = (a.top_k + static_cast<int>(S) - 1) / static_cast<int>(S);
            const int q = (a.top_k + j - 1) / j;
            const uint64_t mine = has ? joined[lane * a.top_k + j - 1] : 0ull;
            int above = 0;
            for (int l = 0; l < static_cast<int>(S); ++l) {
                const uint64_t other = __shfl_sync(0xffffffffu, mine, l);
                above += other > mine || (other == mine && l < lane);
            }
            const uint32_t at = __ballot_sync(0xffffffffu, has && above == q - 1);
            const uint64_t bound = __shfl_sync(0xffffffffu, mine, __ffs(at) - 1);
            if (tid == 0) sh.ncand = 0;
            meet();
            for (int e = tid; e < static_cast<int>(S) * a.top_k; e += kThreads)
                if (joined[e] >= bound && joined[e] != 0ull) sh.cand[atomicAdd(&sh.ncand, 1)] = joined[e];
            meet();
            const int n = sh.ncand;
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t one = sh.cand[i];
                int rank_of = 0;
#pragma unroll 8
                for (int l = 0; l < n; ++l) rank_of += sh.cand[l] > one;
                if (rank_of < a.top_k) sh.list[rank_of] = one;
            }
            meet();
        }
    }

    // not (a <= b) is also true of a NaN
    if (!(fabsf(r.mx) <= kFar) || r.mx <= F::kFloor + 500.0f || r.s != r.s || bad) {
        plain_row<kType>(a, m, sh);
        return;
    }
    const float ls = logf(r.s);
    if (tid < a.T) a.token_lp[int64_t{m} * a.T + tid] = known ? logp_of(F::value(tok_w), r.c, ls) : -INFINITY;
    for (int i = tid + kThreads; i < a.T; i += kThreads) {
        const int64_t id = a.tokens[int64_t{m} * a.ldt + i];
        a.token_lp[int64_t{m} * a.T + i] = id < 0 || id >= a.V ? -INFINITY : logp_of(value_at<F>(row, id), r.c, ls);
    }
    if (a.entropy && tid == 0) a.entropy[m] = fmaxf(ls - kLn2 * (r.w / r.s), 0.0f);
    if (tid < a.top_k) {
        const uint64_t e = sh.list[tid];
        a.top_ids[int64_t{m} * a.top_k + tid] = entry_index(e);
        a.top_lp[int64_t{m} * a.top_k + tid] = logp_of(key_value(static_cast<uint32_t>(e >> 32)), r.c, ls);
    }
}

__host__ __device__ constexpr uint32_t joined_bytes(uint32_t S, int top_k) {
    return S > 1 ? (S * static_cast<uint32_t>(top_k) * 8u + 127u) & ~127u : 0u;
}

template <int kType>
__global__ void __launch_bounds__(kThreads + 32, kCtasPerSm)
    logprobs_kernel(const LogprobArgs a, int stages, uint64_t timeout_ns, uint32_t* status) {
    extern __shared__ __align__(128) uint4 dynamic[];   // the lists of a split row's parts, then the ring
    __shared__ Shared sh;
    const uint32_t S = cluster_size(), rank = cluster_cta_rank();
    uint64_t* joined = reinterpret_cast<uint64_t*>(dynamic);   // [S][top_k]
    uint4* ring = dynamic + joined_bytes(S, a.top_k) / 16;     // [stages][kTurn]
    if (S > 1) cluster_arrive_all();   // waited for in front of the first store to a peer
    if (threadIdx.x == kThreads) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kWarps);
        }
        sh.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const WaitCtl wc{timeout_ns, status, &sh.abort};
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t row0 = blockIdx.x / S;
    const uint32_t rows = gridDim.x / S;   // rows in flight; more than one each only where S is 1
    const uint32_t M = static_cast<uint32_t>(a.M);

    if (threadIdx.x >= kThreads) {
        if (threadIdx.x == kThreads) {
            const uint64_t pol = policy_evict_normal();   // what reaches a bound is read again
            int issued = 0, slot = 0;
            uint32_t turned = 0u;   // parity of the times round the ring
            bool ok = true;
            for (uint32_t m = row0; m < M && ok; m += rows) {
                const Part<kType> part(a, m, rank, S);
                for (int n = 0; n < part.turns; ++n) {
                    if (issued >= stages) ok = wait_bounded(smem_u32(&sh.empty[slot]), turned ^ 1u, wc);
                    if (!ok) break;
                    const int v = part.v0 + n * kTurn;
                    const uint32_t bytes = (part.v1 - v < kTurn ? part.v1 - v : kTurn) * 16u;
                    const uint32_t bar = smem_u32(&sh.full[slot]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_load(smem_u32(ring + slot * kTurn), part.vec + v, bytes, bar, pol);
                    ++issued;
                    if (++slot == stages) {
                        slot = 0;
                        turned ^= 1u;
                    }
                }
            }
            // every copy lands before the CTA may end
            for (int i = issued - stages < 0 ? 0 : issued - stages; i < issued; ++i)
                gemm::drain_wait(smem_u32(&sh.full[i % stages]), (i / stages) & 1, timeout_ns);
        }
        if (S > 1) {   // the two of take_row
            __syncwarp();
            cluster_wait_all();
            cluster_meet();
        }
        return;
    }
    int stage = 0;
    uint32_t phase = 0;
    int64_t ahead = rank == 0 && threadIdx.x < a.T ? a.tokens[row0 * a.ldt + threadIdx.x] : -1;
    for (uint32_t m = row0; m < M; m += rows)
        take_row<kType>(a, m, rank, S, sh, ring, joined, stages, rows >= M, m + rows, ahead, stage, phase, wc);
}

// CTAs per row: a power of two up to 16, so that the CTAs are at most two per
// SM and take 2048 logits or more each.  More of them cost more to launch as
// clusters and to join than the shorter parts save (32 x 131072 FP32, 20
// alternatives: 12.3 us in 16 parts, 11.3 in 8, 13.1 in 4; 57 x 131072 BF16, 5:
// 12.0 in 8, 10.8 in 4; 380 x 8000: 9.5 in 2, 6.1 whole; but 100 x 50000: 10.4 in
// 4, 10.8 in 2).
int parts_of(int M, int V, int sms) {
    int s = 1;
    while (s < kMaxCluster && static_cast<int64_t>(M) * 2 * s <= 2 * sms && V / (2 * s) >= 2048) s *= 2;
    return s;
}

// CTAs that take whole rows: as many as run at once, unless few of them would
// take the last round, which reads slower than memory gives; then all take the
// same number (800 x 131072 BF16: 48.6 us on 760 CTAs, 41.4 on 400; 1600: 77.8 and
// 76.6 on 534; but 2500 with a third of them in the last round 105 and 112).
int64_t row_ctas(int M, int sms) {
    const int64_t most = static_cast<int64_t>(kCtasPerSm) * sms;
    if (M <= most) return M;
    const int64_t rounds = (M + most - 1) / most;
    const int64_t last = M - (rounds - 1) * most;
    return last * 8 < most ? (M + rounds - 1) / rounds : most;
}

// The ring's turns: what an SM's shared memory holds for its CTAs (two turns
// each where there are four or more, four where there are two: 260 x 160000
// FP32 38.5 -> 34.2 us, 128 x 131072 BF16, 20 alternatives, 17.5 -> 16.5).
int stages_of(int64_t ctas, int sms) {
    const int64_t per_sm = (ctas + sms - 1) / sms;
    return per_sm <= 2 ? 4 : per_sm == 3 ? 3 : 2;
}

template <int kType>
cudaError_t launch(const LogprobArgs& a, const LaunchCtl& c, cudaStream_t st) {
    const int parts = parts_of(a.M, a.V, c.num_sms);
    const int64_t ctas = parts > 1 ? static_cast<int64_t>(a.M) * parts : row_ctas(a.M, c.num_sms);
    // A CTA with one part to take needs no more of the ring than its turns (a
    // part has at most V / parts / kE + 1 vectors); one that runs on into
    // another row goes round all of it.
    const int turns = a.V / parts / (kTurn * Fmt<kType>::kE) + 1;
    const bool one_part = parts > 1 || a.M == ctas;
    const int stages = stages_of(ctas, c.num_sms);
    const int ring_bytes = (one_part && turns < stages ? turns : stages) * kTurn * 16;
    static std::atomic<uint64_t> configured{0}, wide{0};
    cudaError_t e = set_smem_once(configured, logprobs_kernel<kType>,
                                 kMostStages * kTurn * 16 + joined_bytes(kMaxCluster, kMaxTopK));
    if (e == cudaSuccess && parts > 8)
        e = set_once(wide, logprobs_kernel<kType>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(ring_bytes) + joined_bytes(parts, a.top_k);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.overlap ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<kType>, a, stages, c.timeout_ns, c.status);
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
