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
// The alternatives come from the same pass.  Every pair of threads knows the
// largest logit it has seen; the k-th largest of these maxima is a bound that
// at least k logits reach, and only the pairs that reach it (k of them, but
// for ties) look at their logits again, in L2.  What reaches the bound (about
// k (1 + k / 256) logits of a row without structure) is ranked by counting.
// They are ordered on 64-bit keys: the value, then the lower index.
//
// Rows where this does not hold are worked out by the plain method at the end
// of this file's row function: a maximum beyond +-1e8 (or at the floor: a row
// of nothing but masks), a NaN or +inf, or more than kCap logits at the bound.
//
// A few CTAs per SM walk over the rows.  One warp of a CTA streams them into a
// ring in shared memory by bulk copies, running on into the next row while the
// other eight finish one (choosing the alternatives takes about as long as
// reading 40 KB: 4 us, with nothing on the way from memory when each row had a
// CTA of its own and registers for its loads).  Rows that are too few for the
// SMs are split over a cluster of up to 16 CTAs, whose sums and lists rank 0
// joins through distributed shared memory (no workspace, no atomics on memory,
// the same order of sums on every call).
#include <cstddef>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_gemm.cuh"
#include "qg_launch.h"
#include "qg_logprobs.h"
#include "qg_pair.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;      // that take logits; one more warp streams them in
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = kThreads / 2;
constexpr int kCtasPerSm = 3;
constexpr int kStages = 4;         // of the ring, one turn each
constexpr int kU = 4;              // 16-byte vectors a thread takes in a turn
constexpr int kTurn = kU * kThreads;
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
    __device__ static float at(const void* row, int64_t v) { return static_cast<const float*>(row)[v]; }
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
    __device__ static float at(const void* row, int64_t v) {
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[v]) << 16);
    }
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
    __device__ static float at(const void* row, int64_t v) { return __half2float(static_cast<const __half*>(row)[v]); }
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
// A word of CTA `rank`'s shared memory at the address `p` has in this CTA's.
__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) { return map_to_cta(smem_u32(p), rank); }
__device__ __forceinline__ float peer_f32(const float* p, uint32_t rank) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(peer_address(p, rank)) : "memory");
    return r;
}
__device__ __forceinline__ uint64_t peer_u64(const uint64_t* p, uint32_t rank) {
    uint64_t r;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(r) : "r"(peer_address(p, rank)) : "memory");
    return r;
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

struct Shared {
    uint64_t full[kStages], empty[kStages];   // of the ring
    int abort;
    float warp_mx[kWarps];
    float warp_s[kWarps], warp_w[kWarps];
    uint32_t warp_u[kWarps];
    alignas(16) uint32_t pair_key[kPairs];   // read four at a time
    float bound;
    int flagged[kPairs];
    int nflagged, ncand, nlist;
    float sums[4];                        // mx, c, s, w of the CTA; read by rank 0
    float bad;                            // the CTA's list is not to be used; read by rank 0
    uint64_t list[kMaxTopK];              // the CTA's best entries, in order; read by rank 0
    uint64_t cand[kCap];
    uint64_t joined[kMaxCluster * kMaxTopK];
    uint32_t slow_keys[kMaxTopK];
    int slow_ids[kMaxTopK];
};

// The barrier of the threads that take logits.
__device__ __forceinline__ void meet() { named_bar_sync(1, kThreads); }
// The barrier of all threads of a row's cluster.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    cluster_sync_all();
}

static_assert(offsetof(Shared, pair_key) % 16 == 0 && alignof(Shared) >= 16, "vector reads of the maxima");
static_assert(offsetof(Shared, full) % 8 == 0 && offsetof(Shared, list) % 8 == 0 && offsetof(Shared, cand) % 8 == 0 &&
                  offsetof(Shared, joined) % 8 == 0,
              "barriers and entries");

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

// ----------------------------------------------------------------- the plain way
// The top alternatives of a row, one distinct value at a time: the largest key
// below the previous one, then its occurrences in index order.
template <int kType>
__device__ __noinline__ void top_by_value(const void* row, int V, int k, Shared& sh) {
    using F = Fmt<kType>;
    int have = 0;
    uint64_t below = 1ull << 32;   // keys under this are left
    while (have < k) {
        uint32_t best = 0u;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const uint32_t key = order_key(F::at(row, v));
            if (key < below) best = max(best, key);
        }
        best = block_max(best, sh.warp_u);
        for (int v0 = 0; v0 < V && have < k; v0 += kThreads) {
            const int v = v0 + threadIdx.x;
            const bool hit = v < V && order_key(F::at(row, v)) == best;
            const uint32_t mask = __ballot_sync(0xffffffffu, hit);
            meet();
            if ((threadIdx.x & 31) == 0) sh.warp_u[threadIdx.x >> 5] = __popc(mask);
            meet();
            int before = 0, total = 0;
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                if (j < static_cast<int>(threadIdx.x >> 5)) before += sh.warp_u[j];
                total += sh.warp_u[j];
            }
            const int at = have + before + __popc(mask & ((1u << (threadIdx.x & 31)) - 1u));
            if (hit && at < k) {
                sh.slow_keys[at] = best;
                sh.slow_ids[at] = v;
            }
            have += total;
        }
        below = best;
    }
    meet();
}

// A whole row by its definition: maximum, then sums of differences.
template <int kType>
__device__ __noinline__ void plain_row(const LogprobArgs& a, int64_t m, const void* row, Shared& sh) {
    using F = Fmt<kType>;
    uint32_t best = 0u;
    for (int v = threadIdx.x; v < a.V; v += kThreads) best = max(best, order_key(F::at(row, v)));
    const float mx = key_value(block_max(best, sh.warp_u));
    const bool none = mx == -INFINITY;   // a row with nothing left
    float s = 0.0f, w = 0.0f;
    if (!none)
        for (int v = threadIdx.x; v < a.V; v += kThreads) {
            const float d = F::at(row, v) - mx;
            const float e = ex2(d * kLog2e);
            s += e;
            if (e != 0.0f) w += e * d;
        }
    s = block_sum(s, sh.warp_s);
    w = block_sum(w, sh.warp_w);
    const float ls = logf(s);
    for (int t = threadIdx.x; t < a.T; t += kThreads) {
        const int64_t id = a.tokens[m * a.ldt + t];
        const bool in = id >= 0 && id < a.V;
        a.token_lp[m * a.T + t] = !in || none ? -INFINITY : F::at(row, id) - mx - ls;
    }
    if (a.entropy && threadIdx.x == 0) a.entropy[m] = none ? 0.0f : ls - w / s;
    if (a.top_k > 0) {
        top_by_value<kType>(row, a.V, a.top_k, sh);
        if (threadIdx.x < a.top_k) {
            a.top_ids[m * a.top_k + threadIdx.x] = sh.slow_ids[threadIdx.x];
            a.top_lp[m * a.top_k + threadIdx.x] =
                none ? -INFINITY : key_value(sh.slow_keys[threadIdx.x]) - mx - ls;
        }
    }
}

// ----------------------------------------------------------------- one pass
// ln p of logit x by the row's reference and ln s.  Below -1e30 (where x L may
// leave the range) both are lost in x: it is its own log probability.
__device__ __forceinline__ float logp_of(float x, float c, float ls) {
    return x < -1e30f ? x : fmaf(fmaf(x, kLog2e, -c), kLn2, -ls);
}

// kU vectors of a thread: their maximum first (moving c where it rose), then
// their terms, two at a time.
template <int kType>
__device__ __forceinline__ void take(const uint4 (&x)[kU], float& mx, float& c, uint64_t& s2, uint64_t& w2) {
    using F = Fmt<kType>;
    uint32_t u[kU * 4];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        u[4 * j + 0] = F::floor_word(x[j].x);
        u[4 * j + 1] = F::floor_word(x[j].y);
        u[4 * j + 2] = F::floor_word(x[j].z);
        u[4 * j + 3] = F::floor_word(x[j].w);
    }
    uint32_t mw[kU * 2];
#pragma unroll
    for (int j = 0; j < kU * 2; ++j) mw[j] = F::max_word(u[2 * j], u[2 * j + 1]);
#pragma unroll
    for (int n = kU; n > 0; n >>= 1)
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
    for (int j = 0; j < kU * 4; j += (F::kE == 4 ? 2 : 1)) {
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
}

// The part of a row that one CTA of its cluster takes: up to 15 bytes of head,
// vectors of 16 bytes, a tail; vectors [v0, v1) here, the head in the first
// part and the tail in the last.
template <int kType>
struct Part {
    const uint8_t* row;
    const uint4* vec;
    int head, tail0, v0, v1, turns;
    __device__ Part(const LogprobArgs& a, int64_t m, uint32_t rank, uint32_t S) {
        using F = Fmt<kType>;
        row = static_cast<const uint8_t*>(a.logits) + m * a.ld * F::kSize;
        head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / F::kSize;
        if (head > a.V) head = a.V;
        const int nv = (a.V - head) / F::kE;
        v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / S);
        v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / S);
        vec = reinterpret_cast<const uint4*>(row + head * F::kSize);
        tail0 = head + nv * F::kE;
        turns = (v1 - v0 + kTurn - 1) / kTurn;
    }
};

template <int kType>
__device__ __forceinline__ void take_row(const LogprobArgs& a, int64_t m, uint32_t rank, uint32_t S, Shared& sh,
                                         const uint4* ring, bool resident, int& stage, uint32_t& phase,
                                         const WaitCtl& wc) {
    using F = Fmt<kType>;
    const int tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const Part<kType> part(a, m, rank, S);
    const uint8_t* row = part.row;
    const uint4* vec = part.vec;
    const int head = part.head, v0 = part.v0, v1 = part.v1, tail0 = part.tail0;

    // the asked tokens' logits, on their way while the row is read
    int64_t tok = -1;
    float tok_x = 0.0f;
    if (rank == 0 && tid < a.T) {
        tok = a.tokens[m * a.ldt + tid];
        if (tok >= 0 && tok < a.V) tok_x = F::at(row, tok);
        else tok = -1;
    }
    int lone = -1;   // the index of the head or tail logit this thread takes
    if (rank == 0 && tid < head) lone = tid;
    if (rank == S - 1 && tid >= 32 && tid - 32 < a.V - tail0) lone = tail0 + tid - 32;
    float lone_x = lone >= 0 ? F::at(row, lone) : 0.0f;

    Sums t{-INFINITY, kNoRef, 0.0f, 0.0f};
    uint64_t s2 = pack2(0.0f, 0.0f), w2 = pack2(0.0f, 0.0f);
    const uint4 empty = make_uint4(F::kEmpty, F::kEmpty, F::kEmpty, F::kEmpty);
    for (int n = 0; n < part.turns; ++n) {
        // a wait that gives up raises the abort flag and the status; the row
        // goes on (with what the ring holds), so that every thread meets the others
        wait_bounded(smem_u32(&sh.full[stage]), phase, wc);
        const uint4* at = ring + stage * kTurn + tid;
        const int left = v1 - v0 - n * kTurn - tid;
        uint4 x[kU];
        if (left > (kU - 1) * kThreads) {
#pragma unroll
            for (int j = 0; j < kU; ++j) x[j] = at[j * kThreads];
        } else {
#pragma unroll
            for (int j = 0; j < kU; ++j) x[j] = left > j * kThreads ? at[j * kThreads] : empty;
        }
        take<kType>(x, t.mx, t.c, s2, w2);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        if (++stage == kStages) {
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
    const float pair = fmaxf(t.mx, __shfl_xor_sync(0xffffffffu, t.mx, 1));
    if ((tid & 1) == 0) sh.pair_key[tid >> 1] = (order_key(pair) & ~(kPairs - 1u)) | (kPairs - 1u - (tid >> 1));
    float mx = pair;
#pragma unroll
    for (int s = 16; s > 1; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    if (lane == 0) sh.warp_mx[warp] = mx;
    if (tid == 0) sh.nflagged = sh.ncand = sh.nlist = 0;
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
        // The bound: the top_k-th largest of the pairs' maxima, by counting, on
        // their keys with the pair's number in the low bits (which makes them
        // distinct, and the bound at most that much lower than the maximum).
        // Each thread counts for one pair against half of them.
        float bound = mx;
        if (a.top_k > 1) {
            const uint32_t mine = sh.pair_key[tid >> 1];
            const uint4* p4 = reinterpret_cast<const uint4*>(sh.pair_key) + (tid & 1) * (kPairs / 8);
            int above = 0;
#pragma unroll
            for (int j = 0; j < kPairs / 8; ++j) {
                const uint4 o = p4[j];
                above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
            }
            above += __shfl_xor_sync(0xffffffffu, above, 1);
            if (above == a.top_k - 1)   // both threads of the pair
                sh.bound = key_value(max(mine & ~(kPairs - 1u), order_key(-INFINITY)));
            meet();
            bound = sh.bound;
        }
        if (!(tid & 1) && pair >= bound) sh.flagged[atomicAdd(&sh.nflagged, 1)] = tid >> 1;
        auto push = [&](float x, uint32_t index) {
            const int at = atomicAdd(&sh.ncand, 1);
            if (at < kCap) sh.cand[at] = entry_of(x, index);
        };
        if (lone >= 0 && (lone_x < F::kFloor ? F::kFloor : lone_x) >= bound) push(lone_x, lone);
        meet();
        // Two threads to a round of a pair's vectors, up to 64 rounds of a pair at
        // once, and as many pairs at once as that leaves threads for.
        // a part that went into the ring without a second turn round it is still there
        const uint4* from = resident && part.turns <= kStages ? ring - v0 : vec;
        const int nflagged = sh.nflagged;
        auto look = [&](const uint4& x, int u) {
            const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = F::floor_word(raw[j]);
            if (F::max_of(F::max_word(F::max_word(w[0], w[1]), F::max_word(w[2], w[3]))) < bound) return;
            const uint32_t index = head + u * F::kE;
#pragma unroll
            for (int e = 0; e < F::kE; ++e) {
                const float y = F::element(raw, e);
                if ((y < F::kFloor ? F::kFloor : y) >= bound) push(y, index + e);
            }
        };
        const int rounds = (v1 - v0 + kThreads - 1) / kThreads;
        int lg = 0;
        while (lg < 6 && (1 << lg) < rounds) ++lg;
        const int group = tid >> (lg + 1), groups = kThreads >> (lg + 1);
        const int r0 = (tid & ((2 << lg) - 1)) >> 1;
        for (int u0 = v0 + (tid & 1) + r0 * kThreads; u0 < v1; u0 += kThreads << lg) {
            int f = group;
            for (; f + 3 * groups < nflagged; f += 4 * groups) {   // four loads in flight
                uint4 x[4];
                int u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = u0 + 2 * sh.flagged[f + j * groups];
                    x[j] = u[j] < v1 ? from[u[j]] : empty;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (u[j] < v1) look(x[j], u[j]);
            }
            for (; f < nflagged; f += groups) {
                const int u = u0 + 2 * sh.flagged[f];
                if (u < v1) look(from[u], u);
            }
        }
        meet();
        const int n = sh.ncand;
        // (fewer than asked for in a part that holds them: NaNs, which no bound sees)
        const int size = (v1 - v0) * F::kE + (rank == 0 ? head : 0) + (rank == S - 1 ? a.V - tail0 : 0);
        bad = n > kCap || n < (a.top_k < size ? a.top_k : size);
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
        if (tid == 0) {
            sh.sums[0] = r.mx;
            sh.sums[1] = r.c;
            sh.sums[2] = r.s;
            sh.sums[3] = r.w;
            sh.bad = bad ? 1.0f : 0.0f;
        }
        meet();
        cluster_meet();
        if (rank == 0) {
            // every warp adds the parts up for itself, lane l holding part l
            const bool has = lane < static_cast<int>(S);
            Sums p{-INFINITY, kNoRef, 0.0f, 0.0f};
            bool any_bad = false;
            if (has) {
                p = Sums{peer_f32(sh.sums, lane), peer_f32(sh.sums + 1, lane), peer_f32(sh.sums + 2, lane),
                         peer_f32(sh.sums + 3, lane)};
                any_bad = peer_f32(&sh.bad, lane) != 0.0f;
            }
            bad = __any_sync(0xffffffffu, any_bad);
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
            for (int e = tid; e < static_cast<int>(S) * a.top_k; e += kThreads) {
                const int q = e / a.top_k;
                sh.joined[e] = peer_u64(sh.list + (e - q * a.top_k), q);
            }
            if (tid == 0) sh.ncand = 0;
        }
        cluster_meet();   // nobody's lists are read any more
        if (rank != 0) return;
        if (a.top_k > 0) {
            // what reaches the largest of the lists' last entries holds the answer
            uint64_t bound = 0ull;
            for (int q = 0; q < static_cast<int>(S); ++q) {
                const uint64_t last = sh.joined[q * a.top_k + a.top_k - 1];
                bound = last > bound ? last : bound;
            }
            for (int e = tid; e < static_cast<int>(S) * a.top_k; e += kThreads)
                if (sh.joined[e] >= bound && sh.joined[e] != 0ull) sh.cand[atomicAdd(&sh.ncand, 1)] = sh.joined[e];
            meet();
            const int n = sh.ncand;
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t mine = sh.cand[i];
                int above = 0;
                for (int j = 0; j < n; ++j) above += sh.cand[j] > mine;
                if (above < a.top_k) sh.list[above] = mine;
            }
            meet();
        }
    }

    // not (a <= b) is also true of a NaN
    if (!(fabsf(r.mx) <= kFar) || r.mx <= F::kFloor + 500.0f || r.s != r.s || bad) {
        plain_row<kType>(a, m, row, sh);
        return;
    }
    const float ls = logf(r.s);
    if (tid < a.T) a.token_lp[m * a.T + tid] = tok < 0 ? -INFINITY : logp_of(tok_x, r.c, ls);
    for (int i = tid + kThreads; i < a.T; i += kThreads) {
        const int64_t id = a.tokens[m * a.ldt + i];
        a.token_lp[m * a.T + i] = id < 0 || id >= a.V ? -INFINITY : logp_of(F::at(row, id), r.c, ls);
    }
    if (a.entropy && tid == 0) a.entropy[m] = fmaxf(ls - kLn2 * (r.w / r.s), 0.0f);
    if (tid < a.top_k) {
        const uint64_t e = sh.list[tid];
        a.top_ids[m * a.top_k + tid] = entry_index(e);
        a.top_lp[m * a.top_k + tid] = logp_of(key_value(static_cast<uint32_t>(e >> 32)), r.c, ls);
    }
}

template <int kType>
__global__ void __launch_bounds__(kThreads + 32, kCtasPerSm)
    logprobs_kernel(const LogprobArgs a, uint64_t timeout_ns, uint32_t* status) {
    extern __shared__ __align__(128) uint4 ring[];   // [kStages][kTurn]
    __shared__ Shared sh;
    const uint32_t S = cluster_size(), rank = cluster_cta_rank();
    if (threadIdx.x == kThreads) {
        for (int s = 0; s < kStages; ++s) {
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
    const int64_t row0 = blockIdx.x / S;
    const int64_t rows = gridDim.x / S;   // rows in flight; more than one each only where S is 1

    if (threadIdx.x >= kThreads) {
        if (threadIdx.x == kThreads) {
            const uint64_t pol = policy_evict_normal();   // what reaches a bound is read again
            int issued = 0;
            gemm::Ring<kStages> r(0);
            bool ok = true;
            for (int64_t m = row0; m < a.M && ok; m += rows) {
                const Part<kType> part(a, m, rank, S);
                for (int n = 0; n < part.turns; ++n, r.step(1)) {
                    if (issued >= kStages) ok = wait_bounded(smem_u32(&sh.empty[r.slot]), r.phase ^ 1u, wc);
                    if (!ok) break;
                    const int v = part.v0 + n * kTurn;
                    const uint32_t bytes = (part.v1 - v < kTurn ? part.v1 - v : kTurn) * 16u;
                    const uint32_t bar = smem_u32(&sh.full[r.slot]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_load(smem_u32(ring + r.slot * kTurn), part.vec + v, bytes, bar, pol);
                    ++issued;
                }
            }
            // every copy lands before the CTA may end
            for (int i = issued - kStages < 0 ? 0 : issued - kStages; i < issued; ++i)
                gemm::drain_wait(smem_u32(&sh.full[i % kStages]), (i / kStages) & 1, timeout_ns);
        }
        if (S > 1) {   // the two meetings of take_row
            cluster_meet();
            cluster_meet();
        }
        return;
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t m = row0; m < a.M; m += rows)
        take_row<kType>(a, m, rank, S, sh, ring, rows >= a.M, stage, phase, wc);
}

// CTAs per row: 1 once the rows fill the SMs, else the row is cut into up to
// 16 parts of at least 2048 logits while their CTAs all run at once.
int parts_of(int M, int V, int sms) {
    int s = 1;
    while (s < kMaxCluster && static_cast<int64_t>(M) * 2 * s <= kCtasPerSm * sms * 3 / 4 && V / (2 * s) >= 2048) s *= 2;
    return s;
}

template <int kType>
cudaError_t launch(const LogprobArgs& a, const LaunchCtl& c, cudaStream_t st) {
    const int parts = parts_of(a.M, a.V, c.num_sms);
    const int most = kCtasPerSm * c.num_sms;
    // A CTA with one part to take needs no more of the ring than its turns (a
    // part has at most V / parts / kE + 1 vectors); one that runs on into
    // another row goes round all of it.
    const int turns = a.V / parts / (kTurn * Fmt<kType>::kE) + 1;
    const bool one_part = parts > 1 || a.M <= most;
    const int ring_bytes = (one_part && turns < kStages ? turns : kStages) * kTurn * 16;
    static std::atomic<uint64_t> configured{0}, wide{0};
    cudaError_t e = set_smem_once(configured, logprobs_kernel<kType>, kStages * kTurn * 16);
    if (e == cudaSuccess && parts > 8)
        e = set_once(wide, logprobs_kernel<kType>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(parts > 1 ? a.M * parts : a.M < most ? a.M : most));
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(ring_bytes);
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<kType>, a, c.timeout_ns, c.status);
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
