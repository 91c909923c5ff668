// W8A8 block-scaled GEMM grouped by expert for sm_103a: the rows of the
// activations are ordered by expert, every expert has a weight matrix of its
// own, and how many rows each one has is known on the device only.
//
//   Y[r, n] = sum_kb (sx[kb, r] * s[e, n/128, kb]) * (sum_{k in kb} xq[r, k] * w[e, n, k])
//   for offsets[e] <= r < offsets[e + 1]
//
// Both operands go to tcgen05.mma kind::f8f6f4 as stored (TMA, 128-byte
// swizzle), the weights on the MMA's M side.  A K block of 128 has an
// accumulator of its own in TMEM, which the fold multiplies by the block's
// factors (activation scale x weight scale, one per row of the activations) and
// adds to FP32 outer sums in registers, as the ungrouped kernel does.
//
// The output is tiled in 128 weight rows (256 on a CTA pair) x up to NT rows of
// one expert.  A tile's MMA is as wide as its rows (rounded up to 16 or 32), so that a
// ragged group costs the tensor cores only its rows; columns of TMEM and of the
// activation boxes beyond them hold other rows' values, which nothing stores.
// Every CTA lists the experts that hold rows, with the tiles in front of each,
// at its start; workers then take tiles worker, worker + workers, ..., so that
// those in flight share an expert's weights and activations in L2.
//
// One persistent CTA (or pair) per SM; warps by role:
//   warp 0     producer: a unit's weight and activation boxes into one stage of
//              the ring, one barrier for all of them
//   warp 2     MMA issuer (the pair's first CTA)
//   warp 3     factors: sx * s of the unit's rows into shared memory, the scales
//              fetched some units ahead
//   warps 4-   fold and epilogue: one per TMEM lane quadrant (two in a pair)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_gemm.cuh"
#include "qg_grouped.h"
#include "qg_launch.h"
#include "qg_pair.cuh"

namespace qg {
namespace {

using gemm::Ring;

constexpr int kWarpProd = 0, kWarpMma = 2, kWarpFactor = 3, kWarpFold0 = 4;
constexpr int kMaxExperts = QG_MAX_EXPERTS;
constexpr int kAhead = 4;   // units whose scales the factor warp fetches ahead

template <int NT, bool kPair>
struct GLayout {
    static constexpr int kCtas = kPair ? 2 : 1;
    // K blocks of 128 a unit: with narrow tiles a block's MMAs are short, and two
    // halve the barriers' share
    static constexpr int kBlk = kPair ? 1 : 2;
    static constexpr int kXRows = NT / kCtas;              // activation rows in this CTA's shared memory
    static constexpr int kWBox = 128 * 128;
    static constexpr int kXBox = kXRows * 128;
    static constexpr int kXOff = kBlk * kWBox;             // in a stage, behind the weights
    static constexpr int kStage = kBlk * (kWBox + kXBox);
    static constexpr int kFit = 512 / (kBlk * NT);
    static constexpr int kBufs = kFit < 4 ? kFit : 4;      // accumulator sets (kBlk x NT columns each)
    static constexpr int kFold = kPair ? 8 : 4;            // fold warps
    static constexpr int kCols = NT / (kFold / 4);         // columns of a fold warp
    static constexpr int kThreads = 32 * (kWarpFold0 + kFold);
    static constexpr int kGSlot = kBlk * NT * 4;           // factors of a unit
    static constexpr int kOutWarp = 16 * 64;               // a fold warp's 16 rows x 32 weight rows of 16 bits
    static constexpr int kFixed = kMaxExperts * 16 + kBufs * kGSlot + kFold * kOutWarp + 512;
    static constexpr int kStages = (232448 - kFixed) / kStage;
    static constexpr int kTabOff = kStages * kStage;
    static constexpr int kGOff = kTabOff + kMaxExperts * 16;
    static constexpr int kOutOff = kGOff + kBufs * kGSlot;
    static constexpr int kBarOff = kOutOff + kFold * kOutWarp;
    static constexpr int kNumBars = 2 * kStages + 3 * kBufs;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 32;
    static_assert(kSmemBytes <= 232448, "shared memory");
    static_assert(kBufs >= 2 && kBufs * kBlk * NT <= 512, "TMEM columns");
    static_assert(kXBox % 1024 == 0 && kStage % 1024 == 0, "keep the 1024-byte swizzle alignment");
    static_assert(kCols % 16 == 0 && kXRows % 8 == 0, "fragments");
};

struct GParams {
    const float* Sx;
    int64_t ldsx;
    const float* S;
    const int32_t* offsets;
    void* Y;
    int64_t ldy;
    int y_type;
    int y_vec;        // a 16-bit Y that takes 16-byte stores
    int R, E, N, KB;  // KB: K blocks of 128
    int KU;           // units a tile
    int sn;           // blocks of 128 weight rows (the scales' rows of an expert)
    int tn;           // weight tiles of an expert
    int workers;
    uint64_t timeout_ns;
    int fault_unit;
    uint32_t* status;
};

// ----------------------------------------------------------------- device pieces
// D[tmem] (+)= A[smem] x B[smem]^T, kind::f8f6f4 over a pair (M = 256).
__device__ __forceinline__ void mma_ss_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 8 C columns (C = 2 or 4 groups): lane t holds, of group g, columns
// 2 (t % 4) and the next of rows t / 4 (v[4g], v[4g + 1]) and t / 4 + 8 (v[4g + 2],
// v[4g + 3]).  A lane so meets a quarter of the columns, and of their factors.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// (a0, a1) += (v0, v1) * (f0, f1), each rounded once.
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, float f0, float f1) {
    asm("{\n\t.reg .b64 a, v, f;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 f, {%4, %5};\n\t"
        "fma.rn.f32x2 a, v, f, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(v0), "r"(v1), "f"(f0), "f"(f1));
}

// Four 8 x 8 matrices of 16-bit values, transposed on the way: row j of matrix i
// goes to the address of lane 8 i + j.
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int y_type) {
    if (y_type == QG_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// An expert that holds rows: its first row, how many, the tiles in front of it
// in the grid's order, its number.
struct Group {
    int row0, rows, tile0, expert;
};

// Where tile t lies.  The groups are in ascending order of their tiles.
template <int NT, int kCtas>
struct Place {
    int g;            // the group
    int expert;
    int row0, rows;   // of the tile
    int n0;           // first weight row of this CTA
    int nb;           // its block of 128 weight rows
    __device__ void enter(const Group* tab, int groups, int t, int tn_count, int rank) {
        // the last group whose tiles begin at or before t
        int lo = g, hi = groups - 1;
        if (lo < hi && tab[lo + 1].tile0 <= t) {
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tab[mid].tile0 <= t) lo = mid;
                else hi = mid - 1;
            }
            g = lo;
        }
        const Group q = tab[g];
        expert = q.expert;
        const int tm_count = (q.rows + NT - 1) / NT;
        const int j = t - q.tile0;
        const int tn = j / tm_count;   // a weight tile's row tiles are neighbours: its re-reads come from L2
        const int tm = j - tn * tm_count;
        row0 = q.row0 + tm * NT;
        rows = q.rows - tm * NT < NT ? q.rows - tm * NT : NT;
        nb = tn * kCtas + rank;
        n0 = nb * 128;
    }
    // the MMA's N side: a multiple of 16, on a pair of 32 (16 from each CTA)
    __device__ int width() const { return kCtas == 2 ? (rows + 31) & ~31 : (rows + 15) & ~15; }
};

// The table of the groups and the number of tiles, by one warp.  Offsets are
// taken as they are meant (ascending, from 0 to R); what breaks that is cut so
// that no row lies outside the tensors and none is in two groups.
template <int NT>
__device__ __forceinline__ void list_groups(const GParams& p, Group* tab, int* groups, int* tiles, int lane) {
    int first = __ldcg(p.offsets);
    int end_before = first < 0 ? 0 : first > p.R ? p.R : first;
    int ngroups = 0, ntiles = 0;
    constexpr int kBatch = 8;   // loads in flight
    for (int e0 = 0; e0 < p.E; e0 += 32 * kBatch) {
        int raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int e = e0 + 32 * i + lane;
            raw[i] = e < p.E ? __ldcg(p.offsets + e + 1) : 0;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (e0 + 32 * i >= p.E) break;
            const int e = e0 + 32 * i + lane;
            int end = raw[i] > p.R ? p.R : raw[i];
            if (lane == 0 && end < end_before) end = end_before;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int other = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o && other > end) end = other;
            }
            if (end < end_before) end = end_before;
            int begin = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane == 0) begin = end_before;
            const int rows = e < p.E ? end - begin : 0;
            const int mine = (rows + NT - 1) / NT * p.tn;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int other = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += other;
            }
            const uint32_t active = __ballot_sync(0xffffffffu, rows > 0);
            if (rows > 0)
                tab[ngroups + __popc(active & ((1u << lane) - 1u))] = Group{begin, rows, ntiles + upto - mine, e};
            ngroups += __popc(active);
            ntiles += __shfl_sync(0xffffffffu, upto, 31);
            end_before = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    if (lane == 0) {
        *groups = ngroups;
        *tiles = ntiles;
    }
}

template <int NT, bool kPair>
__global__ void __launch_bounds__(GLayout<NT, kPair>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GParams p) {
    using L = GLayout<NT, kPair>;
    using Pl = Place<NT, L::kCtas>;
    constexpr int kStages = L::kStages, kBufs = L::kBufs, kBlk = L::kBlk, kFold = L::kFold, kCols = L::kCols;
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_u32(gbase);
    if (base & 1023u) {   // the swizzle needs the alignment asked for above
        if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
        return;
    }
    const uint32_t bar0 = base + L::kBarOff;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto dfull = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto dempty = [&](int b) { return bar0 + 8u * (2 * kStages + kBufs + b); };
    auto fempty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 * kBufs + b); };
    const Group* tab = reinterpret_cast<const Group*>(gbase + L::kTabOff);
    int* misc = reinterpret_cast<int*>(gbase + L::kMiscOff);
    volatile int* abort_flag = misc + 1;
    auto factors_at = [&](int b) { return reinterpret_cast<float*>(gbase + L::kGOff + b * L::kGSlot); };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int worker = blockIdx.x / L::kCtas;
    const int rank = kPair ? static_cast<int>(cluster_cta_rank()) : 0;
    const bool leader = rank == 0;
    const WaitCtl wc{p.timeout_ns, p.status, abort_flag};

    // Set-up under the end of the preceding grid; everything that touches
    // memory comes behind it (the offsets decide which weights are read).
    if (warp == kWarpProd && lane == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);    // the (leader's) producer; the pair's copies count on it
            mbar_init(empty(s), 1);   // commit: the unit's MMAs are complete
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(dfull(b), 2);                   // commit, and the factor warp
            mbar_init(dempty(b), kFold * L::kCtas);   // every fold warp: to the MMA issuer
            mbar_init(fempty(b), kFold);              // this CTA's: to its factor warp
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        __syncwarp();
        if constexpr (kPair) tmem_alloc_pair(smem_u32(misc), 512);
        else tmem_alloc(smem_u32(misc), 512);
    }
    grid_dependents_launch();
    grid_dependency_wait();
    if (warp == kWarpFactor)
        list_groups<NT>(p, reinterpret_cast<Group*>(gbase + L::kTabOff), misc + 2, misc + 3, lane);
    tc_fence_before();
    __syncwarp();
    if constexpr (kPair) cluster_sync_all();   // the peer's barriers are set up too
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const int groups = misc[2], tiles = misc[3];

    if (warp == kWarpProd) {
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), once = policy_evict_first();
            Ring<kStages> rs(0);
            Pl at;
            at.g = 0;
            int i = 0;
            bool ok = true;
            for (int t = worker; ok && t < tiles; t += p.workers) {
                at.enter(tab, groups, t, p.tn, rank);
                // a weight tile of several row tiles is read again soon
                const uint64_t pol_w = tab[at.g].rows > NT ? keep : once;
                const int wrow = at.expert * p.N + at.n0;
                const int xrow = at.row0 + (kPair ? rank * (at.width() >> 1) : 0);
                for (int ku = 0; ku < p.KU; ++ku, ++i, rs.step(1)) {
                    if (i >= kStages) {
                        ok = wait_bounded(empty(rs.slot), rs.phase ^ 1u, wc);
                        if (!ok) break;
                    }
                    if (blockIdx.x == 0 && i == p.fault_unit) continue;   // failure-path test hook
                    const uint32_t dst = base + rs.slot * L::kStage;
                    if (leader) mbar_arrive_expect_tx(full(rs.slot), L::kStage * L::kCtas);
                    const uint32_t bar = kPair ? map_to_cta(full(rs.slot), 0) : full(rs.slot);
#pragma unroll
                    for (int b = 0; b < kBlk; ++b) {   // a block past K reads as zeros
                        const int k0 = (ku * kBlk + b) * 128;
                        if constexpr (kPair) {
                            tma_load_2d_pair(dst + b * L::kWBox, &tmW, bar, k0, wrow, pol_w);
                            tma_load_2d_pair(dst + L::kXOff + b * L::kXBox, &tmX, bar, k0, xrow, keep);
                        } else {
                            tma_load_2d(dst + b * L::kWBox, &tmW, bar, k0, wrow, pol_w);
                            tma_load_2d(dst + L::kXOff + b * L::kXBox, &tmX, bar, k0, xrow, keep);
                        }
                    }
                }
            }
            // a unit whose MMAs are complete has its copies, and those before it
            // theirs; after a wait that gave up they may not run, and the drain
            // gives up as well
            if (i > 0) gemm::drain_wait(empty((i - 1) % kStages), ((i - 1) / kStages) & 1, p.timeout_ns);
        }
    } else if (warp == kWarpMma && leader) {
        const bool elected = elect_one();
        const uint64_t d0 = smem_desc_sw128(base);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if constexpr (kPair) return __all_sync(0xffffffffu, wait_bounded_cluster(bar, parity, wc)) != 0;
            else return gemm::warp_wait(bar, parity, wc);
        };
        auto commit = [&](uint32_t bar) {
            if constexpr (kPair) tc_commit_pair(bar, static_cast<uint16_t>(3u));
            else tc_commit(bar);
        };
        Ring<kStages> rs(0);
        Ring<kBufs> rb(0);
        Pl at;
        at.g = 0;
        int i = 0;
        bool ok = true;
        for (int t = worker; ok && t < tiles; t += p.workers) {
            at.enter(tab, groups, t, p.tn, rank);
            uint32_t idesc = idesc_f8_e4m3(at.width());
            if constexpr (kPair) idesc = (idesc & ~(31u << 24)) | (static_cast<uint32_t>(256 >> 4) << 24);
            for (int ku = 0; ku < p.KU; ++ku, ++i, rs.step(1), rb.step(1)) {
                ok = wait(full(rs.slot), rs.phase);
                if (ok && i >= kBufs) ok = wait(dempty(rb.slot), rb.phase ^ 1u);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = d0 + static_cast<uint64_t>((rs.slot * L::kStage) >> 4);
                const uint64_t bd = ad + static_cast<uint64_t>(L::kXOff >> 4);
                if (elected) {
#pragma unroll
                    for (int b = 0; b < kBlk; ++b) {
                        const uint32_t dt = tmem + (rb.slot * kBlk + b) * NT;
                        const uint64_t adb = ad + static_cast<uint64_t>((b * L::kWBox) >> 4);
                        const uint64_t bdb = bd + static_cast<uint64_t>((b * L::kXBox) >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (kPair) mma_ss_f8_pair(dt, adb + 2 * j, bdb + 2 * j, idesc, j > 0 ? 1u : 0u);
                            else mma_ss_f8(dt, adb + 2 * j, bdb + 2 * j, idesc, j > 0 ? 1u : 0u);
                        }
                    }
                    commit(empty(rs.slot));
                    commit(dfull(rb.slot));
                }
                __syncwarp();
            }
        }
        if (i > 0 && elected) gemm::drain_wait(empty((i - 1) % kStages), ((i - 1) / kStages) & 1, p.timeout_ns);
    } else if (warp == kWarpFactor) {
        // Lane l has columns l, l + 32, ... of the tile; their scales are fetched
        // kAhead units before they are used (a load takes longer than a unit).
        constexpr int kHeld = (kBlk * NT + 31) / 32;
        float held[kAhead][kHeld];
        float sw[kAhead][kBlk];
        Pl at;
        at.g = 0;
        int t = worker, ku = 0;
        bool live = t < tiles;
        if (live) at.enter(tab, groups, t, p.tn, rank);
        auto fetch = [&](float (&h)[kHeld], float (&w)[kBlk]) {
            if (!live) return;
            const float* srow = p.S + (static_cast<int64_t>(at.expert) * p.sn + at.nb) * p.KB;
#pragma unroll
            for (int b = 0; b < kBlk; ++b) {
                const int kb = ku * kBlk + b;
                w[b] = kb < p.KB && at.nb < p.sn ? __ldg(srow + kb) : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < kHeld; ++c) {
                const int col = c * 32 + lane;
                const int b = kBlk == 1 ? 0 : col / NT;
                const int j = kBlk == 1 ? col : col % NT;
                const int kb = ku * kBlk + b;
                h[c] = b < kBlk && kb < p.KB && j < at.rows
                           ? __ldcg(p.Sx + static_cast<int64_t>(kb) * p.ldsx + at.row0 + j)
                           : 0.0f;
            }
            if (++ku == p.KU) {
                ku = 0;
                t += p.workers;
                live = t < tiles;
                if (live) at.enter(tab, groups, t, p.tn, rank);
            }
        };
#pragma unroll
        for (int a = 0; a < kAhead; ++a) fetch(held[a], sw[a]);
        const int mine = worker < tiles ? (tiles - worker + p.workers - 1) / p.workers * p.KU : 0;
        Ring<kBufs> rb(0);
        bool ok = true;
        for (int i0 = 0; ok && i0 < mine; i0 += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int i = i0 + a;
                if (i >= mine) break;
                if (i >= kBufs) {
                    ok = gemm::warp_wait(fempty(rb.slot), rb.phase ^ 1u, wc);
                    if (!ok) break;
                }
                float* f = factors_at(rb.slot);
#pragma unroll
                for (int c = 0; c < kHeld; ++c) {
                    const int col = c * 32 + lane;
                    const int b = kBlk == 1 ? 0 : col / NT;
                    const int j = kBlk == 1 ? col : col % NT;
                    // in the order in which a fold lane reads them (fold below)
                    if (b < kBlk)
                        f[b * NT + (j & ~15) + ((j & 7) >> 1) * 4 + ((j >> 3) & 1) * 2 + (j & 1)] =
                            __fmul_rn(held[a][c], b == 0 ? sw[a][0] : sw[a][kBlk - 1]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(dfull(rb.slot));
                rb.step(1);
                fetch(held[a], sw[a]);
            }
        }
    } else if (warp >= kWarpFold0) {
        const int fw = warp - kWarpFold0;
        const int q = warp & 3;
        const int col0 = (fw >> 2) * kCols;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + col0;
        uint8_t* out = gbase + L::kOutOff + fw * L::kOutWarp;
        constexpr int kChunk = kCols < 32 ? kCols : 32;   // columns of a TMEM load
        Ring<kBufs> rb(0);
        Pl at;
        at.g = 0;
        bool ok = true;
        for (int t = worker; ok && t < tiles; t += p.workers) {
            at.enter(tab, groups, t, p.tn, rank);
            const int cols = at.width() - col0;   // of this warp that the MMA writes; <= 0: none
            float acc[2][kCols / 8][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < kCols / 8; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][g][e] = 0.0f;
            for (int ku = 0; ku < p.KU; ++ku, rb.step(1)) {
                ok = gemm::warp_wait(dfull(rb.slot), rb.phase, wc);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < kBlk; ++b) {
                    const float* f = factors_at(rb.slot) + b * NT + col0 + (lane & 3) * 4;
                    const uint32_t tb = tl + (rb.slot * kBlk + b) * NT;
#pragma unroll
                    for (int c = 0; c < kCols / kChunk; ++c) {
                        if (c * kChunk >= cols) break;
                        uint32_t v0[kChunk / 2], v1[kChunk / 2];
                        tmem_ld_frag(tb + c * kChunk, v0);
                        tmem_ld_frag(tb + (16u << 16) + c * kChunk, v1);
                        float4 g4[kChunk / 16];
#pragma unroll
                        for (int e = 0; e < kChunk / 16; ++e)
                            g4[e] = *reinterpret_cast<const float4*>(f + c * kChunk + e * 16);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < kChunk / 8; ++e) {
                            const float fa = e & 1 ? g4[e / 2].z : g4[e / 2].x;
                            const float fb = e & 1 ? g4[e / 2].w : g4[e / 2].y;
                            float* a0 = acc[0][c * (kChunk / 8) + e];
                            float* a1 = acc[1][c * (kChunk / 8) + e];
                            fma2(a0[0], a0[1], v0[4 * e], v0[4 * e + 1], fa, fb);
                            fma2(a0[2], a0[3], v0[4 * e + 2], v0[4 * e + 3], fa, fb);
                            fma2(a1[0], a1[1], v1[4 * e], v1[4 * e + 1], fa, fb);
                            fma2(a1[2], a1[3], v1[4 * e + 2], v1[4 * e + 3], fa, fb);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair && !leader) mbar_arrive_cluster(map_to_cta(dempty(rb.slot), 0));
                    else mbar_arrive(dempty(rb.slot));
                    mbar_arrive(fempty(rb.slot));
                }
            }
            if (!ok) break;
            // ------------------------------------------------ the tile's outputs
            const int nw = at.n0 + q * 32;          // the warp's first weight row
            const int rows = at.rows - col0;        // of this warp's columns that exist
            if (nw >= p.N || rows <= 0) continue;
            const int64_t r0 = at.row0 + col0;
            if (p.y_type == QG_FP32) {
                float* y = static_cast<float*>(p.Y) + r0 * p.ldy + nw + (lane >> 2);
#pragma unroll
                for (int g = 0; g < kCols / 8; ++g)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = 8 * g + 2 * (lane & 3) + (e & 1);
                        const int dn = 8 * (e >> 1);
                        if (j < rows && nw + dn + (lane >> 2) < p.N) y[j * p.ldy + dn] = acc[e >> 2][g][e & 3];
                    }
                continue;
            }
            // 16 bits: 16 rows of Y at a time through the warp's shared memory, as
            // [row][32 weight rows] with the 16-byte chunks of a row exchanged so
            // that neither side meets bank conflicts
            const uint32_t so = smem_u32(out);
            const uint32_t st_at = so + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
            for (int g = 0; g < kCols / 16; ++g) {
                if (16 * g >= rows) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float* a0 = acc[0][2 * g + e];
                    const float* a1 = acc[1][2 * g + e];
                    stmatrix_t4(st_at + e * 512, pack_out(a0[0], a0[1], p.y_type), pack_out(a0[2], a0[3], p.y_type),
                                pack_out(a1[0], a1[1], p.y_type), pack_out(a1[2], a1[3], p.y_type));
                }
                __syncwarp();
                if (p.y_vec) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = e * 8 + (lane >> 2);
                        const uint4 x = *reinterpret_cast<const uint4*>(out + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                        const int n = nw + (lane & 3) * 8;
                        if (16 * g + r < rows && n < p.N)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.Y) + (r0 + 16 * g + r) * p.ldy + n) = x;
                    }
                } else {
                    const int n = nw + lane;
#pragma unroll 1
                    for (int r = 0; r < 16 && 16 * g + r < rows; ++r)
                        if (n < p.N)
                            static_cast<uint16_t*>(p.Y)[(r0 + 16 * g + r) * p.ldy + n] = *reinterpret_cast<const uint16_t*>(
                                out + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
                }
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncwarp();
    // a pair leaves together: the leader's MMAs read both CTAs' operands, and
    // either's threads arrive on the other's barriers
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

__global__ void zero_group_rows_kernel(const int32_t* offsets, int E, int R, void* Y, int64_t ldy, int y_type, int N) {
    int rows = offsets[E];
    rows = rows > R ? R : rows;
    const int64_t total = rows > 0 ? static_cast<int64_t>(rows) * N : 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t at = t / N * ldy + t % N;
        if (y_type == QG_FP32) static_cast<float*>(Y)[at] = 0.0f;
        else static_cast<uint16_t*>(Y)[at] = 0;
    }
}

template <int NT, bool kPair>
cudaError_t launch_grouped_nt(const GroupedArgs& a, const CUtensorMap& tmW, const CUtensorMap& tmX, const LaunchCtl& c,
                              cudaStream_t st) {
    using L = GLayout<NT, kPair>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(configured, grouped_kernel<NT, kPair>, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    GParams p{};
    p.Sx = a.Sx;
    p.ldsx = a.ldsx;
    p.S = a.S;
    p.offsets = a.offsets;
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.y_type = a.y_type;
    p.y_vec = a.y_type != QG_FP32 && a.N % 8 == 0 && a.ldy % 8 == 0 && aligned_16(a.Y);
    p.R = a.R;
    p.E = a.E;
    p.N = a.N;
    p.KB = (a.K + 127) / 128;
    p.KU = (p.KB + L::kBlk - 1) / L::kBlk;
    p.sn = (a.N + 127) / 128;
    p.tn = (p.sn + L::kCtas - 1) / L::kCtas;
    p.workers = c.num_sms / L::kCtas;
    p.timeout_ns = c.timeout_ns;
    p.fault_unit = c.fault_unit;
    p.status = c.status;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.workers * L::kCtas));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (kPair) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, grouped_kernel<NT, kPair>, tmW, tmX, p);
}

}  // namespace

int grouped_tile_rows(int R, int E) {
    const int64_t mean = R / E;
    return mean <= 8 ? 16 : mean <= 48 ? 64 : 256;
}

size_t grouped_workspace_bytes(int R, int E, int sms) { return 0; }

cudaError_t launch_grouped(const GroupedArgs& a, const CUtensorMap& tmW, const CUtensorMap& tmX, const LaunchCtl& c,
                           cudaStream_t st) {
    switch (grouped_tile_rows(a.R, a.E)) {
        case 16: return launch_grouped_nt<16, false>(a, tmW, tmX, c, st);
        case 64: return launch_grouped_nt<64, false>(a, tmW, tmX, c, st);
        default: return launch_grouped_nt<256, true>(a, tmW, tmX, c, st);
    }
}

cudaError_t launch_grouped_zero(const GroupedArgs& a, cudaStream_t st) {
    zero_group_rows_kernel<<<304, 256, 0, st>>>(a.offsets, a.E, a.R, a.Y, a.ldy, a.y_type, a.N);
    return cudaGetLastError();
}

}  // namespace qg
