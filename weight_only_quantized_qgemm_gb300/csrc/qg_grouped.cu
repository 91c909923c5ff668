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
// Few rows an expert (W): a tile is 128 weight rows, on the MMA's M side, x up to NT
// rows of one expert on its N side, which is as wide as the tile's rows (rounded
// up to 16).  Columns of TMEM and of the activation boxes beyond them hold other
// rows' values, which nothing stores.  Bound by the weights' bytes: 64 tokens x 8 of
// 128 experts, 2048 x 5120, 174 us (7 TB/s of the experts that hold rows).
//
// Many rows (T): a tile is 256 rows of one expert on the M side of a CTA pair's
// MMAs x 256 weight rows.  A fold lane then is a row and needs one factor a K
// block; with the weights on the M side it needs a factor for each of its columns,
// whose way out of shared memory took longer than the MMAs.  The pair's MMAs of a K
// block take 512 cycles, a third of a unit's round of barriers beside them: MMAs,
// commit, fold (two waits, two loads of 64 columns, the products), release, the
// issuer's wait.  Two accumulators of 256 columns are all that TMEM holds, so the
// round sets the pace: 440 ns a unit at K = 16384, 2.9 PFLOP/s (at 456, 374 without
// the copies' power and traffic, 347 without the MMAs).
//
// Every CTA lists the experts that hold rows, with the tiles in front of each, at
// its start; workers then take tiles worker, worker + workers, ..., so that those
// in flight share an expert's weights and activations in L2.
//
// One persistent CTA (or pair) per SM; warps by role:
//   warp 0     producer: a unit's weight and activation boxes into one stage of
//              the ring, one barrier for all of them
//   warp 1     MMA issuer (T: warps 1 and 2 of the pair's first CTA take alternate
//              units; a K block is summed on its own, so that they need no order)
//   warp 3     the activation scales of a unit into a ring of their own
//   warps 4-   fold and epilogue: one per TMEM lane quadrant (T: two)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "qg_gemm.cuh"
#include "qg_grouped.h"
#include "qg_launch.h"
#include "qg_pair.cuh"

namespace qg {
namespace {

using gemm::Ring;

constexpr int kWarpProd = 0, kWarpMma = 1, kWarpScales = 3, kWarpFold0 = 4;
constexpr int kMaxExperts = QG_MAX_EXPERTS;

// The experts that hold rows (the groups), in order.  Their rows follow one
// another, so that a group ends where the next one begins: the entry behind the
// last says where the rows and the tiles end.
struct Groups {
    int2 at[kMaxExperts + 1];        // first row, tiles in front
    uint16_t expert[kMaxExperts];
    int count, tiles;
};

template <int NT, bool kPair>
struct GLayout {
    static constexpr int kCtas = kPair ? 2 : 1;
    // K blocks of 128 a unit: with narrow tiles a block's MMAs are short, and two
    // halve the barriers' share
    static constexpr int kBlk = kPair ? 1 : 2;
    static constexpr int kXRows = NT / kCtas;              // activation rows in this CTA's shared memory
    static constexpr int kWBox = 128 * 128;
    static constexpr int kXBlock = kXRows * 128;           // a K block's activations
    static constexpr int kXOff = kBlk * kWBox;             // in a stage, behind the weights
    static constexpr int kStage = kBlk * (kWBox + kXBlock);
    static constexpr int kFit = 512 / (kBlk * NT);
    static constexpr int kBufs = kFit < 4 ? kFit : 4;      // accumulator sets (kBlk x NT columns each)
    // MMA issuers, each with accumulator sets of its own (alternate units)
    static constexpr int kIssuers = kPair ? 2 : 1;
    static constexpr int kTabBytes = (sizeof(Groups) + 15) / 16 * 16;
    static constexpr int kFold = kPair ? 8 : 4;            // fold warps
    static constexpr int kCols = NT / (kFold / 4);         // columns of a fold warp
    static constexpr int kThreads = 32 * (kWarpFold0 + kFold);
    // The ring of activation scales: of a block, the tile's rows from a multiple of
    // four on (bulk copies start and end at 16 bytes)
    static constexpr int kSSlots = kPair ? 4 : 8;
    static constexpr int kSRow = (NT + 4) * 4;
    static constexpr int kSSlot = kBlk * kSRow;
    static constexpr int kOutWarp = (kPair ? 32 : 16) * 64;   // a fold warp's 32 (16) rows x 32 weight rows of 16 bits
    static constexpr int kSpots = 16;                      // places of tiles
    static constexpr int kFixed = kTabBytes + kSSlots * kSSlot + kFold * kOutWarp + kSpots * 16 + 512;
    static constexpr int kStages = (232448 - kFixed) / kStage / kIssuers * kIssuers;
    static constexpr int kTabOff = kStages * kStage;
    static constexpr int kSOff = kTabOff + kTabBytes;
    static constexpr int kOutOff = kSOff + kSSlots * kSSlot;
    static constexpr int kSpotOff = kOutOff + kFold * kOutWarp;
    static constexpr int kBarOff = kSpotOff + kSpots * 16;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 2 * kSSlots;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 32;
    static_assert(kSmemBytes <= 232448, "shared memory");
    static_assert(kBufs >= 2 && kBufs * kBlk * NT <= 512, "TMEM columns");
    static_assert(kXBlock % 1024 == 0 && kStage % 1024 == 0, "keep the 1024-byte swizzle alignment");
    static_assert(kCols % 16 == 0, "fragments");
    // the fold reads a tile's place and the next one's, the warp that writes them is up
    // to kSSlots tiles in front of it
    static_assert(kSpots >= kSSlots + 2, "places");
    // a set and a stage always belong to one issuer, whose parity waits are then for
    // the phase after one that it has seen
    static_assert(kBufs % kIssuers == 0 && kStages % kIssuers == 0, "ring ownership");
    static_assert(kSRow % 16 == 0 && kOutOff % 16 == 0 && kNumBars * 8 <= 512 - 32, "alignment, barriers");
};

struct GParams {
    const float* Sx;
    int64_t ldsx;
    const float* S;
    const int32_t* offsets;
    void* Y;
    int64_t ldy;
    int y_type;
    int y_word;       // bytes of the stores that N, ldy and Y allow: 16, 4 or 2
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

// 16 lanes x 4 C columns (C = 4 or 8 groups of four): lane t holds, of group j,
// column 4 j + t % 4 of rows t / 4 (v[2j]) and t / 4 + 8 (v[2j + 1]).  A lane so meets
// a quarter of the columns, and of their scales: with a row to a lane (32x32b)
// every lane reads all of them, and a K block of 256 columns takes eight warps
// 586 cycles; 463 this way, and 590 with 16x256b, which reads TMEM at half the rate.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
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

__device__ __forceinline__ void fma2(uint64_t& a, uint32_t v0, uint32_t v1, uint64_t f) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(a) : "r"(v0), "r"(v1), "l"(f));
}
__device__ __forceinline__ uint64_t twice(float f) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
    return r;
}

// Each thread of the warp reads 64 consecutive 32-bit columns of its own lane.
__device__ __forceinline__ void tmem_ld_x64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
        "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, "
        "%60, %61, %62, %63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed on the way: row j of matrix i
// goes to the address of lane 8 i + j.
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// Registers between the warpgroups of a block: every warp of one executes it.
template <int kRegs>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_fewer() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int y_type) {
    if (y_type == QG_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The way out of kRows rows of 64 bytes that a warp holds in shared memory, the 16-byte
// chunks of a row exchanged by (row / 2) % 4, so that neither side meets bank
// conflicts: the first `here` rows and `bytes` bytes of each, kWord at a time (a warp
// covers 64 bytes of 2 kWord / 4 rows a store), eight loads in front of their stores.
// (19 x 1024 rows, 512 x N, BF16: N = 2048 35 us, 2044 37, 2041 43; FP32 48, 50, 61.
// With a load and a multiplied address in front of each store of an element: 74.)
template <int kWord>
struct Word {
    using T = uint4;
};
template <>
struct Word<4> {
    using T = uint32_t;
};
template <>
struct Word<2> {
    using T = uint16_t;
};
template <int kWord, int kRows>
__device__ __forceinline__ void store_words(const uint8_t* from, uint8_t* y, int64_t pitch, int here, int bytes, int lane) {
    using T = typename Word<kWord>::T;
    constexpr int kLanes = 64 / kWord, kStep = 32 / kLanes, kTurns = kRows / kStep, kBatch = kTurns < 8 ? kTurns : 8;
    const int o = lane % kLanes * kWord, r0 = lane / kLanes;
    const int rows = o < bytes ? here : 0;
    uint8_t* to = y + r0 * pitch + o;
    pitch *= kStep;
#pragma unroll 1
    for (int t = 0; t < kTurns; t += kBatch) {
        T w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + (t + i) * kStep;
            w[i] = *reinterpret_cast<const T*>(from + r * 64 + (((o >> 4) ^ ((r >> 1) & 3)) << 4) + (o & 15));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (r0 + (t + i) * kStep < rows) *reinterpret_cast<T*>(to) = w[i];
            to += pitch;
        }
    }
}
template <int kRows>
__device__ __forceinline__ void store_rows16(int word, const uint8_t* from, uint8_t* y, int64_t pitch, int here, int bytes,
                                             int lane) {
    if (word == 16) store_words<16, kRows>(from, y, pitch, here, bytes, lane);
    else if (word == 4) store_words<4, kRows>(from, y, pitch, here, bytes, lane);
    else store_words<2, kRows>(from, y, pitch, here, bytes, lane);
}

// Bounded waits of this kernel.  The timer is read only once a wait has slept
// for 20 us, since most are short.  wait_on is for the fold, which a unit's chain
// of wait, loads, release bounds: no vote on the outcome, no call around which the
// sums would have to be saved.  A wait that gives up just returns, as does every
// later one; the sums are then worthless, and the tile loop ends.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort) return false;
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 0; it < (1u << 26); ++it) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (*c.abort) return false;
        if (globaltimer() - t0 > c.timeout_ns) break;
    }
    raise_abort(c, kDevTimeout);
    return false;
}
__device__ __forceinline__ bool warp_wait_here(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    return __all_sync(0xffffffffu, wait_here(bar, parity, c));
}
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, const WaitCtl& c) { wait_here(bar, parity, c); }
__device__ __forceinline__ bool aborted(const WaitCtl& c) { return __any_sync(0xffffffffu, *c.abort != 0); }

// One lane's arrival without a branch around it.
__device__ __forceinline__ void arrive_if(bool yes, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 st;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar),
                 "r"(static_cast<uint32_t>(yes))
                 : "memory");
}
// On a barrier of the pair's leader (a mapped address); it carries no memory, as
// mbar_arrive_cluster.
__device__ __forceinline__ void arrive_cluster_if(bool yes, uint32_t mapped) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(mapped),
                 "r"(static_cast<uint32_t>(yes))
                 : "memory");
}

// Where tile t lies.  The groups are in ascending order of their tiles.
template <int NT, int kCtas>
struct Place {
    int g;            // the group
    int expert;
    int row0, rows;   // of the tile
    bool several;     // the group has more row tiles than this
    int n0;           // first weight row of this CTA
    int nb;           // its block of 128 weight rows
    __device__ void enter(const Groups& tab, int t, int tn_count, int rank) {
        // the last group whose tiles begin at or before t
        int lo = g, hi = tab.count - 1;
        if (tab.at[lo + 1].y <= t) {
            ++lo;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tab.at[mid].y <= t) lo = mid;
                else hi = mid - 1;
            }
            g = lo;
        }
        const int2 q = tab.at[g];
        const int group_rows = tab.at[g + 1].x - q.x;
        expert = tab.expert[g];
        several = group_rows > NT;
        const int tm_count = (group_rows + NT - 1) / NT;
        const int j = t - q.y;
        const int tn = j / tm_count;   // a weight tile's row tiles are neighbours: its re-reads come from L2
        const int tm = j - tn * tm_count;
        row0 = q.x + tm * NT;
        rows = group_rows - tm * NT < NT ? group_rows - tm * NT : NT;
        nb = tn * kCtas + rank;
        n0 = nb * 128;
    }
    // The rows (of the tile's share of this CTA) whose scales it needs.
    __device__ void scale_rows(int rank, int R, int& first, int& count) const {
        first = row0;
        count = rows;
        if (kCtas == 2) {   // its half of a pair's tile, as far as the rows go
            first += rank * (NT / 2);
            count = R - first < NT / 2 ? (R > first ? R - first : 0) : NT / 2;
        }
    }
    // W: the MMA's N side
    __device__ int width() const { return (rows + 15) & ~15; }
};

// The table of the groups and the number of tiles, by one warp.  Offsets are
// taken as they are meant (ascending, from 0 to R); what breaks that is cut so
// that no row lies outside the tensors and none is in two groups.
template <int NT>
__device__ __forceinline__ void list_groups(const GParams& p, Groups& tab, int lane) {
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
            if (rows > 0) {
                const int i = ngroups + __popc(active & ((1u << lane) - 1u));
                tab.at[i] = make_int2(begin, ntiles + upto - mine);
                tab.expert[i] = static_cast<uint16_t>(e);
            }
            ngroups += __popc(active);
            ntiles += __shfl_sync(0xffffffffu, upto, 31);
            end_before = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    if (lane == 0) {
        tab.at[ngroups] = make_int2(end_before, ntiles);
        tab.count = ngroups;
        tab.tiles = ntiles;
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
    constexpr int kBarD = 2 * kStages;
    auto dfull = [&](int b) { return bar0 + 8u * (kBarD + b); };
    auto dempty = [&](int b) { return bar0 + 8u * (kBarD + kBufs + b); };
    auto sfull = [&](int s) { return bar0 + 8u * (kBarD + 2 * kBufs + s); };
    auto sempty = [&](int s) { return bar0 + 8u * (kBarD + 2 * kBufs + L::kSSlots + s); };
    Groups& tab = *reinterpret_cast<Groups*>(gbase + L::kTabOff);
    int* misc = reinterpret_cast<int*>(gbase + L::kMiscOff);
    volatile int* abort_flag = misc + 1;
    int4* spots = reinterpret_cast<int4*>(gbase + L::kSpotOff);   // first row, rows, expert, block of 128 weight rows
    auto scales_at = [&](int s) { return reinterpret_cast<const float*>(gbase + L::kSOff + s * L::kSSlot); };

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
            mbar_init(dfull(b), 1);                   // commit
            mbar_init(dempty(b), kFold * L::kCtas);   // every fold warp: to the MMA issuer
        }
        for (int s = 0; s < L::kSSlots; ++s) {
            mbar_init(sfull(s), 1);
            mbar_init(sempty(s), kFold);   // this CTA's
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
    if (warp == kWarpScales) {
        if (lane < L::kSpots) spots[lane] = make_int4(0, 0, 0, 0);   // valid for a fold that gave up waiting
        list_groups<NT>(p, tab, lane);
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (kPair) cluster_sync_all();   // the peer's barriers are set up too
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const int tiles = tab.tiles;

    if (warp < kWarpFold0) {
    // 128 outer sums a fold lane: of the launch's 384 x 168 registers, 256 x 224 +
    // 128 x 56
    if constexpr (kPair) {
        static_assert(L::kThreads == 384 && 256 * 224 + 128 * 56 <= 384 * 168, "registers");
        regs_fewer<56>();
    }
    if (warp == kWarpProd) {
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), once = policy_evict_first();
            Ring<kStages> rs(0);
            Pl at;
            at.g = 0;
            int i = 0;
            bool ok = true;
            for (int t = worker; ok && t < tiles; t += p.workers) {
                at.enter(tab, t, p.tn, rank);
                // a weight tile of several row tiles is read again soon
                const uint64_t pol_w = at.several ? keep : once;
                const int wrow = at.expert * p.N + at.n0;
                // a half of a pair's tile that holds no row: zeros from behind the last row,
                // which cost no traffic and little power (76 x 128 rows, 4096 x 8192: 487 us,
                // 458 with them)
                const int xrow = rank * L::kXRows < at.rows ? at.row0 + rank * L::kXRows : p.R;
                for (int ku = 0; ku < p.KU; ++ku, ++i, rs.step(1)) {
                    if (i >= kStages) {
                        ok = wait_here(empty(rs.slot), rs.phase ^ 1u, wc);
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
                            tma_load_2d_pair(dst + L::kXOff + b * L::kXBlock, &tmX, bar, k0, xrow, keep);
                        } else {
                            tma_load_2d(dst + b * L::kWBox, &tmW, bar, k0, wrow, pol_w);
                            tma_load_2d(dst + L::kXOff + b * L::kXBlock, &tmX, bar, k0, xrow, keep);
                        }
                    }
                }
            }
            // a unit whose MMAs are complete has its copies, and those before it
            // theirs; after a wait that gave up they may not run, and the drain
            // gives up as well
            if (i > 0) gemm::drain_wait(empty((i - 1) % kStages), ((i - 1) / kStages) & 1, p.timeout_ns);
        }
    } else if (warp < kWarpMma + L::kIssuers && leader) {
        const int issuer = warp - kWarpMma;
        constexpr uint32_t kDescT = (idesc_f8_e4m3(256) & ~(31u << 24)) | (static_cast<uint32_t>(256 >> 4) << 24);
        const bool elected = elect_one();
        const uint64_t d0 = smem_desc_sw128(base);
        auto commit = [&](uint32_t bar) {
            if constexpr (kPair) tc_commit_pair(bar, static_cast<uint16_t>(3u));
            else tc_commit(bar);
        };
        Ring<kStages> rs(issuer);
        Ring<kBufs> rb(issuer);
        Pl at;
        at.g = 0;
        int i = issuer, last = -1, ku = issuer;   // the unit, the last one issued, the unit's place in its tile
        bool ok = true;
        for (int t = worker; ok && t < tiles; t += p.workers) {
            if constexpr (!kPair) at.enter(tab, t, p.tn, rank);
            const uint32_t idesc = kPair ? kDescT : idesc_f8_e4m3(at.width());
            // the places in a stage of the operands of the M and the N side
            constexpr uint32_t m_off = kPair ? L::kXOff : 0, n_off = kPair ? 0 : L::kXOff;
            for (; ku < p.KU; ku += L::kIssuers, i += L::kIssuers, rs.step(L::kIssuers), rb.step(L::kIssuers)) {
                // On a pair, too, the arrivals carry no memory of the arriving threads
                // (TMA writes, which the MMA reads, and TMEM accesses ordered by
                // tcgen05.fence), so that the waits need no cluster scope.
                ok = warp_wait_here(full(rs.slot), rs.phase, wc);
                if (ok && i >= kBufs) ok = warp_wait_here(dempty(rb.slot), rb.phase ^ 1u, wc);
                if (!ok) break;
                tc_fence_after();
                const uint64_t stage = d0 + static_cast<uint64_t>((rs.slot * L::kStage) >> 4);
                if (elected) {
#pragma unroll
                    for (int b = 0; b < kBlk; ++b) {
                        const uint32_t dt = tmem + (rb.slot * kBlk + b) * NT;
                        // several blocks a unit: weights, then activations (W alone)
                        const uint64_t ad = stage + ((m_off + b * L::kWBox) >> 4);
                        const uint64_t bd = stage + ((n_off + b * L::kXBlock) >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (kPair) mma_ss_f8_pair(dt, ad + 2 * j, bd + 2 * j, idesc, j > 0 ? 1u : 0u);
                            else mma_ss_f8(dt, ad + 2 * j, bd + 2 * j, idesc, j > 0 ? 1u : 0u);
                        }
                    }
                    commit(dfull(rb.slot));
                    commit(empty(rs.slot));
                }
                __syncwarp();
                last = i;
            }
            ku -= p.KU;
        }
        if (last >= 0 && elected) gemm::drain_wait(empty(last % kStages), (last / kStages) & 1, p.timeout_ns);
    } else if (warp == kWarpScales) {
        // The scales of this CTA's rows of each unit, by bulk copies: loads to
        // registers, however far ahead, held up a warp's other waits (290 ns a unit).
        // And the tiles' places, which took the fold 1300 cycles a tile to work out (19 x
        // 1024 rows, 2048 x 512: 38.6 us, 35.2 this way; 64 x 60, 2048 x 1024: 33.5, 29.6).
        if (lane == 0) {
            const uint64_t keep = policy_evict_last();
            Ring<L::kSSlots> rs(0);
            Pl at;
            at.g = 0;
            int i = 0, n = 0;
            bool ok = true;
            for (int t = worker; ok && t < tiles; t += p.workers, ++n) {
                at.enter(tab, t, p.tn, rank);
                int first, rows;
                at.scale_rows(rank, p.R, first, rows);
                const float* from = p.Sx + (first & ~3);
                const uint32_t bytes = rows > 0 ? ((first & 3) + rows + 3) / 4 * 16 : 0;
                for (int ku = 0; ku < p.KU; ++ku, ++i, rs.step(1)) {
                    if (i >= L::kSSlots) {
                        ok = wait_here(sempty(rs.slot), rs.phase ^ 1u, wc);
                        if (!ok) break;
                    }
                    if (ku == 0) spots[n % L::kSpots] = make_int4(at.row0, at.rows, at.expert, at.nb);
                    const int nblk = kBlk == 1 || ku * kBlk + 2 <= p.KB ? kBlk : 1;
                    mbar_arrive_expect_tx(sfull(rs.slot), bytes * nblk);
                    for (int b = 0; b < nblk && bytes > 0; ++b)
                        bulk_load(base + L::kSOff + rs.slot * L::kSSlot + b * L::kSRow,
                                  from + static_cast<int64_t>(ku * kBlk + b) * p.ldsx, bytes, sfull(rs.slot), keep);
                }
            }
            // the copies of the last turn of the ring (earlier ones were waited for by the fold)
            for (int j = i > L::kSSlots ? i - L::kSSlots : 0; j < i; ++j)
                gemm::drain_wait(sfull(j % L::kSSlots), (j / L::kSSlots) & 1, p.timeout_ns);
        }
    }
    } else {
        if constexpr (kPair) regs_more<224>();
        const int fw = warp - kWarpFold0;
        const int q = warp & 3;
        const int g = fw >> 2;            // columns g kCols ..
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + g * kCols;
        uint8_t* out = gbase + L::kOutOff + fw * L::kOutWarp;
        constexpr int kChunk = kCols % 32 == 0 ? 32 : 16;   // columns of a TMEM load
        static_assert(kCols % kChunk == 0, "whole loads");
        Ring<kBufs> rb(0);
        Ring<L::kSSlots> rg(0);
        struct {
            int row0, rows, expert, nb;
            __device__ void enter(const int4& s) { row0 = s.x, rows = s.y, expert = s.z, nb = s.w; }
        } at{};
        int n = 0;   // tiles so far
        // W: [rows 0-15, 16-31][column group of 4][row, row + 8]; T: [column]
        float acc[kCols];
        const uint32_t to_issuer = kPair && !leader ? map_to_cta(dempty(0), 0) : dempty(0);
        auto release = [&]() {   // the accumulators have been read
            tc_fence_before();
            __syncwarp();
            if constexpr (kPair) arrive_cluster_if(lane == 0, to_issuer + 8u * rb.slot);
            else arrive_if(lane == 0, to_issuer + 8u * rb.slot);
        };
        // The weight scales of the tile's block of rows: lane l holds those of unit
        // u0 + l, of 32 units at a time, fetched 32 units (or an epilogue) ahead.
        float sw[kBlk], sw_next[kBlk];
        auto fetch = [&](int expert, int block, int u0) {
            int nb = kPair ? block - rank + g : block;
            nb = nb < p.sn ? nb : p.sn - 1;
            const float* from = p.S + (static_cast<int64_t>(expert) * p.sn + nb) * p.KB;
#pragma unroll
            for (int b = 0; b < kBlk; ++b) {
                const int kb = (u0 + lane) * kBlk + b;
                sw_next[b] = kb < p.KB ? __ldg(from + kb) : 0.0f;
            }
        };
        auto next_scales = [&](int ku) {   // at the beginning of a unit
            if ((ku & 31) == 0) {
#pragma unroll
                for (int b = 0; b < kBlk; ++b) sw[b] = sw_next[b];
                if (ku + 32 < p.KU) fetch(at.expert, at.nb, ku + 32);
            }
        };
        // a tile's place is there with the scales of its first unit
        auto fetch_tile = [&](int t) {
            if (t >= tiles) return;
            wait_on(sfull(rg.slot), rg.phase, wc);
            const int4 s = spots[n % L::kSpots];
            fetch(s.z, s.w, 0);
        };
        fetch_tile(worker);
        for (int t = worker; t < tiles && !aborted(wc); t += p.workers) {
            at.enter(spots[n % L::kSpots]);
            ++n;
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
            if constexpr (kPair) {
                // ------------------------------------------------ T: a lane is a row, with one factor a unit
                const int nb = at.nb - rank + g;   // the columns' block of weight rows
                uint64_t sums[kCols / 2];   // two columns each
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) sums[i] = 0ull;
                for (int ku = 0; ku < p.KU; ++ku, rb.step(1), rg.step(1)) {
                    next_scales(ku);
                    wait_on(sfull(rg.slot), rg.phase, wc);
                    const float f = __fmul_rn(scales_at(rg.slot)[(at.row0 & 3) + q * 32 + lane],
                                              __shfl_sync(0xffffffffu, sw[0], ku & 31));
                    __syncwarp();   // every lane has read its factor: a shuffle orders no memory
                    arrive_if(lane == 0, sempty(rg.slot));
                    const uint64_t f2 = twice(f);
                    wait_on(dfull(rb.slot), rb.phase, wc);
                    tc_fence_after();
                    // 64 columns a load: two are on their way by turns in the two warps of
                    // a scheduler (of 32, or the next one under the products, the sums
                    // spilled: 530 and 572 ns a unit against 456)
#pragma unroll
                    for (int c = 0; c < kCols / 64; ++c) {
                        uint32_t x[64];
                        tmem_ld_x64(tl + rb.slot * NT + c * 64, x);
                        tmem_wait_ld();
                        if (c + 1 == kCols / 64) release();   // ahead of the last products
#pragma unroll
                        for (int j = 0; j < 32; ++j) fma2(sums[c * 32 + j], x[2 * j], x[2 * j + 1], f2);
                    }
                }
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) {
                    acc[2 * i] = __uint_as_float(static_cast<uint32_t>(sums[i]));
                    acc[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(sums[i] >> 32));
                }
                fetch_tile(t + p.workers);
                // its columns: the 128 weight rows of block nb, in order
                const int n0 = nb * 128;
                const int here = at.rows - rank * 128 - q * 32;   // rows of this warp that exist
                if (n0 >= p.N || here <= 0) continue;
                // 64 bytes of a row at a time through the warp's shared memory (16-byte
                // chunks exchanged so that neither side meets bank conflicts), so that
                // a store covers whole sectors of eight rows (a lane's own row, 16 bytes
                // in each of 32 rows a store: 3.6 us a tile; this way 1.5)
                uint8_t* st = out + lane * 64;
                const int swap = (lane >> 1) & 3;
                const int64_t first_row = static_cast<int64_t>(at.row0) + rank * 128 + q * 32;
                const int left = p.N - n0 < 128 ? p.N - n0 : 128;
                if (p.y_type != QG_FP32) {
                    uint8_t* y = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.Y) + first_row * p.ldy + n0);
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float* v = acc + c + e * 8;
                            *reinterpret_cast<uint4*>(st + ((e ^ swap) << 4)) =
                                make_uint4(pack_out(v[0], v[1], p.y_type), pack_out(v[2], v[3], p.y_type),
                                           pack_out(v[4], v[5], p.y_type), pack_out(v[6], v[7], p.y_type));
                        }
                        __syncwarp();
                        store_rows16<32>(p.y_word, out, y + c * 2, p.ldy * 2, here, (left - c) * 2, lane);
                        __syncwarp();
                    }
                } else {
                    uint8_t* y = reinterpret_cast<uint8_t*>(static_cast<float*>(p.Y) + first_row * p.ldy + n0);
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(st + ((e ^ swap) << 4)) =
                                make_float4(acc[c + 4 * e], acc[c + 4 * e + 1], acc[c + 4 * e + 2], acc[c + 4 * e + 3]);
                        __syncwarp();
                        if (p.y_word == 16)
                            store_words<16, 32>(out, y + c * 4, p.ldy * 4, here, (left - c) * 4, lane);
                        else
                            store_words<4, 32>(out, y + c * 4, p.ldy * 4, here, (left - c) * 4, lane);
                        __syncwarp();
                    }
                }
            } else {
            // ---------------------------------------------------- W: a lane is a weight row
            const int cols = ((at.rows + 15) & ~15) - g * kCols;   // of this warp that the MMA writes; <= 0: none
            const int chunks = cols <= 0 ? 0 : cols >= kCols ? kCols / kChunk : (cols + kChunk - 1) / kChunk;
            for (int ku = 0; ku < p.KU; ++ku, rb.step(1), rg.step(1)) {
                next_scales(ku);
                wait_on(sfull(rg.slot), rg.phase, wc);
                wait_on(dfull(rb.slot), rb.phase, wc);
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < kBlk; ++b) {
                    // a column beyond the tile's rows takes whatever the slot holds
                    const float* f = scales_at(rg.slot) + b * (L::kSRow / 4) + (at.row0 & 3) + g * kCols + (lane & 3);
                    const float w = __shfl_sync(0xffffffffu, sw[b], ku & 31);
                    // the second block of a last unit may lie past K: 0, whatever the slot holds
                    const bool there = kBlk == 1 || ku * kBlk + b < p.KB;
                    const uint32_t tb = tl + (rb.slot * kBlk + b) * NT;
#pragma unroll
                    for (int c = 0; c < kCols / kChunk; ++c) {
                        if (c >= chunks) break;
                        uint32_t x[2][kChunk / 2];
                        tmem_ld_frag(tb + c * kChunk, x[0]);
                        tmem_ld_frag(tb + (16u << 16) + c * kChunk, x[1]);
                        float ff[kChunk / 4];
#pragma unroll
                        for (int e = 0; e < kChunk / 4; ++e) ff[e] = f[c * kChunk + e * 4];
                        tmem_wait_ld();
                        if (b == kBlk - 1 && c + 1 >= chunks) release();   // ahead of the last products
#pragma unroll
                        for (int e = 0; e < kChunk / 4; ++e) {
                            const float m = there ? __fmul_rn(ff[e], w) : 0.0f;
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float* o = acc + r * (kCols / 2) + 2 * (c * (kChunk / 4) + e);
                                fma2(o[0], o[1], x[r][2 * e], x[r][2 * e + 1], m, m);
                            }
                        }
                    }
                }
                if (chunks == 0) release();
                __syncwarp();
                arrive_if(lane == 0, sempty(rg.slot));   // the scales have been read, too
            }
            fetch_tile(t + p.workers);
            const int nw = at.nb * 128 + q * 32;    // the warp's first weight row
            const int rows = at.rows - g * kCols;   // of this warp's columns that exist
            if (nw >= p.N || rows <= 0) continue;
            {
                const int64_t r0 = at.row0 + g * kCols;
                // (row group r, column group j)
                auto sum = [&](int r, int j) { return acc + r * (kCols / 2) + 2 * j; };
                if (p.y_type == QG_FP32) {
                    float* y = static_cast<float*>(p.Y) + r0 * p.ldy + nw + (lane >> 2);
#pragma unroll
                    for (int j4 = 0; j4 < kCols / 4; ++j4) {
                        const int j = 4 * j4 + (lane & 3);
                        if (4 * j4 >= rows) break;
                        if (j < rows) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (nw + 8 * e + (lane >> 2) < p.N) y[j * p.ldy + 8 * e] = sum(e >> 1, j4)[e & 1];
                        }
                    }
                    continue;
                }
                // 16 bits: 16 rows of Y at a time through the warp's shared memory, as
                // [row][32 weight rows] with the 16-byte chunks of a row exchanged so
                // that neither side meets bank conflicts.  Columns 2 c and 2 c + 1 of a
                // lane's 8 x 8 matrices are rows c and c + 4 of the eight.
                const int mrow = ((lane & 7) >> 1) + (lane & 1) * 4;
                const uint32_t st_at = smem_u32(out) + mrow * 64 + (((lane >> 3) ^ ((mrow >> 1) & 3)) << 4);
#pragma unroll
                for (int j16 = 0; j16 < kCols / 16; ++j16) {
                    if (16 * j16 >= rows) break;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float *a0 = sum(0, 4 * j16 + 2 * e), *a1 = a0 + 2;
                        const float *b0 = sum(1, 4 * j16 + 2 * e), *b1 = b0 + 2;
                        stmatrix_t4(st_at + e * 512, pack_out(a0[0], a1[0], p.y_type), pack_out(a0[1], a1[1], p.y_type),
                                    pack_out(b0[0], b1[0], p.y_type), pack_out(b0[1], b1[1], p.y_type));
                    }
                    __syncwarp();
                    store_rows16<16>(p.y_word, out,
                                     reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.Y) + (r0 + 16 * j16) * p.ldy + nw),
                                     p.ldy * 2, rows - 16 * j16, (p.N - nw < 32 ? p.N - nw : 32) * 2, lane);
                    __syncwarp();
                }
            }
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

// Zeros in the rows of the groups, which follow one another: from the first offset to
// the largest, cut as list_groups cuts them.
__global__ void zero_group_rows_kernel(const int32_t* offsets, int E, int R, void* Y, int64_t ldy, int y_type, int N) {
    __shared__ int last;
    int first = offsets[0];
    first = first < 0 ? 0 : first > R ? R : first;
    if (threadIdx.x == 0) last = first;
    __syncthreads();
    for (int e = 1 + static_cast<int>(threadIdx.x); e <= E; e += static_cast<int>(blockDim.x)) {
        const int end = offsets[e];
        atomicMax(&last, end > R ? R : end);
    }
    __syncthreads();
    Y = static_cast<uint8_t*>(Y) + first * ldy * (y_type == QG_FP32 ? 4 : 2);
    const int64_t total = static_cast<int64_t>(last - first) * N;
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
    const int64_t size = a.y_type == QG_FP32 ? 4 : 2;
    const uint64_t all = static_cast<uint64_t>(a.N * size) | static_cast<uint64_t>(a.ldy * size) | reinterpret_cast<uintptr_t>(a.Y);
    p.y_word = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 2;
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

// The host knows R and E, not the groups: experts of about R / E rows each, the last
// tile of a group half full.  Narrow tiles fold fewer columns that hold nothing and
// fill the SMs with few rows, wide ones read a large group's weights fewer times,
// and the pair's have the quickest K blocks and the longest epilogue, on 256 weight
// rows.  A tile's time is K blocks times `block` and `ends` beside them (us); waves count
// half as whole ones, since unlike tiles even out.  The figures are fitted to 120
// shapes in all four forms (R 2 to 65536, 2 to 256 experts, N 65 to 8000, K 128 to
// 7100) with 14 % of scatter; chosen by them, those take 0.2 % more time than with the best
// of the four for each, and 220 other shapes 0.6 % (by the mean number of rows
// alone, 10 / 20 / 52: 2.6 and 4.5 %; with the places worked out by the scales' warp
// since then, 0.5 and 0.7 %).  Of the unlike sides, us for 16 / 32 / 64 / 256:
//   64 experts, 4096 x 2048:   8 rows 81 / 81 / 82 / 114, 24 rows 111 / 92 / 89 / 117, 96
//   rows 312 / 210 / 177 / 132;  21 experts of 46 rows, 337 x 5072: 23 / 15 / 19 / 24;
//   3 of 480, 216 x 2240: - / 9 / 11 / 15
int grouped_tile_rows(int R, int E, int N, int K, int sms) {
    struct Form {
        int rows, channels;
        double block, ends;
    };
    constexpr Form kForms[] = {{16, 128, 0.21, 1.0}, {32, 128, 0.20, 1.5}, {64, 128, 0.30, 1.5}, {256, 256, 0.37, 3.4}};
    const double groups = R < E ? R : E;
    const int blocks = (K + 127) / 128;
    int best = 0;
    double least = 0.0;
    for (const Form& f : kForms) {
        const double tn = (static_cast<int64_t>(N) + f.channels - 1) / f.channels;
        const bool several = 2 * static_cast<int64_t>(R) > static_cast<int64_t>(f.rows) * E;
        const double tiles = tn * (several ? R / static_cast<double>(f.rows) + 0.5 * groups : groups);
        const double x = tiles / (sms * 128 / f.channels);
        const double waves = x <= 1.0 ? 1.0 : 0.5 * (x + std::ceil(x));
        const double us = waves * (blocks * f.block + f.ends);
        if (best == 0 || us < least) {
            best = f.rows;
            least = us;
        }
    }
    return best;
}

cudaError_t launch_grouped(const GroupedArgs& a, const CUtensorMap& tmW, const CUtensorMap& tmX, const LaunchCtl& c,
                           cudaStream_t st) {
    switch (grouped_tile_rows(a.R, a.E, a.N, a.K, c.num_sms)) {
        case 16: return launch_grouped_nt<16, false>(a, tmW, tmX, c, st);
        case 32: return launch_grouped_nt<32, false>(a, tmW, tmX, c, st);
        case 64: return launch_grouped_nt<64, false>(a, tmW, tmX, c, st);
        default: return launch_grouped_nt<256, true>(a, tmW, tmX, c, st);
    }
}

cudaError_t launch_grouped_zero(const GroupedArgs& a, cudaStream_t st) {
    zero_group_rows_kernel<<<304, 256, 0, st>>>(a.offsets, a.E, a.R, a.Y, a.ldy, a.y_type, a.N);
    return cudaGetLastError();
}

}  // namespace qg
