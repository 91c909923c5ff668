// 8-bit integer GEMM with one scale per token and per channel, and the
// activation quantiser in front of it, for sm_103a.
//
//   Y[m, n] = sx[m] * sw[n] * sum_k xq[m, k] * w[n, k] (+ bias[n])
//
// sm_103a has no integer kind of tcgen05.mma, so the products run as
// kind::f16: every value of -128..127 is an FP16 number, every product an
// integer of at most 2^14, and the FP32 accumulator adds integers exactly
// while the partial sums stay below 2^24 (always for K <= 1024; codes of mixed
// signs stay there far longer).  Beyond, every 16 products drop what lies under
// the accumulator's last place: measured 1.7e-5 of a sum of 17408 products of
// one sign and 5.2e-5 of 65536, under half a step of the 16-bit outputs (2^-9
// and 2^-12 of the value).  The floor is therefore the FP16 tensor rate for large M and
// the weight bytes, read once as stored, for small M.
//
// What bounds small M is the stream of weights, with 4 to 5 us of start and end
// around it: 16 x 17408 x 5120 takes 19 us, 14.5 of them at 6.1 TB/s.  Neither the
// MMAs nor the conversion does (one MMA a unit in place of eight: 19.1 -> 18.8 us,
// twice as many 19.9; four convert groups in place of two: 19.5 -> 20.0).
//
// The output is tiled in 128 weight rows x NA activation rows (NA = the MMA's
// N side); a unit is one tile x one 128-wide K block.  Weights stay 8-bit up
// to the SM: TMA brings a unit's 128 x 128 bytes into a shared-memory ring
// (128-byte swizzle), the convert warps turn each row's bytes into FP16 in
// registers (XOR 0x80, a byte permute under the exponent of 1024, one packed
// subtract: five instructions for four values) and store them to TMEM, from
// where the MMA takes its A operand.  Activations are expanded to FP16 once
// per call by a small kernel in front (they are read by every weight tile;
// converting them in each CTA would cost NA/128 of the weight conversion and
// twice the shared memory traffic) and arrive by TMA as the B operand.  Up to
// 16 rows two warps of the GEMM expand them instead, which saves a launch.
//
// One persistent CTA per SM; warps by role:
//   warp 0        weight producer (TMA, one 16 KB box per unit)
//   warp 1        activation producer (TMA, two boxes of 64 K x NA rows a unit),
//                 after the expansion kernel's completion; up to 16 rows warps 1
//                 and 3 load and expand the codes themselves
//   warp 2        MMA issuer: 8 tcgen05.mma (M = 128, N = NA, K = 16) a unit
//   warps 4-      epilogue: one per TMEM lane quadrant (two for NA >= 128)
//   the last 8    convert: two groups of four warps taking alternate units
//
// Each worker (a CTA, or beyond 128 rows a pair of them) first runs the same
// number of whole tiles, the workers side by side so that the tiles in flight
// share their operands in L2; the tiles that are left are cut over the workers
// at any K block, and a tile shared by several is summed, in ascending K order
// of its pieces, by the last to arrive, as in the other kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_gemm.cuh"
#include "qg_int8.h"
#include "qg_launch.h"
#include "qg_pair.cuh"

namespace qg {
namespace {

using gemm::Cursor;
using gemm::Params;
using gemm::Ring;

constexpr int kWarpWProd = 0, kWarpXProd = 1, kWarpMma = 2, kWarpX2 = 3, kWarpEpi0 = 4;
constexpr int kGroups = 2;   // convert groups of four warps
constexpr int kMostPieces = 8;   // equal pieces of a tile in a cluster
constexpr int kMostSplit = 16;   // pieces of a tile summed through the workspace

// NA activation rows a tile; kPair: a tile is 256 weight rows on a CTA pair.
template <int NA, bool kPair>
struct I8Layout {
    static constexpr int kCtas = kPair ? 2 : 1;
    // up to 16 rows the activations are expanded in the kernel (warps 1 and 3,
    // alternate units); beyond, by the kernel in front (at 32 rows the two
    // warps set the pace: 43.7 us against 34.5 on 32 x 32768 x 5120; four took 37.9
    // against 32.5, and eight at 64 rows 29.7 against 21.4 on 64 x 17408 x 5120)
    static constexpr bool kInlineX = NA <= 16;
    static constexpr int kXChunks = NA * 8 / 32;                // a lane's 16-byte pieces of a unit's codes
    static constexpr int kEpi = NA >= 128 ? 8 : 4;
    static constexpr int kEpiCols = NA / (kEpi / 4);            // columns per epilogue warp
    static constexpr int kWarpConv0 = kWarpEpi0 + kEpi;
    static constexpr int kThreads = 32 * (kWarpConv0 + 4 * kGroups);
    // slices of an epilogue warp's columns that the CTAs of a split tile sum
    static constexpr int kSlices = kPair ? kInt8Slices : 1;
    static constexpr int kSliceCols = kEpiCols / kSlices;
    // per epilogue warp, the activation scales of the columns at hand
    static constexpr int kScaleCols = kEpiCols < 64 ? kEpiCols : 64;
    static constexpr int kWBytes = 128 * 128;
    // The operand ring: a slot holds one unit's activations in shared memory
    // (two boxes of 64 K); the unit's A buffer in TMEM (64 columns) is one of
    // kABufs taken in turn.  One barrier of the slot says that both are there,
    // one that the unit's MMAs have read them, so that the MMA warp passes one
    // wait and one commit per unit: each costs it 0.05 to 0.1 us even when
    // nothing is late (with separate rings, three waits and three commits a
    // unit, gate/up at 16 rows took 28.0 us).  More slots than A buffers where
    // they fit: a copy of activations takes most of a microsecond, and with
    // four slots that set the pace of a CTA (0.3 us a unit).
    static constexpr int kABufs = 4;
    static constexpr int kSlots = NA <= 32 ? 8 : NA <= 128 ? 6 : 4;
    static constexpr int kXRows = NA / kCtas;                   // of the tile, in this CTA's shared memory
    static constexpr int kXBox = kXRows * 128;
    static constexpr int kXSlot = 2 * kXBox;
    static constexpr int kWFit = (232448 - 512 - kEpi * kScaleCols * 4 - kSlots * kXSlot) / kWBytes;
    static constexpr int kWStages = (kWFit < 12 ? kWFit : 12) / kGroups * kGroups;
    static constexpr int kD = NA > 128 ? 1 : 2;                 // accumulators, NA columns each
    static constexpr int kDCol0 = kABufs * 64;
    static constexpr int kXOff = kWStages * kWBytes;
    static constexpr int kBarOff = kXOff + kSlots * kXSlot;
    static constexpr int kNumBars = 2 * kWStages + 2 * kSlots + 2 * kD;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kScaleOff = (kMiscOff + 16 + 15) / 16 * 16;
    static constexpr int kSmemBytes = kScaleOff + kEpi * kScaleCols * 4;
    static_assert(kDCol0 + kD * NA <= 512, "TMEM columns");
    static_assert(kSmemBytes <= 232448, "shared memory");
    static_assert(kXBox % 1024 == 0, "keep the 1024-byte swizzle alignment");
    // a weight stage, a slot and an A buffer always belong to one convert
    // group, so that its parity waits are for the phase after one it has seen
    static_assert(kWStages % kGroups == 0 && kSlots % kGroups == 0 && kABufs % kGroups == 0, "ring ownership");
    static_assert(kSlots >= kABufs, "a unit's A buffer is free once the unit kABufs before it is done");
    static_assert(kEpiCols % 16 == 0, "epilogue chunks");
};

struct Out {
    const int8_t* xq;
    int64_t ldxq;
    const float* sx;
    const float* sw;
    const float* bias;
    int y_type;
    int y_pairs;    // a 16-bit Y that takes 32-bit stores of two neighbouring columns
    int tn_count, tm_count;   // weight tiles, activation row blocks
    int workers;              // CTAs or CTA pairs
    int nfull;                // whole tiles each worker runs before its part of the tail
    int pieces;               // kClu: the workers that share a tile
    int early;                // weights may be read before the preceding grid is done
    int tail_q, tail_r;       // the tail's units = tail_q G + tail_r
    // where worker c's part of the tail begins: floor(c U / G), in 32 bits
    __device__ int tail_begin(const Params& p, int c) const { return c * tail_q + c * tail_r / p.G; }
};

// Where tile t lies: bands of kBand activation row blocks, in a band weight
// tile by weight tile.  The tiles in flight at a time then share a few weight
// tiles and one band of activations, which L2 holds.
constexpr int kBand = 16;
__device__ __forceinline__ void place_of(const Out& o, int t, int& tn, int& tm) {
    const int band = t / (o.tn_count * kBand);
    const int r = t - band * o.tn_count * kBand;
    int width = o.tm_count - band * kBand;
    width = width > kBand ? kBand : width < 1 ? 1 : width;   // < 1: a place past the last tile, not used
    tn = r / width;
    tm = band * kBand + r - tn * width;
}

// A worker's units in order: whole tiles worker, worker + workers, ... (nfull
// of them), then units [u0, u1) of the tail, the tiles from nfull * workers on,
// which are cut over the tail's workers (Params U and G) at any K block.  kr is
// the K block a unit covers: tiles start at different ones (see Cursor).
struct Walk {
    int tile, kb, kr, tn, tm;
    int full;                 // whole tiles left, this one included; 0 in the tail
    int tail_tile, tail_kb;
    __device__ Walk(const Params& p, const Out& o, int worker, int u0)
        : full(o.nfull), tail_tile(o.nfull * o.workers + u0 / p.KB), tail_kb(u0 % p.KB) {
        if (full > 0) enter(p, o, worker, 0);
        else enter(p, o, tail_tile, tail_kb);
    }
    __device__ void enter(const Params& p, const Out& o, int t, int k) {
        tile = t;
        kb = k;
        kr = k + Cursor::first_block(t, p.KB);
        if (kr >= p.KB) kr -= p.KB;
        place_of(o, t, tn, tm);
    }
    __device__ void step(const Params& p, const Out& o) {
        if (++kr == p.KB) kr = 0;
        if (++kb < p.KB) return;
        if (full > 1) {
            --full;
            enter(p, o, tile + o.workers, 0);
        } else if (full == 1) {
            full = 0;
            enter(p, o, tail_tile, tail_kb);
        } else {
            enter(p, o, tile + 1, 0);
        }
    }
};

// Four signed bytes of w -> two FP16x2 words, exactly: u = byte + 128 under
// the exponent of 1024 is 1024 + u, minus 1152 is the byte's value.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = prmt(u, 0x64646464u, 0x4140u);
    const uint32_t b = prmt(u, 0x64646464u, 0x4342u);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// 16 accumulators of one weight row (activation rows in order), scaled.
__device__ __forceinline__ void scale16(const float (&v)[16], const float* sx, float sw, float b, float* y) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float4 s = reinterpret_cast<const float4*>(sx)[g];
        y[4 * g + 0] = __fmaf_rn(__fmul_rn(v[4 * g + 0], s.x), sw, b);
        y[4 * g + 1] = __fmaf_rn(__fmul_rn(v[4 * g + 1], s.y), sw, b);
        y[4 * g + 2] = __fmaf_rn(__fmul_rn(v[4 * g + 2], s.z), sw, b);
        y[4 * g + 3] = __fmaf_rn(__fmul_rn(v[4 * g + 3], s.w), sw, b);
    }
}

// The same as 16-bit values, two activation rows to a word.
__device__ __forceinline__ void pack16(const float (&v)[16], const float* sx, float sw, float b, int y_type,
                                       uint32_t* w) {
    float y[16];
    scale16(v, sx, sw, b, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (y_type == QG_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(y[2 * j], y[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
}

// Stores COLS packed columns (activation rows m0 ..) of weight row n.  pairs:
// two neighbouring weight rows to a 32-bit store: of activation rows m and
// m + 1 the even lane of a pair writes (n, n + 1) of row m and the odd lane
// (n - 1, n) of row m + 1, which halves the stores of a tile.  It needs an even
// N and row stride and a 4-byte aligned Y; else every value is a store.
template <int COLS>
__device__ __forceinline__ void store_packed(const Params& p, bool pairs, int n, int m0, const uint32_t* w) {
    const int64_t ldy = p.seg[0].ldy;
    if (pairs) {
        const int odd = threadIdx.x & 1;
        const uint32_t sel = odd ? 0x3276u : 0x5410u;
        uint16_t* at = static_cast<uint16_t*>(p.seg[0].Y) + (static_cast<int64_t>(m0) + odd) * ldy + (n - odd);
        const int rows = n < p.N ? p.M - m0 - odd : 0;   // of this lane's
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 1);
            if (2 * j < rows) *reinterpret_cast<uint32_t*>(at) = prmt(w[j], other, sel);
            at += 2 * ldy;
        }
        return;
    }
    uint16_t* at = static_cast<uint16_t*>(p.seg[0].Y) + static_cast<int64_t>(m0) * ldy + n;
    const int rows = n < p.N ? p.M - m0 : 0;
#pragma unroll
    for (int j = 0; j < COLS / 2; ++j) {
        if (2 * j < rows) *at = static_cast<uint16_t>(w[j]);
        if (2 * j + 1 < rows) at[ldy] = static_cast<uint16_t>(w[j] >> 16);
        at += 2 * ldy;
    }
}

// Stores COLS 32-bit columns (activation rows m0 ..) of weight row n.
template <int COLS>
__device__ __forceinline__ void store_f32(const Params& p, int n, int m0, const float* y) {
    const int64_t ldy = p.seg[0].ldy;
    float* at = static_cast<float*>(p.seg[0].Y) + static_cast<int64_t>(m0) * ldy + n;
    const int rows = n < p.N ? p.M - m0 : 0;
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
        if (j < rows) *at = y[j];
        at += ldy;
    }
}

// 16 output columns (activation rows m0 ..) of weight row n; sx: their scales
// in shared memory.
__device__ __forceinline__ void store16(const Params& p, const Out& o, int n, int m0, const float* sx, float sw, float b,
                                        const float (&v)[16]) {
    if (o.y_type != QG_FP32) {
        uint32_t w[8];
        pack16(v, sx, sw, b, o.y_type, w);
        store_packed<16>(p, o.y_pairs, n, m0, w);
        return;
    }
    float y[16];
    scale16(v, sx, sw, b, y);
    store_f32<16>(p, n, m0, y);
}

template <int NA>
__device__ __forceinline__ float4* part_slot(const Params& p, int cta, int which) {
    return reinterpret_cast<float4*>(p.part) + (static_cast<size_t>(cta) * 2 + which) * (NA / 4) * 128;
}

// Stores and loads of the partial sums that the CTAs of a cluster exchange.
__device__ __forceinline__ void st_cluster(uint32_t mapped, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mapped), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

// kClu: o.pieces workers (CTAs or pairs) of one cluster run equal pieces of a
// tile's K range and sum them through distributed shared memory.
template <int NA, bool kPair, bool kClu>
__global__ void __launch_bounds__(I8Layout<NA, kPair>::kThreads, 1)
    int8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p,
                const Out o) {
    using L = I8Layout<NA, kPair>;
    constexpr int kWStages = L::kWStages, kSlots = L::kSlots, kABufs = L::kABufs, kD = L::kD;
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_u32(gbase);
    if (base & 1023u) {   // the swizzle needs the alignment asked for above
        if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
        return;
    }

    const uint32_t bar0 = base + L::kBarOff;
    auto wfull = [&](int s) { return bar0 + 8u * s; };
    auto wempty = [&](int s) { return bar0 + 8u * (kWStages + s); };
    auto ofull = [&](int a) { return bar0 + 8u * (2 * kWStages + a); };
    auto ofree = [&](int a) { return bar0 + 8u * (2 * kWStages + kSlots + a); };
    constexpr int kBarD = 2 * kWStages + 2 * kSlots;
    auto dfull = [&](int b) { return bar0 + 8u * (kBarD + b); };
    auto dempty = [&](int b) { return bar0 + 8u * (kBarD + kD + b); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMiscOff + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    // the units of a worker: a CTA, or a pair (both CTAs walk the same ones)
    const int worker = cta / L::kCtas;
    const uint32_t crank = kPair || kClu ? cluster_cta_rank() : 0u;
    const uint32_t rank = kPair ? crank & 1u : 0u;   // in the pair
    const uint32_t lead = crank - rank;       // the pair's leader's place in the cluster
    const bool leader = rank == 0;
    int u0, u1;
    if constexpr (kClu) {
        const int tile = worker / o.pieces, piece = worker - tile * o.pieces;
        u0 = tile * p.KB + piece * p.KB / o.pieces;
        u1 = tile * p.KB + (piece + 1) * p.KB / o.pieces;
    } else {
        u0 = worker < p.G ? o.tail_begin(p, worker) : 0;
        u1 = worker < p.G ? o.tail_begin(p, worker + 1) : 0;
    }
    const int nunits = o.nfull * p.KB + u1 - u0;
    const WaitCtl wc{p.timeout_ns, p.status, abort_flag};

    // The kernel may start long before the preceding grid is done.  Every warp
    // waits for that before its first bounded wait for what comes behind it, so
    // that the preceding grid's time does not count against the limit.
    if (warp == kWarpWProd) {
        // Sets the barriers up, announces them and starts the weight stream at
        // once: it needs nothing else of the CTA's set-up (with the first turn
        // of the ring ahead of the CTA's meeting the other warps met 2.7 us
        // after the launch, now 1 us).
        if (lane == 0) {
            prefetch_tmap(&tmW);
            for (int s = 0; s < kWStages; ++s) {
                mbar_init(wfull(s), 1);
                mbar_init(wempty(s), 4);   // the four warps of the convert group
            }
            for (int a = 0; a < kSlots; ++a) {
                // each CTA's four convert warps, and the activations' copies (the
                // leader's barrier counts for the pair)
                mbar_init(ofull(a), 4 * L::kCtas + 1);
                mbar_init(ofree(a), 1);    // commit
            }
            for (int b = 0; b < kD; ++b) {
                mbar_init(dfull(b), 1);    // commit: the piece's MMAs are complete
                mbar_init(dempty(b), L::kEpi * L::kCtas);
            }
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        if constexpr (kPair || kClu) cluster_arrive_all();
        else named_bar_arrive(1, L::kThreads);
        grid_dependents_launch();
        // a weight tile serves tm_count tiles: keep it for their re-reads
        const uint64_t pol = o.tm_count > 1 ? policy_evict_last() : policy_evict_first();
        auto skipped = [&](int i) { return cta == 0 && i == p.fault_unit; };   // failure-path test hook
        Walk cur(p, o, worker, u0);
        Ring<kWStages> rw(0);
        int issued = 0;
        // without an expansion kernel in front the preceding grid may still be
        // writing the weights, unless the caller says it does not
        if (L::kInlineX && !o.early) grid_dependency_wait();
        auto load_w = [&]() {
            if (skipped(issued)) return;
            mbar_arrive_expect_tx(wfull(rw.slot), L::kWBytes);
            tma_load_2d(base + rw.slot * L::kWBytes, &tmW, wfull(rw.slot), cur.kr * 128,
                        (cur.tn * L::kCtas + static_cast<int>(rank)) * 128, pol);
        };
        // The first kFirst copies, and the ring's others once the first has landed:
        // with all of every CTA's on the way at once, some CTAs waited 6 us for
        // their first unit, and a CTA is no faster than memory, so that they ended
        // last (16 x 6144 x 5120 12.1 -> 10.8 us, 64 x 5120 x 17408 26.4 -> 25.0; with
        // 3, 6 or 8 the same within 3%).
        constexpr int kFirst = 4;
        if (lane == 0)
            for (; issued < nunits && issued < kWStages; ++issued, cur.step(p, o), rw.step(1)) {
                if (issued == kFirst && !wait_bounded(wfull(0), 0, wc)) break;
                load_w();
            }
        __syncwarp();
        if constexpr (kPair || kClu) cluster_wait_all();   // of the arrival above
        if (lane == 0) {
            for (; issued < nunits; ++issued, cur.step(p, o), rw.step(1)) {
                // the first stage that an MMA has to free, through an A buffer
                if (issued == kWStages + kABufs) grid_dependency_wait();
                if (!wait_bounded(wempty(rw.slot), rw.phase ^ 1u, wc)) break;
                load_w();
            }
            for (int i = issued - kWStages < 0 ? 0 : issued - kWStages; i < issued; ++i)
                if (!skipped(i)) gemm::drain_wait(wfull(i % kWStages), (i / kWStages) & 1, p.timeout_ns);
        }
    } else {
        if (warp == kWarpMma) {
            if constexpr (kPair) tmem_alloc_pair(smem_u32(tmem_slot), 512);
            else tmem_alloc(smem_u32(tmem_slot), 512);
        }
        if (!L::kInlineX && warp == kWarpXProd && lane == 0) prefetch_tmap(&tmX);
        tc_fence_before();
        __syncwarp();
        if constexpr (kPair || kClu) cluster_sync_all();   // the peer's barriers are set up too
        else named_bar_sync(1, L::kThreads);
        tc_fence_after();
    }
    const uint32_t tmem = *tmem_slot;   // not of the weight producer's business, which has not met the others

    if (warp == kWarpWProd) {
        // done above
    } else if (L::kInlineX && (warp == kWarpXProd || warp == kWarpX2)) {
        // Codes of a unit in registers while the unit two before is stored: 16
        // codes a piece, two 16-byte chunks of FP16 in the swizzled layout the
        // MMA reads.
        const int xi = warp == kWarpXProd ? 0 : 1;
        grid_dependency_wait();
        Walk cur(p, o, worker, u0);
        if (xi == 1) cur.step(p, o);
        auto fetch = [&](int i, uint4 (&x)[L::kXChunks]) {
#pragma unroll
            for (int j = 0; j < L::kXChunks; ++j) {
                const int m = cur.tm * NA + j * 4 + (lane >> 3);
                const int k = cur.kr * 128 + (lane & 7) * 16;
                x[j] = i < nunits && m < p.M && k < p.K
                           ? *reinterpret_cast<const uint4*>(o.xq + static_cast<int64_t>(m) * o.ldxq + k)
                           : make_uint4(0u, 0u, 0u, 0u);
            }
            cur.step(p, o);
            cur.step(p, o);
        };
        uint4 x[L::kXChunks], ahead[L::kXChunks];
        fetch(xi, x);
        Ring<kSlots> ro(xi);
        for (int i = xi; i < nunits; i += 2, ro.step(2)) {
            fetch(i + 2, ahead);
            if (i >= kSlots && !gemm::warp_wait(ofree(ro.slot), ro.phase ^ 1u, wc)) break;
            uint8_t* box = gbase + L::kXOff + ro.slot * L::kXSlot + ((lane & 7) >> 2) * L::kXBox;
            const int c0 = (lane & 3) * 2;
#pragma unroll
            for (int j = 0; j < L::kXChunks; ++j) {
                const int r = j * 4 + (lane >> 3);
                uint4 a, b;
                s8x4_to_f16(x[j].x, a.x, a.y);
                s8x4_to_f16(x[j].y, a.z, a.w);
                s8x4_to_f16(x[j].z, b.x, b.y);
                s8x4_to_f16(x[j].w, b.z, b.w);
                *reinterpret_cast<uint4*>(box + r * 128 + ((c0 ^ (r & 7)) << 4)) = a;
                *reinterpret_cast<uint4*>(box + r * 128 + (((c0 + 1) ^ (r & 7)) << 4)) = b;
                x[j] = ahead[j];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ofull(ro.slot));
        }
    } else if (warp == kWarpXProd) {
        if (lane == 0) {
            grid_dependency_wait();   // the expansion kernel's output
            const uint64_t pol = policy_evict_last();
            int issued = 0;
            Walk cur(p, o, worker, u0);
            Ring<kSlots> ro(0);
            for (int i = 0; i < nunits; ++i, cur.step(p, o), ro.step(1)) {
                if (i >= kSlots && !wait_bounded(ofree(ro.slot), ro.phase ^ 1u, wc)) break;
                const uint32_t dst = base + L::kXOff + ro.slot * L::kXSlot;
                const int m0 = cur.tm * NA + static_cast<int>(rank) * L::kXRows;
                if (leader) mbar_arrive_expect_tx(ofull(ro.slot), L::kXSlot * L::kCtas);
                if constexpr (kPair) {
                    const uint32_t bar = map_to_cta(ofull(ro.slot), lead);
                    tma_load_2d_pair(dst, &tmX, bar, cur.kr * 128, m0, pol);
                    tma_load_2d_pair(dst + L::kXBox, &tmX, bar, cur.kr * 128 + 64, m0, pol);
                } else {
                    tma_load_2d(dst, &tmX, ofull(ro.slot), cur.kr * 128, m0, pol);
                    tma_load_2d(dst + L::kXBox, &tmX, ofull(ro.slot), cur.kr * 128 + 64, m0, pol);
                }
                issued = i + 1;
            }
            // a unit whose MMAs are complete has its copies, and those before it
            // theirs; after a wait that gave up they never run, and the drain
            // gives up as well
            if (issued > 0)
                gemm::drain_wait(ofree((issued - 1) % kSlots), ((issued - 1) / kSlots) & 1, p.timeout_ns);
        }
    } else if (warp == kWarpMma && leader) {
        const bool elected = elect_one();
        constexpr uint32_t idesc = kPair ? idesc_f16_pair(NA) : idesc_f16(NA, false);
        const uint64_t dx0 = smem_desc_sw128(base + L::kXOff);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if constexpr (kPair) return __all_sync(0xffffffffu, wait_bounded_cluster(bar, parity, wc)) != 0;
            else return gemm::warp_wait(bar, parity, wc);
        };
        auto commit = [&](uint32_t bar) {
            if constexpr (kPair) tc_commit_pair(bar, static_cast<uint16_t>(3u << lead));
            else tc_commit(bar);
        };
        // the K block within a tile: whole tiles, then the tail from its first
        int kb = o.nfull > 0 ? 0 : u0 % p.KB;
        grid_dependency_wait();   // the activations come behind it
        Ring<kSlots> ro(0);
        int piece = 0;
        int last_a = -1;
        uint32_t last_ph = 0;
        bool fresh = true;   // the next MMA starts a piece
        for (int i = 0; i < nunits; ++i, ro.step(1)) {
            const int b = piece % kD;
            if (fresh && piece >= kD && !wait(dempty(b), ((piece / kD) - 1) & 1)) break;
            if (!wait(ofull(ro.slot), ro.phase)) break;
            tc_fence_after();
            const uint32_t dt = tmem + L::kDCol0 + b * NA;
            const uint32_t at = tmem + (i % kABufs) * 64;
            const uint64_t xd = dx0 + static_cast<uint64_t>((ro.slot * L::kXSlot) >> 4);
            const bool closes = i == nunits - 1 || kb == p.KB - 1;
            if (elected) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t bd = xd + (((j >> 2) * L::kXBox + (j & 3) * 32) >> 4);
                    if constexpr (kPair) mma_ts_f16_pair(dt, at + j * 8, bd, idesc, (j > 0 || !fresh) ? 1u : 0u);
                    else mma_ts_f16(dt, at + j * 8, bd, idesc, (j > 0 || !fresh) ? 1u : 0u);
                }
                commit(ofree(ro.slot));
                if (closes) commit(dfull(b));
            }
            __syncwarp();
            last_a = ro.slot;
            last_ph = ro.phase;
            fresh = closes;
            if (closes) ++piece;
            if (++kb == p.KB) kb = i + 1 == o.nfull * p.KB ? u0 % p.KB : 0;
        }
        if (last_a >= 0 && elected) gemm::drain_wait(ofree(last_a), last_ph, p.timeout_ns);
    } else if (warp >= L::kWarpConv0) {
        const int q = warp & 3;
        const int grp = (warp - L::kWarpConv0) >> 2;
        const int row = q * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        Ring<kWStages> rw(grp);
        Ring<kSlots> ro(grp);      // the unit's slot
        Ring<kSlots> done(grp);    // that of the unit kABufs before it, whose A buffer it takes
        if (L::kInlineX && !o.early) grid_dependency_wait();   // so do the weights
        for (int i = grp; i < nunits; i += kGroups, rw.step(kGroups), ro.step(kGroups)) {
            if (!gemm::warp_wait(wfull(rw.slot), rw.phase, wc)) break;
            const uint8_t* src = gbase + rw.slot * L::kWBytes + row * 128;
            uint4 c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = *reinterpret_cast<const uint4*>(src + ((j ^ (row & 7)) << 4));
            if (i >= kABufs) {
                if (i < kABufs + kGroups) grid_dependency_wait();   // MMAs are behind it
                if (!gemm::warp_wait(ofree(done.slot), done.phase, wc)) break;
                done.step(kGroups);
            }
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t f[16];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 w = c[2 * t + e];
                    s8x4_to_f16(w.x, f[8 * e + 0], f[8 * e + 1]);
                    s8x4_to_f16(w.y, f[8 * e + 2], f[8 * e + 3]);
                    s8x4_to_f16(w.z, f[8 * e + 4], f[8 * e + 5]);
                    s8x4_to_f16(w.w, f[8 * e + 6], f[8 * e + 7]);
                }
                tmem_st_x16(tl + (i % kABufs) * 64 + t * 16, f);
            }
            // the loads have returned: the TMEM stores above needed them
            __syncwarp();
            if (lane == 0) mbar_arrive(wempty(rw.slot));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair && !leader) mbar_arrive_cluster(map_to_cta(ofull(ro.slot), lead));
                else mbar_arrive(ofull(ro.slot));
            }
        }
    } else if (kClu && warp >= kWarpEpi0) {
        // One tile piece.  Each worker sums 1/pieces of the tile's columns: a
        // warp's chunks of 16 columns go to the pieces in order, kC to each.
        // First every worker is done with its MMAs, and so with its operand
        // rings, which take the partial sums of the others; then each CTA adds up
        // the chunks it owns, in piece order.  (Partial sums through the workspace
        // cost 9 us of a 256-row tile, this way 4; 64 x 5120 x 5120 15.2 and 13.5 us.
        // At 16 rows, where one CTA would sum all of a tile, 1 x 1024 x 5120 took
        // 7.1 us either way and 8 x 2048 x 8192 8.4 and 9.0: not built.)
        constexpr int kChunks = L::kEpiCols / 16;
        const int ew = warp - kWarpEpi0;
        const int q = warp & 3;
        const int col0 = (ew >> 2) * L::kEpiCols;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + L::kDCol0 + col0;
        float* sxs = reinterpret_cast<float*>(gbase + L::kScaleOff) + ew * L::kScaleCols;
        const int pieces = o.pieces;
        const int piece = static_cast<int>(crank) / L::kCtas;
        const int kC = (kChunks + pieces - 1) / pieces;
        // (pieces - 1) kC <= kChunks + pieces - 2 buffers an epilogue warp
        static_assert((kChunks + kMostPieces - 2) * L::kEpi * 2048 <= L::kBarOff,
                      "the others' partial sums fit the rings");
        const int c_lo = piece * kC < kChunks ? piece * kC : kChunks;
        const int c_hi = c_lo + kC < kChunks ? c_lo + kC : kChunks;
        // the buffer of piece j's chunk (the lc-th of an owner's), this warp's part
        auto buffer = [&](int j, int owner, int lc) {
            return (((j < owner ? j : j - 1) * L::kEpi + ew) * kC + lc) * 2048 + lane * 16;
        };
        grid_dependency_wait();   // the scales and Y may be in use by the preceding grid
        int tn, tm;
        place_of(o, worker / pieces, tn, tm);
        const int n = (tn * L::kCtas + static_cast<int>(rank)) * 128 + q * 32 + lane;
        const int m0 = tm * NA + col0;
        const float sw = n < p.N ? o.sw[n] : 0.0f;
        const float bias = o.bias != nullptr && n < p.N ? o.bias[n] : 0.0f;
        // the scales of the owned columns (at most 64, and at most the warp's)
        for (int c = lane; c < (c_hi - c_lo) * 16; c += 32) {
            const int m = m0 + c_lo * 16 + c;
            sxs[c] = m < p.M ? o.sx[m] : 0.0f;
        }
        const bool ok = gemm::warp_wait(dfull(0), 0, wc);
        tc_fence_after();
        auto load16 = [&](int c, float (&f)[16]) {
            uint32_t v[16];
            tmem_ld_x16(tl + 16 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]);
        };
        __syncwarp();
        cluster_sync_all();   // every ring is idle
        if (ok) {
            // start with the next piece's chunks, so that the CTAs write to
            // different ones at a time
#pragma unroll 1
            for (int e = kC; e < pieces * kC; ++e) {
                int c = c_lo + e;
                if (c >= pieces * kC) c -= pieces * kC;
                if (c >= kChunks) continue;
                const int owner = c / kC;
                if (owner == piece) continue;
                const uint32_t to =
                    map_to_cta(base + buffer(piece, owner, c - owner * kC), static_cast<uint32_t>(owner * L::kCtas) + rank);
                float f[16];
                load16(c, f);
#pragma unroll
                for (int g = 0; g < 4; ++g) st_cluster(to + g * 512, f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]);
            }
        }
        __syncwarp();
        cluster_sync_all();   // every partial sum has arrived
        if (ok) {
#pragma unroll 1
            for (int c = c_lo; c < c_hi; ++c) {
                float own[16], acc[16];
                load16(c, own);
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
                for (int j = 0; j < pieces; ++j) {
                    if (j == piece) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[i] = __fadd_rn(acc[i], own[i]);
                    } else {
                        const uint8_t* from = gbase + buffer(j, piece, c - c_lo);
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float4 x = *reinterpret_cast<const float4*>(from + g * 512);
                            acc[4 * g + 0] = __fadd_rn(acc[4 * g + 0], x.x);
                            acc[4 * g + 1] = __fadd_rn(acc[4 * g + 1], x.y);
                            acc[4 * g + 2] = __fadd_rn(acc[4 * g + 2], x.z);
                            acc[4 * g + 3] = __fadd_rn(acc[4 * g + 3], x.w);
                        }
                    }
                }
                store16(p, o, n, m0 + 16 * c, sxs + 16 * (c - c_lo), sw, bias, acc);
            }
        }
    } else if (!kClu && warp >= kWarpEpi0) {
        const int ew = warp - kWarpEpi0;
        const int q = warp & 3;
        const int col0 = (ew >> 2) * L::kEpiCols;
        const int row = q * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + L::kDCol0 + col0;
        const int tail_tile = o.nfull * o.workers + u0 / p.KB;
        const int split_info = u1 > u0 ? gemm::split_info_lane(p, u0, u1, lane) : 0;
        float* sxs = reinterpret_cast<float*>(gbase + L::kScaleOff) + ew * L::kScaleCols;
        // the scales, Y and the workspace may be in use by the preceding grid
        grid_dependency_wait();
        int ps = 0;
        for (int pc = 0; ps < nunits; ++pc) {
            const bool full = pc < o.nfull;
            const int kb0 = pc == o.nfull ? u0 % p.KB : 0;
            const int tile = full ? worker + pc * o.workers : tail_tile + pc - o.nfull;
            const int b = pc % kD;
            int pe = ps + (p.KB - kb0) - 1;
            if (pe > nunits - 1) pe = nunits - 1;
            const bool whole = kb0 == 0 && pe - ps == p.KB - 1;
            int tn, tm;
            place_of(o, tile, tn, tm);
            const int n = (tn * L::kCtas + static_cast<int>(rank)) * 128 + row;
            const int m0 = tm * NA + col0;
            const float sw = n < p.N ? o.sw[n] : 0.0f;
            const float bias = o.bias != nullptr && n < p.N ? o.bias[n] : 0.0f;
            // the tile's activation scales, fetched while its MMAs run: lane l
            // holds columns l, l + 32, ...; they reach the other lanes through
            // the warp's own shared memory, kScaleCols at a time
            constexpr int kHeld = (L::kEpiCols + 31) / 32;
            float held[kHeld];
#pragma unroll
            for (int h = 0; h < kHeld; ++h) {
                const int c = 32 * h + lane;
                held[h] = c < L::kEpiCols && m0 + c < p.M ? o.sx[m0 + c] : 0.0f;
            }
            int window = -1;   // the columns whose scales are in shared memory
            auto scales_from = [&](int c) {   // of the 16 columns from 16 c
                const int at0 = (16 * c) / L::kScaleCols * L::kScaleCols;
                if (at0 != window) {
                    window = at0;
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < kHeld; ++h) {
                        const int at = 32 * h + lane - at0;
                        if (at >= 0 && at < L::kScaleCols) sxs[at] = held[h];
                    }
                    __syncwarp();
                }
                return sxs + 16 * c - at0;
            };
            if (!gemm::warp_wait(dfull(b), (pc / kD) & 1, wc)) break;
            tc_fence_after();
            const int which = pc == o.nfull ? 0 : 1;   // of the tail's first and last tile
            auto release = [&]() {   // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair && !leader) mbar_arrive_cluster(map_to_cta(dempty(b), lead));
                    else mbar_arrive(dempty(b));
                }
            };
            auto load16 = [&](int c, float (&f)[16]) {
                uint32_t v[16];
                tmem_ld_x16(tl + b * NA + 16 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]);
            };
            if (whole && o.y_type != QG_FP32) {
                // all columns into registers, packed, so that the next tile's
                // MMAs run under the stores (with one accumulator per pair the
                // stores held them for 5 us of each tile's 38)
                uint32_t w[L::kEpiCols / 2];
#pragma unroll
                for (int c = 0; c < L::kEpiCols / 16; ++c) {
                    float f[16];
                    load16(c, f);
                    pack16(f, scales_from(c), sw, bias, o.y_type, w + 8 * c);
                }
                release();
                store_packed<L::kEpiCols>(p, o.y_pairs, n, m0, w);
            } else if (whole) {
                // 32-bit outputs.  With one accumulator, as many columns as
                // registers take (64) are read before the release and stored after
                // it, the others go out first (1901 x 18854 x 2048: 108 -> 100 us;
                // with two, the stores hold nothing up).
                constexpr int kHold = kD == 1 ? 64 : 16;
                constexpr int kFirst = (L::kEpiCols - kHold) / 16;
#pragma unroll 1
                for (int c = 0; c < kFirst; ++c) {
                    float f[16], y[16];
                    load16(c, f);
                    scale16(f, scales_from(c), sw, bias, y);
                    store_f32<16>(p, n, m0 + 16 * c, y);
                }
                float y[kHold];
#pragma unroll
                for (int c = 0; c < kHold / 16; ++c) {
                    float f[16];
                    load16(kFirst + c, f);
                    scale16(f, scales_from(kFirst + c), sw, bias, y + 16 * c);
                }
                release();
                store_f32<kHold>(p, n, m0 + 16 * kFirst, y);
            } else {
                // A piece of a split tile: partial sums to the workspace, a slice
                // of the warp's columns at a time, each with an arrival counter of
                // its own; the last of a tile's CTAs to arrive at a slice sums it.
                // The CTAs start at different slices, so that, ending together,
                // they are each last at some: one CTA summing all of a tile was
                // bound by its own reads of L2 (8 to 10 us of a wide tile).
                //
                // A counter is indexed by the CTA that holds the tile's first
                // unit: that CTA's last tile, so no other tile shares it (a pair's
                // CTAs keep partial sums and counters of their own).
                const int cf = __shfl_sync(0xffffffffu, split_info, 3 * which);
                const int cl = __shfl_sync(0xffffffffu, split_info, 3 * which + 1);
                const int w_first = __shfl_sync(0xffffffffu, split_info, 3 * which + 2);
                uint32_t* cnt = p.cnt + ((cf * L::kCtas + static_cast<int>(rank)) * 8 + ew) * kInt8Slices;
                float4* mine = part_slot<NA>(p, cta, which) + (col0 / 4) * 128 + row;
                const int s0 = (worker - cf) * L::kSlices / (cl - cf + 1);
                uint32_t last_at = 0;   // slices this CTA is the last to arrive at
#pragma unroll 1
                for (int e = 0; e < L::kSlices; ++e) {
                    const int sl = (s0 + e) % L::kSlices;
#pragma unroll 1
                    for (int c = sl * L::kSliceCols / 16; c < (sl + 1) * L::kSliceCols / 16; ++c) {
                        float f[16];
                        load16(c, f);
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            __stcg(mine + (4 * c + g) * 128,
                                   make_float4(f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]));
                    }
                    if (e == L::kSlices - 1) release();
                    // every lane's partial visible GPU-wide before lane 0's arrival
                    __threadfence();
                    __syncwarp();
                    uint32_t prev = 0;
                    if (lane == 0) prev = atomicAdd(cnt + sl, 1u);
                    prev = __shfl_sync(0xffffffffu, prev, 0);
                    if (static_cast<int>(prev) == cl - cf) last_at |= 1u << sl;
                }
                if (last_at) __threadfence();
#pragma unroll 1
                for (int c = 0; c < L::kEpiCols / 16; ++c) {
                    const int sl = 16 * c / L::kSliceCols;
                    if (!(last_at >> sl & 1u)) continue;
                    float acc[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
                    // four pieces' loads in flight at a time
#pragma unroll 1
                    for (int c4 = cf; c4 <= cl; c4 += 4) {
                        float4 x[4][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c2 = c4 + e;
                            const float4* src =
                                part_slot<NA>(p, c2 * L::kCtas + static_cast<int>(rank), c2 == cf ? w_first : 0) +
                                (col0 / 4 + 4 * c) * 128 + row;
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                x[e][g] = c2 <= cl ? __ldcg(src + g * 128) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                acc[4 * g + 0] = __fadd_rn(acc[4 * g + 0], x[e][g].x);
                                acc[4 * g + 1] = __fadd_rn(acc[4 * g + 1], x[e][g].y);
                                acc[4 * g + 2] = __fadd_rn(acc[4 * g + 2], x[e][g].z);
                                acc[4 * g + 3] = __fadd_rn(acc[4 * g + 3], x[e][g].w);
                            }
                    }
                    store16(p, o, n, m0 + 16 * c, scales_from(c), sw, bias, acc);
                    // its last columns: the slice is ready for the next call
                    if (lane == 0 && (16 * c + 16) % L::kSliceCols == 0) cnt[sl] = 0u;
                }
            }
            ps = pe + 1;
        }
    }

    tc_fence_before();
    if (kClu && (warp < kWarpEpi0 || warp >= L::kWarpConv0)) {   // the two meetings of the epilogue
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }
    // a pair leaves together: the leader's MMAs read both CTAs' operands, and
    // either's threads arrive on the other's barriers
    __syncwarp();
    if constexpr (kPair || kClu) cluster_sync_all();
    else __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// The activations as FP16 [M, K]: 16 codes (K % 16 == 0) a thread.  The GEMM
// behind it may start, and stream weights, at once: the grid before this one is
// done by then, unless the caller allows the overlap.
__global__ void __launch_bounds__(256) expand_kernel(const int8_t* __restrict__ Xq, int64_t ldxq,
                                                     uint4* __restrict__ out, int M, int K16) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t total = static_cast<int64_t>(M) * K16;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = t / K16;
        const uint4 c = *reinterpret_cast<const uint4*>(Xq + m * ldxq + (t - m * K16) * 16);
        uint4 a, b;
        s8x4_to_f16(c.x, a.x, a.y);
        s8x4_to_f16(c.y, a.z, a.w);
        s8x4_to_f16(c.z, b.x, b.y);
        s8x4_to_f16(c.w, b.z, b.w);
        out[2 * t] = a;
        out[2 * t + 1] = b;
    }
}

// ----------------------------------------------------------------- quantiser
// Row maximum below this: the row counts as zero (codes 0, scale 1), so that
// 1 / max stays finite.
constexpr float kTinyMax = 7.888609052210118e-31f;   // 2^-100

template <bool kBf16>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    if (kBf16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    }
}

// Codes of two values as the low bytes of two words.  The product is rounded
// to FP32; adding 1.5 * 2^23 then rounds it half to even at the unit, and the
// sum's low byte is the code (an FP32 to integer conversion gives the same at a
// quarter of the rate).  Scalar intrinsics: as packed operations the product
// and the sum came out fused, without the rounding in between.
template <bool kBf16>
__device__ __forceinline__ void codes2(uint32_t w, float inv, uint32_t& a, uint32_t& b) {
    float x, y;
    unpack2<kBf16>(w, x, y);
    a = __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
    b = __float_as_uint(__fadd_rn(__fmul_rn(y, inv), 12582912.0f));
}

template <bool kBf16>
__device__ __forceinline__ uint2 codes8(const uint4& w, float inv) {
    uint32_t c[8];
    codes2<kBf16>(w.x, inv, c[0], c[1]);
    codes2<kBf16>(w.y, inv, c[2], c[3]);
    codes2<kBf16>(w.z, inv, c[4], c[5]);
    codes2<kBf16>(w.w, inv, c[6], c[7]);
    const uint32_t l = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
    const uint32_t h = prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u);
    return make_uint2(l, h);
}

// The largest |x| of 8 values so far, as bit patterns (which order like the
// magnitudes), two to a word.
__device__ __forceinline__ uint32_t max8(const uint4& w, uint32_t m) {
    m = max_u16x2(m, max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu));
    return max_u16x2(m, max_u16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
}

// One CTA per row.  A thread keeps its kVec vectors of the row (rows up to
// 2048 kVec elements) in registers between the maximum and the codes, so that
// the row is read once; kVec = 0 reads it twice, the second time from L2.  Bound
// by memory: 2 bytes in and 1 out per element (4096 x 17408: 32 us at the
// measured copy rate).
template <bool kBf16, int kVec>
__global__ void __launch_bounds__(256) quantize_int8_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                            int8_t* __restrict__ Xq, int64_t ldxq,
                                                            float* __restrict__ Sx, int K) {
    __shared__ uint32_t warp_max[8];
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t m = blockIdx.x;
    const uint4* x = reinterpret_cast<const uint4*>(X + m * ldx);
    uint2* q = reinterpret_cast<uint2*>(Xq + m * ldxq);
    const int nv = K / 8;
    uint4 held[kVec > 0 ? kVec : 1];
    uint32_t mx = 0u;
    if constexpr (kVec > 0) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int v = j * 256 + threadIdx.x;
            held[j] = v < nv ? x[v] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) mx = max8(held[j], mx);
    } else {
        for (int v = threadIdx.x; v < nv; v += 256) mx = max8(x[v], mx);
    }
    mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max(mx, warp_max[j]);
    float amax, unused;
    unpack2<kBf16>(mx, amax, unused);
    // A row with a NaN or an infinity (whose bit patterns order above every
    // finite magnitude) has scale NaN, which the GEMM carries to its whole output.
    const bool finite = amax < INFINITY;
    const bool live = finite && amax >= kTinyMax;
    const float inv = live ? __fmul_rn(127.0f, __frcp_rn(amax)) : 0.0f;
    if (threadIdx.x == 0)
        Sx[m] = live ? __fdiv_rn(amax, 127.0f) : finite ? 1.0f : __uint_as_float(0x7FC00000u);
    if constexpr (kVec > 0) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int v = j * 256 + threadIdx.x;
            if (v < nv) q[v] = codes8<kBf16>(held[j], inv);
        }
    } else {
        for (int v = threadIdx.x; v < nv; v += 256) q[v] = codes8<kBf16>(x[v], inv);
    }
}

template <bool kBf16>
cudaError_t launch_quantize(const cudaLaunchConfig_t& cfg, const uint16_t* X, int64_t ldx, int8_t* Xq, int64_t ldxq,
                            float* Sx, int K) {
    if (K <= 2048 * 4) return cudaLaunchKernelEx(&cfg, quantize_int8_kernel<kBf16, 4>, X, ldx, Xq, ldxq, Sx, K);
    if (K <= 2048 * 10) return cudaLaunchKernelEx(&cfg, quantize_int8_kernel<kBf16, 10>, X, ldx, Xq, ldxq, Sx, K);
    return cudaLaunchKernelEx(&cfg, quantize_int8_kernel<kBf16, 0>, X, ldx, Xq, ldxq, Sx, K);
}

__global__ void bias_rows_kernel(const float* bias, void* Y, int64_t ldy, int y_type, int M, int N) {
    const int64_t total = static_cast<int64_t>(M) * N;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = t / N;
        const int64_t n = t - m * N;
        const float b = bias ? bias[n] : 0.0f;
        if (y_type == QG_FP32) static_cast<float*>(Y)[m * ldy + n] = b;
        else if (y_type == QG_BF16) static_cast<__nv_bfloat16*>(Y)[m * ldy + n] = __float2bfloat16_rn(b);
        else static_cast<__half*>(Y)[m * ldy + n] = __float2half_rn(b);
    }
}

template <int NA, bool kPair, bool kClu>
cudaError_t launch_int8_na(const Int8Args& a, const Int8Schedule& s, const CUtensorMap& tmW, const CUtensorMap& tmX,
                           const LaunchCtl& c, cudaStream_t st) {
    using L = I8Layout<NA, kPair>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(configured, int8_kernel<NA, kPair, kClu>, L::kSmemBytes);
    static std::atomic<uint64_t> wide{0};
    if (e == cudaSuccess && kClu && s.pieces * L::kCtas > 8)
        e = set_once(wide, int8_kernel<NA, kPair, kClu>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    Params p = gemm::base_params(s, a.Y, a.ldy, a.M, a.N, a.K, nullptr, c);
    p.U = static_cast<long long>(s.T - s.nfull * s.G) * s.KU;   // the tail
    p.G = s.tail_g;
    uint8_t* w = static_cast<uint8_t*>(a.ws);
    p.cnt = reinterpret_cast<uint32_t*>(w);
    p.part = w ? reinterpret_cast<float*>(w + kInt8CounterBytes + int8_expanded_bytes(s, a.M, a.K)) : nullptr;
    const int y_pairs = a.y_type != QG_FP32 && a.N % 2 == 0 && a.ldy % 2 == 0 &&
                        (reinterpret_cast<uintptr_t>(a.Y) & 3u) == 0;
    const Out o{a.Xq, a.ldxq, a.Sx, a.Sw, a.bias, a.y_type, y_pairs, (a.N + 128 * L::kCtas - 1) / (128 * L::kCtas),
                (a.M + NA - 1) / NA, s.G, s.nfull, s.pieces, c.overlap ? 1 : 0,
                p.G > 0 ? static_cast<int>(p.U / p.G) : 0, p.G > 0 ? static_cast<int>(p.U % p.G) : 0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.G * L::kCtas));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = st;
    // Always launched ahead.  Behind the expansion kernel, which is part of this
    // call, the weight stream starts at once; without one the kernel sets itself
    // up under the end of the preceding grid, but touches no memory before that
    // is done (unless the caller allows it for the weights).
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (kPair || kClu) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(L::kCtas * (kClu ? s.pieces : 1));
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, int8_kernel<NA, kPair, kClu>, tmW, tmX, p, o);
}

template <int NA, bool kPair>
cudaError_t launch_int8_rows(const Int8Args& a, const Int8Schedule& s, const CUtensorMap& tmW, const CUtensorMap& tmX,
                             const LaunchCtl& c, cudaStream_t st) {
    if constexpr (NA > 16)
        if (s.pieces > 1) return launch_int8_na<NA, kPair, true>(a, s, tmW, tmX, c, st);
    return launch_int8_na<NA, kPair, false>(a, s, tmW, tmX, c, st);
}

}  // namespace

// The cost of a schedule is the time of its busiest worker, in nanoseconds:
// what every call takes, units (a tile x 128 of K), and what a split adds.  The
// whole tiles cost floor(T / workers) tiles; for the tail of r tiles the rule
// takes the cheapest of
//   - one worker a tile: KU units
//   - k <= floor(workers / r) equal pieces of every tile: ceil(KU / k) units and
//     a split (storing, counting and summing partial results)
//   - k equal pieces of every tile in a cluster, where all clusters run at once:
//     ceil(KU / k) units and the exchange
//   - all workers, pieces that straddle tiles: ceil(r KU / workers) units and
//     two splits a worker
// and over the tile widths the one that costs least: wide tiles read fewer
// weights and activations per product, narrow ones spread a small product over
// more SMs, split at a lower price, and the narrowest saves a launch (2 us of
// the constant: the host's time, which bounds small calls).  Measured, whole
// tiles / equal pieces / straddling / clusters: 256 x 5120 x 17408 at 256 rows
// 81.0 / 42.4 / 49.8 / 38.6 us; 128 x 6144 x 5120 at 128 rows 19.0 / 17.5 / 22.4 /
// 15.7; 64 x 5120 x 5120 at 64 rows 19.2 / 14.9 / 17.7 / 13.2; 1 x 1024 x 5120 at
// 16 rows 14.8 / 7.0 / 8.8.  And the best of them by width (16, 32, 64, 128 rows):
// 100 x 1000 x 1008 5.5 / 7.2 / 7.6 / 8.6 us, 172 x 4218 x 1456 14.5 / 12.0 / 9.2 /
// 10.1, 64 x 5120 x 5120 20.0 / 16.8 / 13.2 / 14.4, 64 x 1024 x 8192 10.5 / 11.3 /
// 11.2 / 12.5.  On 17 shapes of 1 to 172 rows the rule's choice took at most 2%
// more than the best of all widths and forms.
struct TileCost {
    int rows;
    long long call_ns, unit_ns, split_ns, straddle_ns;
    long long cluster_ns;   // of equal pieces in a cluster; 0: not offered
};
constexpr TileCost kTiles[] = {{16, 4000, 305, 3000, 7500, 0},
                               {32, 6300, 310, 4000, 7500, 2800},
                               {64, 6500, 340, 6500, 10500, 3000},
                               {128, 7700, 350, 7500, 14500, 3500},
                               {256, 8500, 560, 9500, 24000, 4500}};

Int8Schedule schedule_with(const TileCost& tc, int M, int N, int K, int sms, int forced, const int* clusters,
                           long long* cost) {
    Int8Schedule s;
    s.nmma = tc.rows;
    const int ctas = int8_ctas(s.nmma);
    const long long tn = (N + 128ll * ctas - 1) / (128 * ctas);
    s.T = static_cast<int>(tn * ((M + s.nmma - 1) / s.nmma));
    s.KU = static_cast<int>((static_cast<int64_t>(K) + 127) / 128);
    s.U = static_cast<long long>(s.T) * s.KU;
    long long w = forced > 0 ? (forced + ctas - 1) / ctas : sms / ctas;
    if (w < 1) w = 1;
    s.max_ctas = static_cast<int>(w * ctas);
    if (w > s.U) w = s.U;
    s.nfull = static_cast<int>(s.T / w);
    long long r = s.T - s.nfull * w;
    long long g = 0;
    *cost = tc.call_ns + static_cast<long long>(s.nfull) * s.KU * tc.unit_ns;
    if (r > 0) {
        // no tile in more than kMostSplit pieces, which one CTA sums in turn, and
        // 0.2 us for each beyond 8 (1 x 128 x 17408 in 8 pieces 10.1 us, in 12 9.2, in
        // 16 8.7, in 136 21.3; 1 x 1024 x 5120 7.0, 7.6, 8.0)
        auto up = [](long long a, long long b) { return (a + b - 1) / b; };
        long long all = w < r * s.KU ? w : r * s.KU;
        if (all > r * kMostSplit && forced == 0) all = r * kMostSplit;
        const long long straddle = up(r * s.KU, all) * tc.unit_ns + tc.straddle_ns;
        long long best = s.KU * tc.unit_ns;
        g = r;
        for (long long k = 2; k <= w / r && k <= kMostSplit && k <= s.KU; ++k) {
            const long long cost_k = up(s.KU, k) * tc.unit_ns + tc.split_ns + (k > 8 ? (k - 8) * 200 : 0);
            if (cost_k >= best) continue;
            best = cost_k;
            g = k * r;
        }
        if (straddle < best || forced > 0) {
            best = straddle;
            g = all;
        }
        // equal pieces in clusters, as many as run at once; of odd sizes, which share
        // SM pairs with their neighbours, nine tenths of what the device states (64 x
        // 8192 with 42 tiles in clusters of 3, of 46: 16.5 us, 45 tiles 19.6, 46 22.0;
        // even sizes run to the last)
        if (tc.cluster_ns > 0 && s.nfull == 0 && forced == 0) {
            for (int c = 2; c * ctas <= kMostClusterCtas && c <= kMostPieces && c <= s.KU; ++c) {
                const int fit = c * ctas % 2 != 0 ? clusters[c * ctas] * 9 / 10 : clusters[c * ctas];
                if (s.T > fit || up(s.KU, c) * tc.unit_ns + tc.cluster_ns >= best) continue;
                best = up(s.KU, c) * tc.unit_ns + tc.cluster_ns;
                g = static_cast<long long>(c) * r;
                s.pieces = c;
            }
        }
        *cost += best;
        // A few rounds of whole tiles on single CTAs: as many workers as keep
        // all of them busy in every round.  These shapes are bound by memory,
        // and a last round on part of the SMs does not fill it (32 x 32768 x
        // 5120: 34.8 us on 152 CTAs, 32.9 on 128; from five rounds on, and on
        // pairs, which are bound by the tensor cores, it costs up to 1%).
        if (g == r && ctas == 1 && s.nfull >= 1 && s.nfull <= 3 && forced == 0) {
            w = up(s.T, s.nfull + 1);
            s.nfull = static_cast<int>(s.T / w);
            g = r = s.T - s.nfull * w;
        }
    }
    s.tail_g = static_cast<int>(g);
    s.G = static_cast<int>(s.nfull > 0 ? w : g);
    return s;
}

Int8Schedule int8_schedule(int M, int N, int K, int sms, int forced, const int* clusters) {
    Int8Schedule best;
    long long least = 0;
    int narrower = 0;   // rows of the next narrower tile
    for (const TileCost& tc : kTiles) {
        if (narrower >= M) break;   // the narrower one takes the batch as it is
        narrower = tc.rows;
        long long cost = 0;
        const Int8Schedule s = schedule_with(tc, M, N, K, sms, forced, clusters, &cost);
        if (best.T == 0 || cost < least) {
            best = s;
            least = cost;
        }
    }
    // splits: some worker's part of the tail begins inside a tile
    const long long units = (best.T - static_cast<long long>(best.nfull) * best.G) * best.KU;
    for (long long c = 1; c < best.tail_g && !best.split && best.pieces == 0; ++c)
        best.split = c * units / best.tail_g % best.KU != 0;
    return best;
}

// The clusters of c CTAs that a device runs at once (a cluster lies within one
// of the device's groups of SMs, so that they are fewer than the SMs would
// hold).  Every kernel here takes an SM to itself; one is asked for all.
void int8_cluster_capacity(int (&clusters)[kMostClusterCtas + 1]) {
    for (int c = 0; c <= kMostClusterCtas; ++c) {
        clusters[c] = 0;
        if (c < 2 || (c > 8 && c % 2 != 0)) continue;   // pairs only beyond 8
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(c * 64);
        cfg.blockDim = dim3(I8Layout<256, true>::kThreads);
        cfg.dynamicSmemBytes = I8Layout<256, true>::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = c;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const auto kernel = int8_kernel<256, true, true>;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, I8Layout<256, true>::kSmemBytes) ==
                cudaSuccess &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess)
            clusters[c] = n;
        else
            cudaGetLastError();   // not offered; no later call shall find the error
    }
}

size_t int8_expanded_bytes(const Schedule& s, int M, int K) {
    if (int8_inline_x(s)) return 0;
    return (static_cast<size_t>(M) * K * 2 + 255) & ~static_cast<size_t>(255);
}

size_t int8_workspace_bytes(const Int8Schedule& s, int M, int K) {
    const size_t part = s.split ? static_cast<size_t>(s.G) * int8_ctas(s.nmma) * 2 * 128 * s.nmma * sizeof(float) : 0;
    const size_t x = int8_expanded_bytes(s, M, K);
    return part + x > 0 ? kInt8CounterBytes + x + part : 0;
}

cudaError_t launch_int8(const Int8Args& a, const Int8Schedule& s, const CUtensorMap& tmW, const CUtensorMap& tmX,
                        const LaunchCtl& c, cudaStream_t st) {
    if (static_cast<size_t>(s.G) * int8_ctas(s.nmma) * 8 * kInt8Slices * sizeof(uint32_t) > kInt8CounterBytes)
        return cudaErrorInvalidValue;
    if (!int8_inline_x(s)) {
        const int K16 = a.K / 16;
        int64_t blocks = (static_cast<int64_t>(a.M) * K16 + 255) / 256;
        if (blocks > 4 * c.num_sms) blocks = 4 * c.num_sms;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(blocks));
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        // waiting resident for the preceding grid even where the caller did not
        // ask for overlap took 0.3 us off small calls, but slowed large ones by 3%
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = c.overlap ? 1 : 0;
        uint4* xf = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.ws) + kInt8CounterBytes);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, expand_kernel, a.Xq, a.ldxq, xf, a.M, K16);
        if (e != cudaSuccess) return e;
    }
    switch (s.nmma) {
        case 16: return launch_int8_rows<16, false>(a, s, tmW, tmX, c, st);
        case 32: return launch_int8_rows<32, false>(a, s, tmW, tmX, c, st);
        case 64: return launch_int8_rows<64, false>(a, s, tmW, tmX, c, st);
        case 128: return launch_int8_rows<128, true>(a, s, tmW, tmX, c, st);
        case 256: return launch_int8_rows<256, true>(a, s, tmW, tmX, c, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_quantize_int8(const void* X, int x_type, int64_t ldx, int8_t* Xq, int64_t ldxq, float* Sx, int M,
                                 int K, const LaunchCtl& c, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    if (c.overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const uint16_t* x = static_cast<const uint16_t*>(X);
    if (x_type == QG_BF16) return launch_quantize<true>(cfg, x, ldx, Xq, ldxq, Sx, K);
    return launch_quantize<false>(cfg, x, ldx, Xq, ldxq, Sx, K);
}

cudaError_t launch_int8_bias_rows(const Int8Args& a, cudaStream_t st) {
    const int64_t total = static_cast<int64_t>(a.M) * a.N;
    const int64_t blocks = total / 256 + 1 < 4096 ? total / 256 + 1 : 4096;
    bias_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(a.bias, a.Y, a.ldy, a.y_type, a.M, a.N);
    return cudaGetLastError();
}

}  // namespace qg
