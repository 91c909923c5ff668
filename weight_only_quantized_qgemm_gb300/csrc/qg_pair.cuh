// Device building blocks of the kernels that work in clusters (the 8-bit
// integer GEMM's CTA pairs, the log probabilities' split rows): cluster
// barriers and remote arrivals, the cta_group::2 forms of TMEM allocation, MMA
// and commit, and two small pieces beside those of qg_device.cuh.
#pragma once

#include "qg_device.cuh"

namespace qg {

// Arrives at a named barrier without waiting (others named_bar_sync on it).
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Instruction descriptor of kind::f16 for a pair: idesc_f16 (FP16 operands)
// with M = 256.
__host__ __device__ constexpr uint32_t idesc_f16_pair(int n) {
    return (idesc_f16(n, false) & ~(31u << 24)) | (static_cast<uint32_t>(256 >> 4) << 24);
}

// ----------------------------------------------------------------- CTA pairs (cta_group::2)
// Two CTAs of a cluster run one MMA of twice the rows: each holds its 128 rows
// of A and D in its own TMEM and half of B's rows in its own shared memory;
// the even one (the leader) issues.
__device__ __forceinline__ uint32_t cluster_cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_all() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    cluster_arrive_all();
    cluster_wait_all();
}
// The shared::cluster address of `addr` (a shared::cta address) in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive on a barrier of another CTA of the cluster (a mapped address).  It
// carries no memory of this thread's: what it announces are TMEM accesses, which
// tcgen05.wait and tcgen05.fence::before_thread_sync in front of it order (a
// release at cluster scope here cost the 8-bit integer GEMM 0.4 us a unit: 37
// against 22 us on 128 x 17408 x 5120).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t mapped) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapped) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// wait_bounded for a barrier that threads of other CTAs arrive on.
static __device__ __noinline__ bool wait_bounded_cluster_slow(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 0; it < (1u << 26); ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if (*c.abort) return false;
        if (globaltimer() - t0 > c.timeout_ns) break;
    }
    raise_abort(c, kDevTimeout);
    return false;
}
__device__ __forceinline__ bool wait_bounded_cluster(uint32_t bar, uint32_t parity, const WaitCtl& c) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    return wait_bounded_cluster_slow(bar, parity, c);
}
// tma_load_2d whose completion is counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t mapped_bar, int c0,
                                                 int c1, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::"
        "cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(m), "r"(mapped_bar), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// mma_ts_f16 over the pair (M = 256).
__device__ __forceinline__ void mma_ts_f16_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// tc_commit of the pair's operations: arrives once on `bar` in both CTAs (mask:
// their places in the cluster).
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(mask)
        : "memory");
}

}  // namespace qg
