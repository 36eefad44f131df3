// experts_ptx.cuh -- PTX wrappers the expert products need beside ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace dg {

// mbar_wait with acquire semantics over the cluster: for barriers that the peer
// CTA of a pair arrives on after writing memory this thread's MMAs will read.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                  uint64_t limit_ns) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait_cluster(a, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (true) {
        if (mbar_try_wait_cluster(a, parity)) return true;
        if (abort != nullptr && *abort) return false;
        if (globaltimer() - t0 > limit_ns) return false;
    }
}

// One lane of a converged warp. The MMA issuers run their loops as whole warps and let
// this lane issue: in a branch of one lane the operand addresses cannot stay in uniform
// registers, and an MMA took ~110 clocks to issue whatever its size.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Arrive on a barrier of the pair's other CTA, releasing at CTA scope. What is
// handed over lies in this CTA's own shared memory and is read by its own SM's
// tensor core, so CTA scope orders it; a release at cluster scope waits for every
// memory operation that the thread has outstanding (~0.9 us a stage, measured).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A bounded wait that polls with test_wait. (try_wait, which may suspend the thread,
// costs more where many warps of a CTA wait: with eight converter warps polling, the
// MMA issuer took 1300 clocks a stage instead of 1060.)
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_test(bar, parity)) return true;
        if (abort != nullptr && *abort) return false;
        if (globaltimer() - t0 > limit_ns) return false;
    }
}

// A wait by a whole warp, polled by one lane (32 polling lanes take 32 turns in the
// shared-memory unit). The outcome is the same in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    unsigned ok = 1;
    if ((threadIdx.x & 31) == 0) ok = mbar_poll(bar, parity, abort, limit_ns);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// 4-D and 5-D tiled loads global -> shared (coordinates innermost first), counted
// in bytes on an mbarrier given by its shared::cluster address; PAIR: the barrier
// may be in the peer CTA.
template <bool PAIR>
__device__ __forceinline__ void tma_load_nd(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            uint64_t pol) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(pol)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_load_nd(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, uint64_t pol) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_load_nd(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w, uint64_t pol) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(pol)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_load_nd(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w, int32_t v, uint64_t pol) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "l"(pol)
            : "memory");
}

}  // namespace dg
