// rgg_warp_issue.cuh -- waits and asynchronous instructions for roles that a
// whole warp runs in step, one lane of it issuing.
//
// A role run by one lane inside a divergent branch computes every address and
// descriptor in vector registers and moves each into the uniform registers
// that TMA and tcgen05 instructions take, one by one; on a GB300 a 64 x (256 x
// 256) stage of bf16 MMAs then took about 800 cycles to issue, where the MMAs
// take 512.  Here all lanes run the role's loop, so its addresses stay in
// uniform registers, and each instruction is predicated on the elected lane.
#pragma once

#include "rgg_ptx.cuh"

namespace rgg {

constexpr int kStatusTimeout = 5;

// 1 in one lane of the warp (all lanes present), 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// The calling thread's warp in its block, as a warp-uniform value.
__device__ __forceinline__ int uniform_warp() {
    return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// Bounded wait of a whole warp, the same answer in every lane.  kPair: on a
// cluster of two CTAs, where a timeout also raises the other CTA's abort flag
// (its shared::cluster address), so that both leave their loops instead of
// waiting on arrivals that will not come.  kAcquire: the barrier is arrived on
// by the other CTA after it wrote (or read) this CTA's shared memory, so the
// wait acquires at cluster scope.
template <bool kPair, bool kAcquire>
__device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                            uint32_t peer_flag, int32_t* status, uint64_t timeout_ns) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        const bool done = kAcquire ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, done)) return true;
        if (__any_sync(0xffffffffu, *abort_flag != 0u)) return false;
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > timeout_ns)) {
            *abort_flag = 1u;
            if constexpr (kPair) st_shared_cluster_u32(peer_flag, 1u);
            atomicCAS(status, 0, kStatusTimeout);
            return false;
        }
    }
}

template <bool kPair, bool kAcquire = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t peer_flag, int32_t* status, uint64_t timeout_ns) {
    const bool done = kAcquire ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    return warp_wait_slow<kPair, kAcquire>(bar, parity, abort_flag, peer_flag, status, timeout_ns);
}

// In each of the following `lead` is elect_one()'s value: the lane with 1 issues.

__device__ __forceinline__ void expect_tx_if(uint32_t lead, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(lead)
        : "memory");
}

// 2-D and 3-D box loads; kPair: counted on an mbarrier of either CTA of the pair (its cluster address).
template <bool kPair>
__device__ __forceinline__ void load_2d_if(uint32_t lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                           int32_t y) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(lead)
            : "memory");
}

template <bool kPair>
__device__ __forceinline__ void load_3d_if(uint32_t lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                           int32_t y, int32_t z) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
            "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(lead)
            : "memory");
}

// Arrive once on `bar` (kPair: at that offset in both CTAs) when the lane's earlier tcgen05 operations are done.
template <bool kPair>
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
            "%1;\n\t}" ::"r"(bar),
            "h"(static_cast<uint16_t>(0x3)), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(lead)
            : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], both operands bf16 (K = 16 an instruction) or,
// kFp8, E4M3 (kind::f8f6f4, K = 32), fp32 accumulator.
template <bool kFp8>
__device__ __forceinline__ void mma_single_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    if constexpr (kFp8)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
            : "memory");
}

// D[tmem of both CTAs] (+)= A[smem of both CTAs] * B[smem of both CTAs], bf16:
// M = 256 rows split 128/128 over the pair, B's N columns split in halves.
__device__ __forceinline__ void mma_bf16_pair_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

}  // namespace rgg
