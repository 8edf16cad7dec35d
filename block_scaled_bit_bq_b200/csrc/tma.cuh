// tma.cuh -- tensor-map bulk copies (TMA) from global into shared memory, completed on
// an mbarrier, and waits on them that give up after about a second instead of hanging.
#pragma once

#include <cuda.h>   // CUtensorMap (the type only; the map is encoded on the host)

#include "common.cuh"

namespace bq {

// cuTensorMapEncodeTiled, reached through the runtime's driver entry point (no link to
// libcuda); null if the driver does not offer it.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}

// Makes mbarrier initialisation visible to the async proxy (the TMA unit).
__device__ __forceinline__ void fence_mbar_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Orders this thread's generic-proxy shared-memory accesses before later async-proxy ones.
__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Arrive on the barrier (count 1) and expect `bytes` more bytes of transactions.
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}

// Box {x, y} of a 2-D tensor map into shared memory at dst; completes `box bytes` of
// transactions on bar. x must be a multiple of 16 bytes / element size (x = 0 here).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}

// tma_load_2d in a pair of CTAs (cta_group::2): into this CTA's shared memory, its bytes
// completed on the first CTA's barrier (bar: that barrier's address in this CTA).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    asm volatile(
        "{\n.reg .b32 b;\nmapa.shared::cluster.u32 b, %2, 0;\n"
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%3, %4}], [b];\n}"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}

// Box {x, y, z} of a 3-D tensor map (same rules as tma_load_2d).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}

// What a wait makes visible to the waiting thread: ACQ_CTA what threads of its CTA wrote before
// they arrived (and copies that completed on the barrier); ACQ_CLUSTER what threads of another
// CTA of the cluster did before an arrival released at cluster scope; ACQ_SHARED the same for
// shared memory alone, after fence_release_shared and a relaxed arrival (without the trip to L2
// that ordering global memory takes).
enum { ACQ_CTA = 0, ACQ_CLUSTER = 1, ACQ_SHARED = 2 };

// One try at the phase with the given parity, which may sleep up to hint_ns in hardware until it
// completes. ACQ_SHARED: relaxed, fence_acquire_shared is to follow.
template <int ACQ>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity, uint32_t hint_ns)
{
    uint32_t ok;
    if constexpr (ACQ == ACQ_CTA)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(hint_ns) : "memory");
    else if constexpr (ACQ == ACQ_CLUSTER)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(hint_ns) : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(hint_ns) : "memory");
    return ok != 0u;
}

__device__ __forceinline__ void fence_acquire_shared()
{
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

__device__ __forceinline__ void fence_release_shared()
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0u;
}

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;   // one second

// Wait for the phase with the given parity of the barrier to complete. Returns false
// if it has not completed after WAIT_LIMIT_NS.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (global_ns() - t0 > WAIT_LIMIT_NS) return false;
    }
}

// mbar_wait for stage rings, whose waits are short and many: each try may sleep in hardware
// until the phase completes (a hint of up to a millisecond) instead of polling, and the clock
// is read only after tries have failed (reading it takes longer than most waits last).
template <int ACQ = ACQ_CTA>
__device__ __forceinline__ bool mbar_wait_ring(uint32_t bar, uint32_t parity)
{
    bool ok = false;
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try<ACQ>(bar, parity, 1000000u);
    if (!ok) {
        const uint64_t t0 = global_ns();
        do ok = mbar_try<ACQ>(bar, parity, 1000000u);
        while (!ok && global_ns() - t0 <= WAIT_LIMIT_NS);
    }
    if constexpr (ACQ == ACQ_SHARED) fence_acquire_shared();
    return ok;
}

// About WAIT_LIMIT_NS, for copies in flight that nothing waits for any more to land.
__device__ __forceinline__ void linger()
{
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < WAIT_LIMIT_NS) __nanosleep(100000);
}

// 16-byte shared-memory accesses.
__device__ __forceinline__ void lds_v4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3)
{
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a));
}

__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}

}  // namespace bq
