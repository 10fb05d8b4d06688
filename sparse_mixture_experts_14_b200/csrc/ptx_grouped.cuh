// PTX wrappers of the ragged grouped products beyond those of ptx_sm100.cuh.
#pragma once

#include "ptx_sm100.cuh"

namespace moe {
namespace ptx {

// mbar_wait for a phase that threads of the other CTA of the pair arrive on:
// their writes before the (releasing) arrive are visible afterwards.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
    const uint32_t addr = smem_addr(bar);
    const uint64_t t0 = global_timer_ns();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*w.abort) return false;
        if (global_timer_ns() - t0 > w.limit_ns) {
            record_status(w.status, MOE_ERR_TIMEOUT);
            *w.abort = 1;
            return false;
        }
    }
}

// This thread's shared-memory writes become visible to the asynchronous proxy (tcgen05.mma operands).
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Descriptor of a K-major bf16 tile with 32-byte swizzle: rows of 32 bytes (16 bf16), 8-row groups of
// 256 bytes (the stride byte offset); layout type 6.  The fields are those of desc_kmajor_sw128.
__device__ __forceinline__ uint64_t desc_kmajor_sw32(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(256 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(6) << 61;
    return d;
}

}  // namespace ptx
}  // namespace moe
