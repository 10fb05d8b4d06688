// PTX wrappers of the ragged grouped products beyond those of ptx_sm100.cuh.
#pragma once

#include "ptx_sm100.cuh"

namespace moe {
namespace ptx {

// Arrive on an mbarrier of either CTA of the pair after this thread (or, behind a __syncwarp, its warp) has
// prepared tcgen05.mma operands in its own CTA's shared memory and called fence_proxy_async.  The operands
// are read through the asynchronous proxy, which that fence orders; an arrive with cluster-wide release would
// also wait for every other access of the thread.
__device__ __forceinline__ void mbar_arrive_operands(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// This thread's shared-memory writes become visible to the asynchronous proxy (tcgen05.mma operands).
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Descriptor of a K-major bf16 tile whose rows of 32, 64 or 128 bytes are swizzled over their own length:
// 8-row groups follow each other (the stride byte offset), layout type 6, 4 or 2.  The fields are those of
// desc_kmajor_sw128.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t saddr, int row_bytes) {
    const uint64_t layout = row_bytes == 128 ? 2 : row_bytes == 64 ? 4 : 6;
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(8 * row_bytes >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= layout << 61;
    return d;
}

// Two fp32 fused multiply-adds in one instruction, each rounded as fmaf rounds.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// One warp's 16 x 8 += 16 x 16 times 16 x 8, bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a cluster's shared memory.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 16 bytes to shared memory; zeros where !live (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

}  // namespace ptx
}  // namespace moe
