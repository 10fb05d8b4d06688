// Low-rank adapters beside a grouped product: u_r = s_a A_{a,e} x_r for every row r
// of expert e's segment with adapter a = adapter[r] (a row without adapter, -1,
// takes no part), the first half of y_r = W_e x_r + B_{a,e} u_r.
// One warp computes one element of u.
#include "grouped.cuh"

namespace moe {
namespace {

__global__ void __launch_bounds__(256) lora_shrink_kernel(const __nv_bfloat16* __restrict__ x,
                                                          const __nv_bfloat16* __restrict__ A,
                                                          const float* __restrict__ scale,
                                                          const int32_t* __restrict__ adapter, const Segments seg,
                                                          int K, int L, int R, float* __restrict__ u, int* status) {
    pdl_trigger();
    pdl_wait();
    __shared__ SegTable tab;
    if (threadIdx.x < 32) build_segments(&tab, seg, 1, status);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const long long total = (long long)tab.total * R;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
        const int t = (int)(i / R), j = (int)(i % R);
        const int e = segment_of(&tab, seg.E, t);
        const size_t r = (size_t)tab.row0[e] + (t - tab.base[e]);
        const int a = adapter[r];
        if (a < 0 || a >= L) {   // -1: no adapter; anything else is an error, the row gets none
            if (a != -1 && lane == 0) record_status(status, MOE_ERR_DEVICE);
            continue;
        }
        const uint4* xr = reinterpret_cast<const uint4*>(x + r * K);
        const uint4* ar = reinterpret_cast<const uint4*>(A + (((size_t)a * seg.E + e) * R + j) * K);
        float s = 0.f;
        for (int k = lane; k < K / 8; k += 32) {
            const uint4 p = __ldg(xr + k), q = __ldg(ar + k);
            s += bf16_lo(p.x) * bf16_lo(q.x) + bf16_hi(p.x) * bf16_hi(q.x) + bf16_lo(p.y) * bf16_lo(q.y) +
                 bf16_hi(p.y) * bf16_hi(q.y) + bf16_lo(p.z) * bf16_lo(q.z) + bf16_hi(p.z) * bf16_hi(q.z) +
                 bf16_lo(p.w) * bf16_lo(q.w) + bf16_hi(p.w) * bf16_hi(q.w);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) u[r * R + j] = s * scale[a];
    }
}

}  // namespace

size_t lora_workspace_bytes(int M, int E, int L, int R) {
    (void)E;
    (void)L;
    return align_up((size_t)M * R * 4, 256);
}

cudaError_t launch_lora_shrink(const GroupedArgs& a, cudaStream_t s) {
    const long long warps = (long long)a.seg.M * a.R;
    const long long blocks = (warps + 7) / 8;
    const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
    return launch_pdl(lora_shrink_kernel, dim3(grid), dim3(256), 0, s, static_cast<const __nv_bfloat16*>(a.rows),
                      static_cast<const __nv_bfloat16*>(a.A), a.scale, a.adapter, a.seg, a.K, a.L, a.R,
                      reinterpret_cast<float*>(a.ws), a.status);
}

}  // namespace moe
