// Low-rank adapters beside a grouped product, first half: u_r = s_a A_{a,e} x_r for
// every row r of expert e's segment with adapter a = adapter[r] (-1: none, the row
// takes no part), rounded once to bf16, the operand type of the second half
// y_r = W_e x_r + B_{a,e} u_r (grouped_tc.cu).
//
// A block takes a window of a segment's rows (64, or 16 where that gives too few
// windows for the SMs), finds the adapters that occur in it and, for each, gathers
// its rows in groups of 16 for mma.m16n8k16: x's rows are the 16 rows, A's ranks the
// columns.  Both are read from global memory straight into fragments, 16 bytes a
// lane: the k order inside a 32-wide step is permuted the same way for both sides.  The
// 8 warps interleave over the reduction and add their partial sums in a fixed order
// through shared memory.  What bounds it is reading x and the adapters once per window.
//
// Further blocks of the same launch write down, for every column tile of the
// product, the adapters that occur among its rows, each once, in order of first
// occurrence.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int RED_BYTES = 64 * 1024;

struct ShrinkParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* A;
    const float* scale;
    LoraView v;
    Segments seg;
    int K;
    int window;    // rows of a window
    int windows;   // blocks of the first kind (an upper bound of the windows)
    int* status;
};

struct ShrinkSmem {
    SegTable seg;
    int ids[kColumnTile];
    int list[kColumnTile];
    int rows[64];
    int warp_n[WARPS];
    int n, m;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The distinct ids of ids[0, n), in order of first occurrence, into list; sm->n of them (all threads).
__device__ __forceinline__ void distinct(ShrinkSmem* sm, int n) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    bool first = t < n && sm->ids[t] >= 0;
    for (int j = 0; j < t && first; ++j) first = sm->ids[j] != sm->ids[t];
    const uint32_t b = __ballot_sync(0xffffffffu, first);
    if (lane == 0) sm->warp_n[warp] = __popc(b);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sm->warp_n[w];
        total += sm->warp_n[w];
    }
    if (first) sm->list[before + __popc(b & ((1u << lane) - 1))] = sm->ids[t];
    if (t == 0) sm->n = total;
    __syncthreads();
}

// A row's adapter; an id that is none and no adapter is an error, the row then gets none.
__device__ __forceinline__ int adapter_of(const ShrinkParams& p, size_t r) {
    const int id = p.v.adapter[r];
    if (id >= 0 && id < p.v.L) return id;
    if (id != -1) record_status(p.status, MOE_ERR_DEVICE);
    return -1;
}

// NT: tiles of 8 ranks (R <= 8 NT); G: groups of 16 rows at a time.
template <int NT, int G>
__global__ void __launch_bounds__(32 * WARPS) lora_shrink_kernel(const ShrinkParams p) {
    extern __shared__ __align__(16) float red[];   // [WARPS][G * 16][NT * 8]
    __shared__ ShrinkSmem sm;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool lists = (int)blockIdx.x >= p.windows;
    if (warp == 0) build_segments(&sm.seg, p.seg, lists ? kColumnTile : p.window, p.status);
    __syncthreads();
    const int tile = lists ? blockIdx.x - p.windows : blockIdx.x;
    if (tile >= sm.seg.total) return;
    const int e = segment_of(&sm.seg, p.seg.E, tile);
    const int rows = sm.seg.rows[e], h = lists ? column_tile_height(rows) : p.window;
    const int r0 = (tile - sm.seg.base[e]) * h, n = min(h, rows - r0);
    const size_t row0 = (size_t)sm.seg.row0[e] + r0;
    if ((int)threadIdx.x < n) sm.ids[threadIdx.x] = adapter_of(p, row0 + threadIdx.x);
    __syncthreads();
    distinct(&sm, n);
    const int na = sm.n;
    if (lists) {
        if ((int)threadIdx.x < na) p.v.tile_list[(size_t)tile * kColumnTile + threadIdx.x] = sm.list[threadIdx.x];
        if (threadIdx.x == 0) p.v.tile_count[tile] = na;
        return;
    }
    const int R = p.v.R, K = p.K;
    const int g = lane >> 2, q = lane & 3;
    for (int i = 0; i < na; ++i) {
        const int a = sm.list[i];
        // this adapter's rows of the window, in order (the window has at most 64)
        if (warp < 2) {
            const uint32_t b0 = __ballot_sync(0xffffffffu, lane < n && sm.ids[lane] == a);
            const uint32_t b1 = __ballot_sync(0xffffffffu, lane + 32 < n && sm.ids[lane + 32] == a);
            const uint32_t mine = warp ? b1 : b0;
            if (mine >> lane & 1)
                sm.rows[(warp ? __popc(b0) : 0) + __popc(mine & ((1u << lane) - 1))] = warp * 32 + lane;
            if (threadIdx.x == 0) sm.m = __popc(b0) + __popc(b1);
        }
        __syncthreads();
        const int m = sm.m;
        const __nv_bfloat16* Aa = p.A + ((size_t)a * p.seg.E + e) * R * K;
        const float scale = p.scale[a];
        for (int m0 = 0; m0 < m; m0 += 16 * G) {
            float acc[G][NT][4];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[u][t][c] = 0.f;
            const __nv_bfloat16* xr[G][2];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = m0 + 16 * u + 8 * j + g;
                    xr[u][j] = r < m ? p.x + (row0 + sm.rows[r]) * K : nullptr;
                }
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
            for (int k0 = warp * 32; k0 < K; k0 += WARPS * 32) {
                const int k = k0 + 8 * q;
                const bool in = k < K;
                uint4 bv[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    bv[t] = in && t * 8 + g < R
                                ? __ldg(reinterpret_cast<const uint4*>(Aa + (size_t)(t * 8 + g) * K + k))
                                : zero;
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    if (u > 0 && m0 + 16 * u >= m) break;
                    const uint4 lo = in && xr[u][0] ? __ldg(reinterpret_cast<const uint4*>(xr[u][0] + k)) : zero;
                    const uint4 hi = in && xr[u][1] ? __ldg(reinterpret_cast<const uint4*>(xr[u][1] + k)) : zero;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma16816(acc[u][t], lo.x, hi.x, lo.y, hi.y, bv[t].x, bv[t].y);
                        mma16816(acc[u][t], lo.z, hi.z, lo.w, hi.w, bv[t].z, bv[t].w);
                    }
                }
            }
            float* mine = red + (size_t)warp * G * 16 * NT * 8;
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        mine[(16 * u + g + 8 * (c >> 1)) * (NT * 8) + t * 8 + 2 * q + (c & 1)] = acc[u][t][c];
            __syncthreads();
            for (int o = threadIdx.x; o < G * 16 * NT * 8; o += 32 * WARPS) {
                const int r = m0 + o / (NT * 8), j = o % (NT * 8);
                if (r >= m || j >= p.v.R16) continue;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) s += red[(size_t)w * G * 16 * NT * 8 + o];
                p.v.u[(row0 + sm.rows[r]) * p.v.R16 + j] = __float2bfloat16_rn(j < R ? s * scale : 0.f);
            }
            __syncthreads();
        }
    }
}

template <int NT, int G>
cudaError_t launch(const ShrinkParams& p, int blocks, cudaStream_t s) {
    static_assert(WARPS * G * 16 * NT * 8 * 4 <= RED_BYTES, "reduction buffer");
    static PerDeviceOnce attr;
    const cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(lora_shrink_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, RED_BYTES);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(lora_shrink_kernel<NT, G>, dim3(blocks), dim3(32 * WARPS), RED_BYTES, s, p);
}

}  // namespace

cudaError_t launch_lora_shrink(const GroupedArgs& a, cudaStream_t s) {
    ShrinkParams p{};
    p.x = static_cast<const __nv_bfloat16*>(a.rows);
    p.A = static_cast<const __nv_bfloat16*>(a.A);
    p.scale = a.scale;
    p.v = lora_view(a);
    p.seg = a.seg;
    p.K = a.K;
    p.status = a.status;
    const int M = a.seg.M, E = a.seg.E, sms = a.num_sms > 0 ? a.num_sms : 148;
    p.window = M >= 64 * sms ? 64 : 16;
    const long long w = (long long)M / p.window + E;
    p.windows = (int)(w < M ? w : M);
    const long long t = (long long)M / kColumnTile + E;
    const int blocks = p.windows + (int)(t < M ? t : M);
    if (a.R <= 16) return launch<2, 4>(p, blocks, s);
    if (a.R <= 32) return launch<4, 4>(p, blocks, s);
    if (a.R <= 64) return launch<8, 2>(p, blocks, s);
    return launch<16, 1>(p, blocks, s);
}

}  // namespace moe
