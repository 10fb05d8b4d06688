// Grouped products for few rows per expert (decode batches), bf16, rows [M][K] -> [M][N]:
//     y_r = W_e x_r  (+ B_{a,e} u_r, the adapters' second half; lora.cu computes u)
// What bounds it is reading the weights of the experts that have rows, once.  A block
// takes 32 features of one expert and up to 8 NT of its rows; its 8 warps interleave
// over the reduction in steps of 32, so that a block reads 512 contiguous bytes of
// each weight row at a time and a matrix of 4096 features gives 128 blocks per expert:
// enough bytes in flight on every SM without a ring in shared memory (the 256-feature
// tiles of grouped_tc.cu give 16 pairs of CTAs there).
//
// mma.m16n8k16 with the weights as the 16 rows and x's rows as the 8 columns; both come
// straight from global memory, 16 bytes a lane, the k order inside a step permuted the
// same way on both sides.  The warps' partial sums are added in warp order through
// shared memory.
//
// Measured: 32 rows of 8 experts, 4096 x 14336, 148 us (6.34 TB/s); one token's two experts, 14336 x 4096, 43 us.
//
// Adapters: an output's own B row and u row are multiplied on the CUDA cores after that.
// Only there does the block wait for the kernel that makes u: the weights stream
// while that one runs.
#include "grouped.cuh"
#include "ptx_grouped.cuh"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int MT = 2;                  // 16-feature tiles of a warp
constexpr int FEATURES = 16 * MT;      // of a block

struct FewParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* W;
    void* out;
    Segments seg;
    int N, K;
    LoraView lora;
    int* status;
};

// Weights are read once: past L1.
__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int NT, bool OUT16, bool LORA>
__global__ void __launch_bounds__(32 * WARPS, 2) grouped_few_kernel(const FewParams p) {
    constexpr int ROWS = 8 * NT;
    constexpr int U = 4;                   // steps whose loads are in flight together
    constexpr int PITCH = FEATURES + 1;
    __shared__ SegTable seg;
    __shared__ float red[WARPS][ROWS][PITCH];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!LORA) pdl_wait();   // (adapters: the kernel before has waited for everything but u)
    pdl_trigger();
    if (warp == 0) build_segments(&seg, p.seg, ROWS, blockIdx.x == 0 ? p.status : nullptr);
    __syncthreads();
    const int nf = (p.N + FEATURES - 1) / FEATURES;
    if ((int)blockIdx.x >= seg.total * nf) {
        if (LORA) pdl_wait();
        return;
    }
    // row tiles fastest: they share the weights through L2
    const int e = segment_of(&seg, p.seg.E, blockIdx.x / nf);
    const int tt = seg.base[e + 1] - seg.base[e], local = blockIdx.x - seg.base[e] * nf;
    const int f0 = local / tt * FEATURES, r0 = local % tt * ROWS;
    const int rows = min(ROWS, seg.rows[e] - r0);
    const size_t row0 = (size_t)seg.row0[e] + r0;
    const int K = p.K, N = p.N, g = lane >> 2, q = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);

    // this lane's rows: features f0 + 16 i + 8 j + g, rows r0 + 8 t + g
    const __nv_bfloat16* w[MT][2];
    bool wl[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int f = f0 + 16 * i + 8 * j + g;
            wl[i][j] = f < N;
            w[i][j] = p.W + ((size_t)e * N + (f < N ? f : 0)) * K + 8 * q;
        }
    const __nv_bfloat16* x[NT];
    bool xl[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + g;
        xl[t] = r < rows;
        x[t] = p.x + (row0 + (r < rows ? r : 0)) * K + 8 * q;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][t][c] = 0.f;
    if (LORA) {
        // the adapters' rows of B that this thread's outputs need, on their way to L2 meanwhile
        for (int o = tid; o < rows * FEATURES; o += 32 * WARPS) {
            const int id = p.lora.adapter[row0 + o / FEATURES], f = f0 + o % FEATURES;
            if (f >= N || id < 0 || id >= p.lora.L) continue;
            const __nv_bfloat16* bl = p.lora.B + (((size_t)id * p.seg.E + e) * N + f) * p.lora.R;
            for (int j = 0; j < p.lora.R; j += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(bl + j));
        }
    }
    for (int k0 = warp * 32; k0 < K; k0 += WARPS * 32 * U) {
        uint4 a[U][MT][2], b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * WARPS * 32;
            const bool in = k + 8 * q < K;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) a[u][i][j] = in && wl[i][j] ? load_stream(w[i][j] + k) : zero;
#pragma unroll
            for (int t = 0; t < NT; ++t)
                b[u][t] = in && xl[t] ? __ldg(reinterpret_cast<const uint4*>(x[t] + k)) : zero;
        }
        // fp32 outputs: the tensor cores truncate as they accumulate, so they take a few steps at a time and
        // the sums go on with rounding (a reduction of 14336: error 1.8e-6 -> 1.5e-7 of the result)
        float part[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) part[i][t][c] = OUT16 ? acc[i][t][c] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    ptx::mma16816(part[i][t], a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y, b[u][t].x,
                                  b[u][t].y);
                    ptx::mma16816(part[i][t], a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w, b[u][t].z,
                                  b[u][t].w);
                }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][t][c] = OUT16 ? part[i][t][c] : acc[i][t][c] + part[i][t][c];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                red[warp][8 * t + 2 * q + (c & 1)][16 * i + 8 * (c >> 1) + g] = acc[i][t][c];
    if (LORA) pdl_wait();   // u, from here on
    __syncthreads();
    for (int o = tid; o < rows * FEATURES; o += 32 * WARPS) {
        const int r = o / FEATURES, fl = o % FEATURES, f = f0 + fl;
        if (f >= N) continue;
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) s += red[v][r][fl];
        if (LORA) {
            const int id = p.lora.adapter[row0 + r];
            if (id >= 0 && id < p.lora.L) {
                const size_t ae = (size_t)id * p.seg.E + e;
                if (!OUT16) s += adapter_term<3>(p.lora, ae, N, row0 + r, f);
                else s += p.lora.terms == 2 ? adapter_term<2>(p.lora, ae, N, row0 + r, f)
                                            : adapter_term<1>(p.lora, ae, N, row0 + r, f);
            }
        }
        const size_t at = (row0 + r) * N + f;
        if (OUT16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s);
        else static_cast<float*>(p.out)[at] = s;
    }
}

template <int NT, bool OUT16, bool LORA>
cudaError_t launch(const GroupedArgs& a, const FewParams& p, cudaStream_t s) {
    long long t = (long long)a.seg.M / (8 * NT) + a.seg.E;
    const long long high = (long long)a.seg.E * ((a.seg.most + 8LL * NT - 1) / (8 * NT));
    if (t > high) t = high;
    const long long blocks = (t < a.seg.M ? t : a.seg.M) * ((a.N + FEATURES - 1) / FEATURES);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(grouped_few_kernel<NT, OUT16, LORA>, dim3((unsigned)blocks), dim3(32 * WARPS), 0, s, p);
}

template <int NT>
cudaError_t launch_rows(const GroupedArgs& a, const FewParams& p, cudaStream_t s) {
    if (a.A) return a.out16 ? launch<NT, true, true>(a, p, s) : launch<NT, false, true>(a, p, s);
    return a.out16 ? launch<NT, true, false>(a, p, s) : launch<NT, false, false>(a, p, s);
}

}  // namespace

// Packed segments (no counts): this kernel for up to 8 rows per expert on average, or 32 in all.  Measured
// (8 experts, 14336 x 4096; us here, us on 256-feature tiles): 8 rows 143, 159; 32 rows 162, 196; 64 rows 178, 198;
// 128 rows 304, 197.  With counts M is the capacity and says little about the rows (a dispatch pads every
// expert to 128 and leaves room for 127 more): up to 144 of it per expert both kernels are launched, each for the
// segments it suits (32 rows in padded segments: 170 us, 194 on 256-feature tiles alone; 256 rows: 213, 197).
Choice grouped_choice(const GroupedArgs& a) {
    if (a.op != kGroupedMm) return {false, true, 0};
    const bool few = a.seg.M <= 32 || a.seg.M <= 8LL * a.seg.E;
    if (few || !a.seg.counts || a.seg.M > 144LL * a.seg.E) return {few, !few, 0};
    return {true, true, 16};
}

cudaError_t launch_grouped_few(const GroupedArgs& a, cudaStream_t s) {
    FewParams p{};
    p.x = static_cast<const __nv_bfloat16*>(a.rows);
    p.W = static_cast<const __nv_bfloat16*>(a.other);
    p.out = a.out;
    p.seg = a.seg;
    p.N = a.N;
    p.K = a.K;
    if (a.A) p.lora = lora_view(a);
    p.status = a.status;
    // 8 rows of a segment to a block, or 16 where segments surely have more than a dozen: a second block that
    // finds the weights in L2 costs less than the wider one's registers (us with 8 and 16: 64 rows of 8 experts
    // 178, 190; 16 rows of one, 4096 x 4096, 16.4, 18.4; 24 rows 22.5, 18.4).
    if (a.seg.counts || a.seg.M <= 16LL * a.seg.E) return launch_rows<1>(a, p, s);
    return launch_rows<2>(a, p, s);
}

}  // namespace moe
