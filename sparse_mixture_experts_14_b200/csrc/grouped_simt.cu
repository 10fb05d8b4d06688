// Ragged grouped products on the CUDA cores, fp32 arithmetic: with segments of
// rows per expert e (grouped.cuh),
//     mm     y_r  = W_e x_r                      rows [M][K] -> [M][N]
//     dgrad  dx_r = W_e^T dy_r                   rows [M][N] -> [M][K]
//     wgrad  dW_e = sum_{r in e} dy_r x_r^T      -> [E][N][K]
// A block computes a 128 x 128 tile of the output, 8 x 8 a thread, over slices
// of 16 of the reduction; the next slice is read into registers while this one
// is multiplied.  Sums run in ascending order of the reduction index.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int ST = 128, SK = 16, SPAD = ST + 4;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// One operand of the tile: element (i, k), i < ni along the tile, k < nk along the
// reduction, at base[i * ld + k] (KMAJ) or base[k * ld + i].
template <typename T, bool KMAJ>
struct Operand {
    const T* base;
    size_t ld;
    int ni, nk;
    float4 v[2];
    __device__ __forceinline__ void fetch(int k0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int i, k;
            if (KMAJ) {
                i = (threadIdx.x >> 2) + 64 * j;
                k = k0 + (threadIdx.x & 3) * 4;
            } else {
                k = k0 + (threadIdx.x >> 5) + 8 * j;
                i = (threadIdx.x & 31) * 4;
            }
            v[j] = i < ni && k < nk ? load4(base + (KMAJ ? (size_t)i * ld + k : (size_t)k * ld + i))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void put(float (*s)[SPAD]) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (KMAJ) {
                const int i = (threadIdx.x >> 2) + 64 * j, k = (threadIdx.x & 3) * 4;
                s[k][i] = v[j].x;
                s[k + 1][i] = v[j].y;
                s[k + 2][i] = v[j].z;
                s[k + 3][i] = v[j].w;
            } else {
                store4(&s[(threadIdx.x >> 5) + 8 * j][(threadIdx.x & 31) * 4], v[j]);
            }
        }
    }
};

template <typename TI, typename TO, int OP>
__global__ void __launch_bounds__(256) grouped_simt_kernel(const TI* __restrict__ rows, const TI* __restrict__ other,
                                                           TO* __restrict__ out, const Segments seg, int N, int K,
                                                           int* status) {
    pdl_trigger();
    pdl_wait();
    __shared__ SegTable tab;
    __shared__ __align__(16) float As[SK][SPAD];
    __shared__ __align__(16) float Bs[SK][SPAD];
    if (threadIdx.x < 32) build_segments(&tab, seg, ST, status);
    __syncthreads();
    constexpr bool AK = OP != kGroupedWgrad;   // reduction-contiguous operands
    constexpr bool BK = OP == kGroupedMm;
    Operand<TI, AK> a;
    Operand<TI, BK> b;
    int e, n_red, m_rows;
    TO* dst;
    size_t ldc;
    int row0 = 0, col0 = 0;
    if (OP == kGroupedWgrad) {
        if (tab.total == 0 && tab.base[seg.E] != 0) return;   // bad segments: nothing is written
        const int tk = (K + ST - 1) / ST, tn = (N + ST - 1) / ST;
        e = blockIdx.x / (tk * tn);
        const int n0 = blockIdx.x / tk % tn * ST, k0 = blockIdx.x % tk * ST;
        n_red = tab.rows[e];
        a.base = rows + (size_t)tab.row0[e] * N + n0;
        a.ld = N;
        a.ni = N - n0;
        b.base = other + (size_t)tab.row0[e] * K + k0;
        b.ld = K;
        b.ni = K - k0;
        dst = out + ((size_t)e * N + n0) * K + k0;
        ldc = K;
        m_rows = N - n0;
        col0 = k0;
    } else {
        const int ncol = OP == kGroupedMm ? N : K;
        n_red = OP == kGroupedMm ? K : N;
        const int tc = (ncol + ST - 1) / ST;
        const int tile = blockIdx.x / tc, c0 = blockIdx.x % tc * ST;
        if (tile >= tab.total) return;
        e = segment_of(&tab, seg.E, tile);
        const int r0 = (tile - tab.base[e]) * ST;
        row0 = tab.row0[e] + r0;
        m_rows = tab.rows[e] - r0;
        col0 = c0;
        a.base = rows + (size_t)row0 * n_red;
        a.ld = n_red;
        a.ni = m_rows;
        b.ni = ncol - c0;
        b.ld = K;
        b.base = other + (size_t)e * N * K + (OP == kGroupedMm ? (size_t)c0 * K : (size_t)c0);
        dst = out + (size_t)row0 * ncol + c0;
        ldc = ncol;
    }
    a.nk = b.nk = n_red;
    const int n_cols = b.ni;
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (n_red > 0) {
        a.fetch(0);
        b.fetch(0);
    }
    for (int k0 = 0; k0 < n_red; k0 += SK) {
        a.put(As);
        b.put(Bs);
        __syncthreads();
        if (k0 + SK < n_red) {
            a.fetch(k0 + SK);
            b.fetch(k0 + SK);
        }
#pragma unroll
        for (int c = 0; c < SK; ++c) {
            float av[8], bv[8];
            *reinterpret_cast<float4*>(av) = *reinterpret_cast<const float4*>(&As[c][ty * 4]);
            *reinterpret_cast<float4*>(av + 4) = *reinterpret_cast<const float4*>(&As[c][64 + ty * 4]);
            *reinterpret_cast<float4*>(bv) = *reinterpret_cast<const float4*>(&Bs[c][tx * 4]);
            *reinterpret_cast<float4*>(bv + 4) = *reinterpret_cast<const float4*>(&Bs[c][64 + tx * 4]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = (i >> 2) * 64 + ty * 4 + (i & 3);
        if (m >= m_rows) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = h * 64 + tx * 4;
            if (n < n_cols)
                store4(dst + (size_t)m * ldc + n,
                       make_float4(acc[i][4 * h], acc[i][4 * h + 1], acc[i][4 * h + 2], acc[i][4 * h + 3]));
        }
    }
}

template <typename TI, typename TO, int OP>
cudaError_t launch(const GroupedArgs& a, cudaStream_t s) {
    long long tiles;
    if (OP == kGroupedWgrad) {
        tiles = (long long)a.seg.E * ((a.N + ST - 1) / ST) * ((a.K + ST - 1) / ST);
    } else {
        const int ncol = OP == kGroupedMm ? a.N : a.K;
        tiles = ((long long)a.seg.M / ST + a.seg.E) * ((ncol + ST - 1) / ST);
    }
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(grouped_simt_kernel<TI, TO, OP>, dim3((unsigned)tiles), dim3(256), 0, s,
                      static_cast<const TI*>(a.rows), static_cast<const TI*>(a.other), static_cast<TO*>(a.out), a.seg,
                      a.N, a.K, a.status);
}

template <typename TI, typename TO>
cudaError_t launch_op(const GroupedArgs& a, cudaStream_t s) {
    switch (a.op) {
        case kGroupedMm: return launch<TI, TO, kGroupedMm>(a, s);
        case kGroupedDgrad: return launch<TI, TO, kGroupedDgrad>(a, s);
        default: return launch<TI, TO, kGroupedWgrad>(a, s);
    }
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t s) {
    if (!a.in16) return launch_op<float, float>(a, s);
    return a.out16 ? launch_op<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_op<__nv_bfloat16, float>(a, s);
}

}  // namespace moe
