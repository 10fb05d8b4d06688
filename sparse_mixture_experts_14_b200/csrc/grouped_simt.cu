// Ragged grouped products in fp32 on the CUDA cores: with segments of rows per
// expert e (grouped.cuh),
//     mm     y_r  = W_e x_r                      rows [M][K] -> [M][N]
//     dgrad  dx_r = W_e^T dy_r                   rows [M][N] -> [M][K]
//     wgrad  dW_e = sum_{r in e} dy_r x_r^T      -> [E][N][K]
// A block computes BM rows x 128 columns of the output over slices of BK of the
// reduction; the next ones are read into registers while this one is multiplied.
// BM is 128 (8 x 8 outputs a thread), or 64, 32 or 8 (8 x 4) where segments have few rows:
// there the weights' bytes bound the product, as long as no more than the rows' own work is
// done on them.  The thread groups of a low tile split every slice, and where tiles are few,
// the blocks of a cluster split the reduction; their sums are added through (distributed)
// shared memory in a fixed order.
//
// Measured: 6296 rows of 7 experts, 1416 x 1264, 0.57 ms (0.67 with a product to an instruction); 1003 rows
// of 5, 79 us; weight gradients of 8192 rows, 4 experts of 2048 x 1024, 0.68 ms (51 TFLOP/s; 0.92 with one).
// What bounds it is the multiply-adds (73 % of the FMA pipe), and the last wave of blocks where it is not full.  One
// or two experts are one or two library products, which are ahead there (mm of 96 rows, 4096 x 2048, 103 us against
// 56; dgrad of 128 rows, 12032 x 104, 175 against 72): few tiles of 128 columns, and at most 8 parts of the reduction.
//
// Every output's part of the reduction is one chain of rounded additions: RMS error 7.6e-7 to 1.1e-6 of the result at a
// reduction of 14336, where the library's fp32 product has 2.1e-6.
//
// Operands lie in shared memory with the reduction outermost.  Those that are read along
// the reduction are turned on the way in; in the low tiles, where the weights' way into
// shared memory is most of the work, the columns of row k are permuted by k / 4 (in groups
// of 4), so that a warp's scattered stores meet 32 different banks (15 rows, 8 experts,
// 7592 x 6240: 344 -> 197 us).
#include "grouped.cuh"
#include "ptx_grouped.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int BN = 128;
constexpr int MAX_SPLIT = 8;

template <int BM_>
struct Tile {
    static constexpr int BM = BM_;
    static constexpr int TM = 8, TN = BM == 128 ? 8 : 4;
    static constexpr int LANES = (BM / TM) * (BN / TN);   // threads that cover the tile once
    static constexpr int G = THREADS / LANES;             // thread groups
    static constexpr int BK = BM == 128 ? 16 : 32;
    static constexpr int APITCH = BM == 32 || BM == 64 ? BM : BM + 4, BPITCH = BM == 128 ? BN + 4 : BN;
    static constexpr int SLICE = BK * (APITCH + BPITCH);   // floats
    static constexpr int OPERANDS = 2 * SLICE * 4;         // two slices in turn
    // slices on their way in registers: two where the weights' bytes bound the product (dgrad, 15 rows of 8
    // experts, 7592 x 6240: 257 -> 233 us; in tiles of 32 rows the registers are short: 478 rows of 26, 306 -> 380)
    static constexpr int AHEAD = BM == 8 ? 2 : 1;
    static constexpr int SUMS = G * BM * BN * 4;
    static constexpr int SMEM = OPERANDS > SUMS ? OPERANDS : SUMS;
    // Two products to an instruction (fma.rn.f32x2): of neighbouring columns, or of neighbouring rows.  The
    // other factor is doubled on the way, so the fewer of those the better (200 rows of 8 experts, 4096 x 2048:
    // 176 us in columns, 160 in rows); the high tile has as many of either and fewer registers to spare in rows
    // (6296 rows of 7, 1416 x 1264: 569 in columns, 610 in rows).
    static constexpr bool COLS = BM == 128;
    static constexpr int AM = COLS ? TM : TM / 2, AN = COLS ? TN / 2 : TN;   // a thread's sums, in pairs
    // the row and the column of a thread's i-th and j-th output
    __device__ static int row(int ty, int i) { return BM == 128 ? (i >> 2) * 64 + ty * 4 + (i & 3) : ty * 8 + i; }
    __device__ static int col(int tx, int j) { return TN == 8 ? (j >> 2) * 64 + tx * 4 + (j & 3) : tx * 4 + j; }
};

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// One operand of the tile: element (i, k), i < ni along the tile, k in [k0, nk) along the reduction, at
// base[i * ld + k] (KMAJ) or base[k * ld + i].
template <int ROWS, int BK, bool KMAJ, int AHEAD>
struct Operand {
    static constexpr int VECS = ROWS * BK / 4;
    static constexpr int NV = (VECS + THREADS - 1) / THREADS;
    const float* base;
    size_t ld;
    int ni, nk;
    float4 v[AHEAD][NV];
    __device__ __forceinline__ void place(int j, int& i, int& k) const {
        const int x = threadIdx.x + THREADS * j;
        if (KMAJ) {
            i = x / (BK / 4);
            k = x % (BK / 4) * 4;
        } else {
            k = x / (ROWS / 4);
            i = x % (ROWS / 4) * 4;
        }
    }
    __device__ __forceinline__ void fetch(int k0, int d) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            int i, k;
            place(j, i, k);
            k += k0;
            const bool in = (VECS % THREADS == 0 || (int)threadIdx.x + THREADS * j < VECS) && i < ni && k < nk;
            v[d][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) v[d][j] = load4(base + (KMAJ ? (size_t)i * ld + k : (size_t)k * ld + i));
        }
    }
    // position of column i in row k
    static __device__ __forceinline__ int at(int i, int k) {
        return BK == 32 && ROWS >= 32 ? i ^ ((k >> 2) % (BK / 4) * 4) : i;
    }
    __device__ __forceinline__ void put(float* s, int pitch, int d) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (VECS % THREADS != 0 && (int)threadIdx.x + THREADS * j >= VECS) continue;
            int i, k;
            place(j, i, k);
            if (KMAJ) {
                float* p = s + k * pitch + at(i, k);   // (k is a multiple of 4: one permutation for all four)
                p[0] = v[d][j].x;
                p[pitch] = v[d][j].y;
                p[2 * pitch] = v[d][j].z;
                p[3 * pitch] = v[d][j].w;
            } else {
                *reinterpret_cast<float4*>(s + k * pitch + at(i, k)) = v[d][j];
            }
        }
    }
};

template <int OP, int BM_>
__global__ void __launch_bounds__(THREADS, 2)
    grouped_simt_kernel(const float* __restrict__ rows, const float* __restrict__ other, float* __restrict__ out,
                        const Segments seg, int N, int K, int split, int* status) {
    using T = Tile<BM_>;
    constexpr int BK = T::BK;
    extern __shared__ __align__(16) float sm[];
    __shared__ SegTable tab;
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) build_segments(&tab, seg, BM_, blockIdx.x == 0 ? status : nullptr);
    __syncthreads();
    const int part = blockIdx.x % split, tile = blockIdx.x / split;   // CTA of the cluster, cluster
    Operand<BM_, BK, OP != kGroupedWgrad, T::AHEAD> a;
    Operand<BN, BK, OP == kGroupedMm, T::AHEAD> b;
    int red, m_rows, n_cols;   // reduction, rows and columns of the tile that exist
    float* dst;
    size_t ldc;
    if (OP == kGroupedWgrad) {
        if (!tab.good) return;   // bad segments: nothing is written
        const int tk = (K + BN - 1) / BN, tn = (N + BM_ - 1) / BM_;
        const int e = tile / (tk * tn), n0 = tile / tk % tn * BM_, k0 = tile % tk * BN;
        red = tab.rows[e];
        a.base = rows + (size_t)tab.row0[e] * N + n0;
        a.ld = N;
        m_rows = N - n0;
        b.base = other + (size_t)tab.row0[e] * K + k0;
        b.ld = K;
        n_cols = K - k0;
        dst = out + ((size_t)e * N + n0) * K + k0;
        ldc = K;
    } else {
        const int ncol = OP == kGroupedMm ? N : K;
        red = OP == kGroupedMm ? K : N;
        const int tc = (ncol + BN - 1) / BN;
        if (tile >= tab.total * tc) return;   // the whole cluster
        // row tiles fastest: they share the weights through L2
        const int e = segment_of(&tab, seg.E, tile / tc);
        const int tt = tab.base[e + 1] - tab.base[e], local = tile - tab.base[e] * tc;
        const int r0 = local % tt * BM_, c0 = local / tt * BN;
        const size_t row0 = (size_t)tab.row0[e] + r0;
        m_rows = tab.rows[e] - r0;
        n_cols = ncol - c0;
        a.base = rows + row0 * red;
        a.ld = red;
        b.base = other + (size_t)e * N * K + (OP == kGroupedMm ? (size_t)c0 * K : (size_t)c0);
        b.ld = K;
        dst = out + row0 * ncol + c0;
        ldc = ncol;
    }
    a.ni = m_rows;
    b.ni = n_cols;
    a.nk = b.nk = red;
    const int slices = (red + BK - 1) / BK;
    const int s0 = (int)((long long)slices * part / split), s1 = (int)((long long)slices * (part + 1) / split);
    float2 acc[T::AM][T::AN];
#pragma unroll
    for (int i = 0; i < T::AM; ++i)
#pragma unroll
        for (int j = 0; j < T::AN; ++j) acc[i][j] = make_float2(0.f, 0.f);
    const int group = threadIdx.x / T::LANES, lane = threadIdx.x % T::LANES;
    const int tx = lane % (BN / T::TN), ty = lane / (BN / T::TN);
#pragma unroll
    for (int d = 0; d < T::AHEAD; ++d)
        if (s0 + d < s1) {
            a.fetch((s0 + d) * BK, d);
            b.fetch((s0 + d) * BK, d);
        }
    for (int t = s0; t < s1; t += T::AHEAD) {
#pragma unroll
        for (int d = 0; d < T::AHEAD; ++d) {
            const int s = t + d;
            if (s >= s1) break;
            // (the slice before the last was read by everyone before the barrier of the last one)
            float* As = sm + (s & 1) * T::SLICE;
            float* Bs = As + BK * T::APITCH;
            a.put(As, T::APITCH, d);
            b.put(Bs, T::BPITCH, d);
            __syncthreads();
            if (s + T::AHEAD < s1) {
                a.fetch((s + T::AHEAD) * BK, d);
                b.fetch((s + T::AHEAD) * BK, d);
            }
#pragma unroll
            for (int i = 0; i < BK / T::G; ++i) {
                const int c = group * (BK / T::G) + i;
                __align__(16) float av[T::TM], bv[T::TN];
#pragma unroll
                for (int h = 0; h < T::TM; h += 4)
                    *reinterpret_cast<float4*>(av + h) =
                        *reinterpret_cast<const float4*>(As + c * T::APITCH + a.at(T::row(ty, h), c));
#pragma unroll
                for (int h = 0; h < T::TN; h += 4)
                    *reinterpret_cast<float4*>(bv + h) =
                        *reinterpret_cast<const float4*>(Bs + c * T::BPITCH + b.at(T::col(tx, h), c));
#pragma unroll
                for (int m = 0; m < T::AM; ++m)
#pragma unroll
                    for (int n = 0; n < T::AN; ++n) {
                        float2 p, q;
                        if constexpr (T::COLS) {
                            p = make_float2(av[m], av[m]);
                            q = make_float2(bv[2 * n], bv[2 * n + 1]);
                        } else {
                            p = make_float2(av[2 * m], av[2 * m + 1]);
                            q = make_float2(bv[n], bv[n]);
                        }
                        acc[m][n] = ptx::fma2(p, q, acc[m][n]);
                    }
            }
        }
    }
    // outputs (i, j) to (i, j + 3) of the thread
    auto sums = [&](int i, int j) {
        if constexpr (T::COLS) {
            return make_float4(acc[i][j / 2].x, acc[i][j / 2].y, acc[i][j / 2 + 1].x, acc[i][j / 2 + 1].y);
        } else {
            const float2* q = acc[i / 2] + j;
            return i % 2 ? make_float4(q[0].y, q[1].y, q[2].y, q[3].y) : make_float4(q[0].x, q[1].x, q[2].x, q[3].x);
        }
    };
    if (T::G == 1 && split == 1) {
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            const int m = T::row(ty, i);
#pragma unroll
            for (int j = 0; j < T::TN; j += 4) {
                const int n = T::col(tx, j);
                if (m < m_rows && n < n_cols)
                    *reinterpret_cast<float4*>(dst + (size_t)m * ldc + n) = sums(i, j);
            }
        }
        return;
    }
    __syncthreads();
    // sums of the thread groups [G][BM][BN], then of the cluster's blocks, which share out the rows
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; j += 4)
            *reinterpret_cast<float4*>(sm + (group * BM_ + T::row(ty, i)) * BN + T::col(tx, j)) =
                sums(i, j);
    if (split > 1) ptx::cluster_sync();
    else __syncthreads();
    const uint32_t base = ptx::smem_addr(sm);
    for (int u = threadIdx.x; u < BM_ / split * (BN / 4); u += THREADS) {
        const int m = u / (BN / 4) * split + part, n = u % (BN / 4) * 4;
        if (m >= m_rows || n >= n_cols) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int g = 0; g < T::G; ++g) {
            const int o = (g * BM_ + m) * BN + n;
            float4 v[MAX_SPLIT];   // all in flight together
#pragma unroll
            for (int c = 0; c < MAX_SPLIT; ++c)
                if (c < split)
                    v[c] = split > 1 ? ptx::ld_cluster4(ptx::map_to_rank(base + o * 4, c))
                                     : *reinterpret_cast<const float4*>(sm + o);
#pragma unroll
            for (int c = 0; c < MAX_SPLIT; ++c)
                if (c < split) {
                    s.x += v[c].x;
                    s.y += v[c].y;
                    s.z += v[c].z;
                    s.w += v[c].w;
                }
        }
        *reinterpret_cast<float4*>(dst + (size_t)m * ldc + n) = s;
    }
    if (split > 1) ptx::cluster_sync();   // no block leaves while its sums are read
}

template <int OP, int BM>
cudaError_t launch(const GroupedArgs& a, cudaStream_t s) {
    using T = Tile<BM>;
    static PerDeviceOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(grouped_simt_kernel<OP, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int M = a.seg.M, E = a.seg.E, sms = a.num_sms > 0 ? a.num_sms : 148;
    long long tiles;   // at most
    float likely;      // tiles
    int red;
    if (OP == kGroupedWgrad) {
        tiles = (long long)E * ((a.N + BM - 1) / BM) * ((a.K + BN - 1) / BN);
        likely = (float)tiles;
        red = M / E;   // on average
    } else {
        const int ncol = OP == kGroupedMm ? a.N : a.K, cols = (ncol + BN - 1) / BN;
        red = OP == kGroupedMm ? a.K : a.N;
        const long long t = (long long)M / BM + E;
        tiles = (t < M ? t : M) * cols;
        // half a tile of every segment is empty; with counts M is a capacity: a dispatch rounds segments up to
        // 128 rows, half of them empty again
        const float live = a.seg.counts ? fmaxf((float)M - 64.f * E, 0.f) : (float)M;
        likely = (live / BM + 0.5f * E) * cols;
    }
    // Parts of the reduction: the time of a part (its slices, one to fill the pipe and half of one for each of
    // the sums to add) times the parts that an SM gets, the last wave half full.  (8192 rows of 4 experts, weight
    // gradients of 2048 x 1024, in 1, 2, 4, 8 parts: 791, 676, 725, 801 us; 645 rows of 8, 720 x 2072: 287, 152,
    // 125, 113.)  Eight slices a part at least.
    int split = 1;
    float best = 1e30f;
    for (int s = 1; s <= MAX_SPLIT && (s == 1 || red >= 8 * T::BK * s); s *= 2) {
        const float cost = (likely * s / sms + 0.5f) * ((float)red / (T::BK * s) + 1.f + 0.5f * s);
        if (cost < best) {
            best = cost;
            split = s;
        }
    }
    if (tiles * split > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = T::G == 1 && split == 1 ? T::OPERANDS : T::SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, grouped_simt_kernel<OP, BM>, static_cast<const float*>(a.rows),
                           static_cast<const float*>(a.other), static_cast<float*>(a.out), a.seg, a.N, a.K, split,
                           a.status);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Height of the tiles: by the rows of a segment on average (wgrad: by N).
template <int OP>
cudaError_t launch_op(const GroupedArgs& a, cudaStream_t s) {
    const int rows = OP == kGroupedWgrad ? a.N : (a.seg.M + a.seg.E - 1) / a.seg.E;
    if (rows <= 8) return launch<OP, 8>(a, s);
    // (with counts M is a capacity: a dispatch gives every expert 128 rows and room for 127 more)
    if (rows <= 40 || (OP != kGroupedWgrad && a.seg.counts && rows <= 144)) return launch<OP, 32>(a, s);
    // (8 experts of 4096 x 2048: tiles of 32, 64 and 128 rows take 137, 252 and 412 us where each expert has one;
    // segments differ in length, so a height is taken up to about its own)
    if (rows <= 64) return launch<OP, 64>(a, s);
    return launch<OP, 128>(a, s);
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t s) {
    switch (a.op) {
        case kGroupedMm: return launch_op<kGroupedMm>(a, s);
        case kGroupedDgrad: return launch_op<kGroupedDgrad>(a, s);
        default: return launch_op<kGroupedWgrad>(a, s);
    }
}

}  // namespace moe
