// Low-rank adapters beside a grouped product, first half: u_r = s_a A_{a,e} x_r for
// every row r of expert e's segment with adapter a = adapter[r] (-1: none, the row
// takes no part), as the bf16 operand of the second half y_r = W_e x_r + B_{a,e} u_r
// (grouped_tc.cu, grouped_few.cu): one bf16 value, or three that add up to the fp32
// one where the output is fp32.
//
// A cluster takes a window of 64 rows of a segment, finds the adapters that occur in
// it, and multiplies the window with 64 rank columns at a time (a column: one rank of
// one of these adapters), so that short adapters share a pass over x.  Each
// output keeps only the columns of its own row's adapter.  The CTAs of the cluster split
// the reduction and add their partial sums through distributed shared memory, in
// CTA order.  Operands go through a 4-stage cp.async ring (64 of the reduction a stage,
// 128-byte rows with their 16-byte chunks permuted by row) into ldmatrix and
// mma.m16n8k16.  What bounds it is reading x and the adapters once per window through L2
// (4096 rows, 12 adapters of rank 64, K = 4096: 137 MB in 36 us; windows of 128 rows and
// 128 columns read 83 MB but had 46 us, with half the loads in flight); the split is
// what gives small batches enough loads in flight (32 rows, 27 pairs of rank 16: 12 us).
//
// Further clusters of the same launch write down, for every column tile of the
// product, the adapters that occur among its rows, each once, in order of first
// occurrence.
#include "grouped.cuh"
#include "ptx_grouped.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int WIN = 64;                      // rows of a window
constexpr int COLS = 64;                     // rank columns of a pass
constexpr int KC = 64;                       // reduction per stage
constexpr int NST = 4;
constexpr int MAX_SPLIT = 8;                 // CTAs of a cluster, a power of two
constexpr int TILE_BYTES = WIN * KC * 2;     // 8 KiB, either operand
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int PITCH = COLS + 4;              // floats of a row of partial sums

struct ShrinkParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* A;
    const float* scale;
    LoraView v;
    Segments seg, listed;   // all segments; those that grouped_tc takes
    int K;
    int split;     // CTAs of a cluster
    int windows;   // clusters of the first kind along x (an upper bound of the windows)
    int* status;
};

struct ShrinkSmem {
    SegTable seg;
    alignas(16) int ids[kColumnTile];
    int list[kColumnTile];
    int warp_n[WARPS];
    int n;
};
constexpr int SMEM_BYTES = NST * STAGE_BYTES;   // also holds the partial sums of a pass
static_assert(WIN * PITCH * 4 <= SMEM_BYTES, "partial sums");

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The distinct ids of ids[0, n), in order of first occurrence, into list; sm->n of them (all threads).
__device__ __forceinline__ void distinct(ShrinkSmem* sm, int n) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int id = t < n ? sm->ids[t] : -1;
    bool first = id >= 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(sm->ids + j);
        first = first && !(j < t && v.x == id) && !(j + 1 < t && v.y == id) && !(j + 2 < t && v.z == id) &&
                !(j + 3 < t && v.w == id);
    }
    const uint32_t b = __ballot_sync(0xffffffffu, first);
    if (lane == 0) sm->warp_n[warp] = __popc(b);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sm->warp_n[w];
        total += sm->warp_n[w];
    }
    if (first) sm->list[before + __popc(b & ((1u << lane) - 1))] = id;
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

__global__ void __launch_bounds__(THREADS) lora_shrink_kernel(const ShrinkParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ ShrinkSmem sm;
    // the next kernel may start once everything before this one is done: it reads all but u without waiting
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / p.split, part = blockIdx.x % p.split;   // cluster, CTA of the cluster
    const bool lists = unit >= p.windows;
    if (lists && (part != 0 || blockIdx.y != 0)) return;
    if (warp == 0) build_segments(&sm.seg, lists ? p.listed : p.seg, lists ? kColumnTile : WIN, p.status);
    __syncthreads();
    const int tile = lists ? unit - p.windows : unit;
    if (tile >= sm.seg.total) return;   // the whole cluster
    const int e = segment_of(&sm.seg, p.seg.E, tile);
    const int rows = sm.seg.rows[e], at = tile - sm.seg.base[e];
    const ColumnTiles ct = column_tiles(rows);
    const int r0 = lists ? ct.start(at) : at * WIN, n = min(lists ? ct.rows(at) : WIN, rows - r0);
    const size_t row0 = (size_t)sm.seg.row0[e] + r0;
    if (tid < n) sm.ids[tid] = adapter_of(p, row0 + tid);
    __syncthreads();
    distinct(&sm, n);
    if (lists) {
        if (tid < sm.n) p.v.tile_list[(size_t)tile * kColumnTile + tid] = sm.list[tid];
        if (tid == 0) p.v.tile_count[tile] = sm.n;
        return;
    }

    const int R = p.v.R, R16 = p.v.R16, K = p.K;
    const int ncols = sm.n * R16;
    const int nk = (K + KC - 1) / KC, kb0 = (int)((long long)nk * part / p.split),
              kb1 = (int)((long long)nk * (part + 1) / p.split);
    const uint32_t ring0 = ptx::smem_addr(ring);
    // loads: thread tid fills chunk tid % 8 of rows tid / 8 and tid / 8 + 32 of either operand
    const int lrow = tid >> 3, lchunk = tid & 7;
    // products: warp w takes rows 16 (w / 2), columns 32 (w % 2)
    const int m0 = warp / 2 * 16, n0 = warp % 2 * 32;
    for (int c0 = blockIdx.y * COLS; c0 < ncols; c0 += gridDim.y * COLS) {
        const __nv_bfloat16* src[4];   // rows of x, then rank columns
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = lrow + 32 * j, c = c0 + r;
            src[j] = r < n ? p.x + (row0 + r) * K + lchunk * 8 : nullptr;
            const int q = c % R16;
            src[2 + j] = c < ncols && q < R
                             ? p.A + (((size_t)sm.list[c / R16] * p.seg.E + e) * R + q) * K + lchunk * 8
                             : nullptr;
        }
        auto load = [&](int kb) {
            const uint32_t stage = ring0 + (uint32_t)((kb - kb0) % NST) * STAGE_BYTES;
            const bool in = kb * KC + lchunk * 8 < K;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = lrow + 32 * (j & 1);
                const bool live = in && src[j];
                ptx::cp_async16(stage + (j >> 1) * TILE_BYTES + r * 128 + ((lchunk ^ (r & 7)) * 16),
                           live ? src[j] + (size_t)kb * KC : p.x, live);
            }
        };
        // (the tensor cores truncate when they add: 64 of the reduction in them, the rest with rounding)
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
        for (int s = 0; s < NST - 1; ++s) {
            if (kb0 + s < kb1) load(kb0 + s);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        for (int kb = kb0; kb < kb1; ++kb) {
            asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
            __syncthreads();
            if (kb + NST - 1 < kb1) load(kb + NST - 1);
            asm volatile("cp.async.commit_group;" ::: "memory");
            const uint32_t sx = ring0 + (uint32_t)((kb - kb0) % NST) * STAGE_BYTES, sa = sx + TILE_BYTES;
            float d[4][4] = {};
#pragma unroll
            for (int kk = 0; kk < KC / 16; ++kk) {
                uint32_t a[4], b[2][4];
                const int ar = m0 + (lane & 15), ac = 2 * kk + (lane >> 4);
                ldmatrix4(a, sx + ar * 128 + ((ac ^ (ar & 7)) * 16));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int br = n0 + 16 * j + (lane & 7) + (lane >> 4) * 8, bc = 2 * kk + (lane >> 3 & 1);
                    ldmatrix4(b[j], sa + br * 128 + ((bc ^ (br & 7)) * 16));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ptx::mma16816(d[i], a[0], a[1], a[2], a[3], b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += d[i][j];
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float* red = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                red[(m0 + (lane >> 2) + 8 * (j >> 1)) * PITCH + n0 + 8 * i + 2 * (lane & 3) + (j & 1)] = acc[i][j];
        ptx::cluster_sync();
        // CTA `part` finishes rows part, part + split, ...: its columns are those of the row's adapter
        for (int o = tid; o < WIN / p.split * (COLS / 4); o += THREADS) {
            const int r = o / (COLS / 4) * p.split + part, q = o % (COLS / 4) * 4, c = c0 + q;
            if (r >= n || c >= ncols) continue;
            const int a = sm.list[c / R16];   // four neighbours belong to one adapter
            if (sm.ids[r] != a) continue;
            const uint32_t at = ptx::smem_addr(red + r * PITCH + q);
            float4 v[MAX_SPLIT];
#pragma unroll
            for (int i = 0; i < MAX_SPLIT; ++i)
                if (i < p.split) v[i] = ptx::ld_cluster4(ptx::map_to_rank(at, i));
            float4 s = v[0];
#pragma unroll
            for (int i = 1; i < MAX_SPLIT; ++i)
                if (i < p.split) {
                    s.x += v[i].x;
                    s.y += v[i].y;
                    s.z += v[i].z;
                    s.w += v[i].w;
                }
            const int j = c % R16;
            const float f = p.scale[a];
            float y[4] = {j < R ? s.x * f : 0.f, j + 1 < R ? s.y * f : 0.f, j + 2 < R ? s.z * f : 0.f,
                          j + 3 < R ? s.w * f : 0.f};
            __nv_bfloat16* u = p.v.u + (row0 + r) * p.v.terms * R16 + j;
            for (int t = 0; t < p.v.terms; ++t) {
                const uint32_t lo = pack_bf16x2(y[0], y[1]), hi = pack_bf16x2(y[2], y[3]);
                *reinterpret_cast<uint2*>(u + t * R16) = make_uint2(lo, hi);
                // what the term leaves over (exact); nothing where it is not finite
                const float z[4] = {bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = isfinite(z[i]) ? y[i] - z[i] : 0.f;
            }
        }
        ptx::cluster_sync();   // the ring is free again, and no CTA exits while its sums are read
    }
}

}  // namespace

cudaError_t launch_lora_shrink(const GroupedArgs& a, cudaStream_t s) {
    ShrinkParams p{};
    p.x = static_cast<const __nv_bfloat16*>(a.rows);
    p.A = static_cast<const __nv_bfloat16*>(a.A);
    p.scale = a.scale;
    p.v = lora_view(a);
    p.seg = p.listed = a.seg;
    const Choice choice = grouped_choice(a);
    if (choice.few && choice.tc) p.listed.least = choice.limit + 1;
    p.K = a.K;
    p.status = a.status;
    const int M = a.seg.M, E = a.seg.E, sms = a.num_sms > 0 ? a.num_sms : 148;
    auto tiles = [&](int h) { return (int)((long long)M / h + E < M ? (long long)M / h + E : M); };
    p.windows = tiles(WIN);
    // split the reduction while the windows leave SMs idle and every part has at least four stages
    p.split = 1;
    while (p.split < MAX_SPLIT && p.windows * p.split < sms && (a.K + KC - 1) / KC >= 8 * p.split) p.split *= 2;
    // passes side by side: as many as a window can have, no more than run at once (three blocks to an SM)
    const long long most = ((long long)(a.L < WIN ? a.L : WIN) * p.v.R16 + COLS - 1) / COLS;
    const long long room = 3LL * sms / ((long long)p.windows * p.split) + 1;
    static PerDeviceOnce attr;
    cudaError_t e = attr.run([] {
        // (the carveout stays the default: with all of an SM's memory given to shared memory for this kernel, the
        // weight-streaming product beside it lost its L1 and took 231 us instead of 183)
        return cudaFuncSetAttribute(lora_shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.split;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((p.windows + tiles(kColumnTile)) * p.split), (unsigned)(most < room ? most : room));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
