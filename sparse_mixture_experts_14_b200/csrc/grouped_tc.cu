// Ragged grouped products on the tensor cores (bf16 operands, fp32 accumulation
// in tensor memory), sm_100a.  With segments of rows per expert e (grouped.cuh):
//     mm     y_r  = W_e x_r                      rows [M][K] -> [M][N]
//     dgrad  dx_r = W_e^T dy_r                   rows [M][N] -> [M][K]
//     wgrad  dW_e = sum_{r in e} dy_r x_r^T      -> [E][N][K]
//
// All three put the contiguous dimension of the output ("features": N, K, K) on
// the MMA's M side, so that the 32 lanes of an epilogue warp hold 32 neighbours
// in memory, and the output's rows ("columns" of the accumulator: tokens, tokens,
// dW's n) on its N side.  The N side is where segments are ragged, and N is an
// instruction field: a segment is cut into nearly equal tiles of up to 256 rows
// (column_tiles), which compute at most 31 rows in vain (a 256-row M side would round
// every segment up to 256).
//
//              M side (A)                     N side (B)                reduction
//     mm       W_e  [f][K]    K-major         x rows   K-major          K
//     dgrad    W_e  [N][f]    MN-major        dy rows  K-major          N
//     wgrad    x    [r][f]    MN-major        dy [r][c] MN-major        the segment's rows
// MN-major operands are read as they lie (64 x 64 boxes, 128-byte swizzle): nothing
// is transposed in memory.
//
// A pair of CTAs computes a 256 x (up to 256) tile with tcgen05.mma.cta_group::2,
// each CTA holding 128 features and half of the columns' operand.  Persistent, one
// CTA per SM: warp 0 TMA producer into a ring of 64-deep stages, warp 1 MMA issuer
// (in the pair's leader), 16 epilogue warps for the CTA's 128 features out of two
// alternating accumulators, a further warp for the ends of wgrad's segments.
//
// fp32 outputs: the tensor cores truncate when they add to the accumulator, which
// costs 1.8e-8 of the result per 16-deep step, all in one direction (1.6e-5 at a
// reduction of 14336, where a blocked fp32 sum has 3e-7).  So the accumulator takes
// 512 of the reduction at a time, and the epilogue adds these partial sums in
// registers with rounding, while the MMAs go on in the other accumulator.  bf16
// outputs, whose own rounding is 2^-8, take the whole reduction in one.
//
// Adapters (lora.cu computes u_r = s_a A_{a,e} x_r, bf16): B_{a,e} u_r is more of the
// same reduction.  For every adapter that occurs among a tile's rows, in slices of 16
// of its rank, the ring takes boxes of B_{a,e} (A side) and, written by two extra warps,
// the tile's rows of u with zeros in the rows of other adapters (B side): one K = 16
// MMA a slice, four slices a stage.  Boxes are 64, 32 or 16 ranks wide, the widest
// that divides the padded rank, with the swizzle of that width.  A zero does not
// hide an infinity or NaN in another request's adapter: it takes that feature of all of the
// tile's rows with it.  The epilogue marks such tiles, and behind the pipeline, where no
// bounded wait depends on it, the CTA computes those outputs again from their own terms.
//
// Outputs of few tiles: a cluster of up to 4 pairs splits a tile's reduction (SPLIT).
// Every pair keeps its fp32 sums in shared memory, and the CTAs add them through
// distributed shared memory, in pair order, each storing its part of the columns.
//
// wgrad: the last 64-row block of a segment also holds rows of the next one, which
// must not count, whatever they hold (NaN times zero is NaN).  The MMA stops at the
// 16-row slice of the segment's last row, and an extra warp in each CTA clears
// the rest of that slice in shared memory, in both operands, before the MMA may
// read it.
//
// Measured (8192 rows of 8 experts, 14336 x 4096, loops of 2 s at the 1000 W cap; us, and the SM clock in GHz that the
// cap leaves): mm 765 (1.29), 1257 TFLOP/s; dgrad 794 (1.35); wgrad 814 (1.35); to fp32, on narrow tiles, 920 (1.44),
// 887 (1.40) and 1131 (1.52).  cuBLAS on one dense matrix of the size: 731 (1.47).  Wide tiles do the most per clock (0.80
// of the tensor cores' rate in mm) and run at the lowest one: power binds them.  Narrow ones wait for operands on their way
// through shared memory (0.67), wgrad's to fp32 also for its epilogue (0.46: 16 blocks of the reduction to a tile of
// 256 KB; the same tiles to bf16 992 us at the same clock).
#include <cuda.h>

#include "grouped.cuh"
#include "ptx_grouped.cuh"
#include "tma_map.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                    // features of one MMA per CTA (256 per pair)
constexpr int BN = 256;                    // columns of a tile at most
constexpr int BK = 64;                     // reduction per stage
constexpr int A_BYTES = BM * BK * 2;       // 16 KiB
constexpr int B_BYTES = BN / 2 * BK * 2;   // 16 KiB
constexpr int BOX = 64;                    // MN-major operands: 64-wide boxes
constexpr uint32_t MN_LBO = BOX * BK * 2;
constexpr uint32_t MN_SBO = 1024;
constexpr int TMEM_COLS = 2 * BN;
constexpr int CHUNK = 512 / BK;            // blocks per accumulator, fp32 outputs

constexpr int SLICE = 16;                   // rank slice of one adapter MMA
constexpr int SLICES = 4;                   // of a stage
constexpr int SLICE_BYTES = BM * SLICE * 2; // 4 KiB, either side (a box w wide is w / 16 of them)

struct Maps {
    CUtensorMap a;
    CUtensorMap b[4];   // boxes of 16, 32, 64 and 128 rows (mm, dgrad); wgrad: b[0] only
    CUtensorMap l;      // adapters: B_{a,e}, boxes of lora.box x 128 features
};

struct Params {
    Segments seg;
    int F;            // features: the output's contiguous dimension
    int C;            // wgrad: columns (N)
    int red;          // mm, dgrad: length of the reduction
    int f_fast;       // wgrad: feature blocks fastest, else column blocks
    int split;        // pairs of a cluster
    int out16;        // split: type of the output
    void* out;
    int* status;
    long long wait_ns;
    // adapters
    LoraView lora;
    const __nv_bfloat16* x;
    const __nv_bfloat16* W;
};

constexpr int MAX_STAGES = 6;
constexpr int MAX_SPLIT = 4;                // pairs of a cluster
constexpr int ODD_WORDS = 8;                // tiles 256 apart share a bit: a tile may be looked through in vain

struct Ctrl {
    uint64_t full[MAX_STAGES];     // leader: both CTAs' bytes of a stage landed
    uint64_t empty[MAX_STAGES];    // each CTA: the MMAs that read a stage are done
    uint64_t land[MAX_STAGES];     // wgrad: this CTA's bytes of a segment's last block landed; adapters: stage free
    uint64_t ready[MAX_STAGES];    // leader: both CTAs prepared the stage by hand
    uint64_t tfull[2];      // each CTA: accumulator b holds a finished tile
    uint64_t tempty[2];     // leader: both CTAs' epilogues released accumulator b
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int total;
    uint32_t odd[ODD_WORDS];   // adapters: this CTA's tiles with features of which no output is finite, in turn
    SegTable seg;
};

template <int OP, bool OUT16, int W, bool LORA, bool SPLIT>
struct Cfg {
    static_assert(!SPLIT || (!OUT16 && W == 1), "a split tile is summed in fp32");
    static constexpr bool WGRAD = OP == kGroupedWgrad;
    static constexpr bool A_MN = OP != kGroupedMm;
    static constexpr bool B_MN = WGRAD;
    static constexpr int AUX_WARPS = WGRAD ? 1 : LORA ? 2 : 0;
    static constexpr int EPI_WARPS = 16;
    static constexpr int COLS = W == 2 ? 128 : 64;   // columns of an epilogue warp
    static constexpr int THREADS = 32 * (2 + EPI_WARPS + AUX_WARPS);
    static constexpr int NST = W == 1 ? 6 : 4;
    static constexpr int STAGE = W * A_BYTES + B_BYTES;
    static constexpr int PAIR_F = W * 2 * BM;   // features of a pair's tile
    static constexpr int ACCS = W == 1 ? 2 : 1; // accumulators in the 512 columns
    static constexpr int SMEM = NST * STAGE + (int)sizeof(Ctrl) + 1024;
};

// One tile: expert, first feature of the pair, first column (row of the row buffers, or n of dW),
// columns of the MMA and those that count, 64-deep blocks.
struct Tile {
    int e, f0, c0, nn, valid, nkb, rows, row0, col_tile;
    bool alone;   // the only column tile of its expert: nobody else reads its weights
};

template <bool WGRAD, int PAIR_F>
__device__ __forceinline__ Tile decode(const Ctrl* c, const Params& p, int tile) {
    Tile t;
    const int nf = (p.F + PAIR_F - 1) / PAIR_F;
    if (WGRAD) {
        const int nc = (p.C + BN - 1) / BN;
        t.e = tile / (nf * nc);
        const int local = tile - t.e * nf * nc;
        const int fi = p.f_fast ? local % nf : local / nc;
        t.f0 = fi * PAIR_F;
        t.c0 = (p.f_fast ? local / nf : local % nc) * BN;
        t.rows = c->seg.rows[t.e];
        t.row0 = c->seg.row0[t.e];
        t.valid = min(BN, p.C - t.c0);
        t.nn = (t.valid + 31) / 32 * 32;
        t.nkb = (t.rows + BK - 1) / BK;
        t.col_tile = 0;
        t.alone = false;
    } else {
        // token tiles fastest: the pairs at work share blocks of the weights
        const int tok = tile / nf;   // any tile of the expert's group
        t.e = segment_of(&c->seg, p.seg.E, tok);
        const int tt = c->seg.base[t.e + 1] - c->seg.base[t.e];
        const int local = tile - c->seg.base[t.e] * nf;
        const int fi = local / tt;
        t.rows = c->seg.rows[t.e];
        const ColumnTiles ct = column_tiles(t.rows);
        const int i = local - fi * tt, r = ct.start(i);
        t.f0 = fi * PAIR_F;
        t.row0 = c->seg.row0[t.e];
        t.c0 = t.row0 + r;
        t.nn = ct.rows(i);
        t.valid = min(t.nn, t.rows - r);
        t.nkb = (p.red + BK - 1) / BK;
        t.col_tile = c->seg.base[t.e] + i;
        t.alone = tt == 1;
    }
    return t;
}

// Pairs of bf16 values: the smaller magnitudes; NaN only where both are.
__device__ __forceinline__ uint32_t min_magnitude(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// Index of the row box that holds n rows (n a multiple of 16, at most 128).
__device__ __forceinline__ int box_of(int n) { return n <= 16 ? 0 : n <= 32 ? 1 : n <= 64 ? 2 : 3; }

// Adapter slices of a tile: (adapters among its rows) x (slices of u's row).
__device__ __forceinline__ int tile_slices(const LoraView& l, int col_tile) {
    return l.tile_count[col_tile] * l.per;
}

// What the TMA's swizzle of rows of 2 box bytes does to row r: its 16-byte chunk c is kept at c ^ swizzle.
__device__ __forceinline__ int swizzle(int r, int box) { return box == 64 ? r & 7 : box == 32 ? r >> 1 & 3 : r >> 2 & 1; }

__device__ __forceinline__ bool not_finite(uint32_t bits) { return (bits & 0x7f800000u) == 0x7f800000u; }

// Outputs of a tile with adapters that are not finite, again from their own terms alone: x_r W_e^T[f] and, with an
// adapter, u_r B_{a,e}^T[f].  One warp, the 16 features from f0 on and n <= 32 rows, row0 and every step-th behind.
// What another request's B does to a feature (zero times an infinity or NaN) it does to all of the tile's rows, so
// a block in which every feature has a finite output is left as it is.  Products as in grouped_few.cu, operands
// straight from global memory, 32 of the reduction in the tensor cores at a time and the rest with rounding.  (All
// outputs hit: 1500 rows of one expert, 2048 x 2048, 43 -> 314 us; 4096 rows of 8, 14336 x 4096, 0.46 -> 5.3 ms, bound by
// L2.  One lane an output took 32 ms for the first, inside the pipeline, whose waits are bounded.)
__device__ __noinline__ void repair(const Params& p, int e, size_t row0, int n, int step, int f0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int F = p.F, K = p.red;
    // this lane's outputs: features f0 + 8 j + g, rows 8 t + 2 q + i
    uint32_t bad = 0;   // bit 8 j + 2 t + i
    bool all[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int f = f0 + 8 * j + g;
        all[j] = f < F;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int r = 8 * (c >> 1) + 2 * q + (c & 1);
            if (f >= F || r >= n) continue;
            const size_t at = (row0 + (size_t)r * step) * F + f;
            const uint32_t bits = p.out16 ? (uint32_t)static_cast<const uint16_t*>(p.out)[at] << 16
                                          : static_cast<const uint32_t*>(p.out)[at];
            if (not_finite(bits)) bad |= 1u << (8 * j + c);
            else all[j] = false;
        }
        // (the lanes of a feature: four neighbours)
        const uint32_t b = __ballot_sync(0xffffffffu, all[j]);
        all[j] = (b >> (4 * g) & 15u) == 15u;
    }
    if (!__any_sync(0xffffffffu, all[0] || all[1])) return;

    const uint4 zero = make_uint4(0, 0, 0, 0);
    const __nv_bfloat16* w[2];
    const __nv_bfloat16* x[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int f = f0 + 8 * j + g;
        w[j] = p.W + ((size_t)e * F + (f < F ? f : f0)) * K + 8 * q;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int r = 8 * t + g;
        x[t] = p.x + (row0 + (size_t)(r < n ? r : 0) * step) * K + 8 * q;
    }
    float acc[4][4] = {};
#pragma unroll 1
    for (int k0 = 0; k0 < K; k0 += 32) {
        const bool in = k0 + 8 * q < K;
        uint4 a[2], b[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) a[j] = in ? __ldg(reinterpret_cast<const uint4*>(w[j] + k0)) : zero;
#pragma unroll
        for (int t = 0; t < 4; ++t) b[t] = in ? __ldg(reinterpret_cast<const uint4*>(x[t] + k0)) : zero;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float d[4] = {};
            ptx::mma16816(d, a[0].x, a[1].x, a[0].y, a[1].y, b[t].x, b[t].y);
            ptx::mma16816(d, a[0].z, a[1].z, a[0].w, a[1].w, b[t].z, b[t].w);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[t][c] += d[c];
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (!(bad >> (8 * j + c) & 1)) continue;
            const int f = f0 + 8 * j + g;
            const size_t r = row0 + (size_t)(8 * (c >> 1) + 2 * q + (c & 1)) * step;
            float s = acc[c >> 1][2 * j + (c & 1)];
            const int id = p.lora.adapter[r];
            if (id >= 0 && id < p.lora.L) {
                const size_t ae = (size_t)id * p.seg.E + e;
                s += p.lora.terms == 1 ? adapter_term<1>(p.lora, ae, F, r, f) : adapter_term<3>(p.lora, ae, F, r, f);
            }
            if (p.out16) static_cast<__nv_bfloat16*>(p.out)[r * F + f] = __float2bfloat16_rn(s);
            else static_cast<float*>(p.out)[r * F + f] = s;
        }
}

template <int OP, bool OUT16, int W, bool LORA, bool SPLIT>
__global__ void __launch_bounds__(Cfg<OP, OUT16, W, LORA, SPLIT>::THREADS, 1)
    grouped_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using CF = Cfg<OP, OUT16, W, LORA, SPLIT>;
    constexpr bool WGRAD = CF::WGRAD;
    constexpr int NST = CF::NST, STAGE = CF::STAGE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + NST * STAGE);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // rank of the CTA in its pair, rank of the pair's leader in the cluster, pair of the cluster
    const uint32_t crank = ptx::cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
    const int part = SPLIT ? (int)(crank >> 1) : 0, parts = SPLIT ? p.split : 1;
    const uint16_t pair_mask = (uint16_t)(0x3u << lead);
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / (2 * parts);
    const int nclusters = gridDim.x / (2 * parts);   // (split: as many as there are tiles)

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(&ctrl->full[s], 1);
            ptx::mbar_init(&ctrl->empty[s], 1);
            ptx::mbar_init(&ctrl->land[s], 1);
            ptx::mbar_init(&ctrl->ready[s], 2 * (CF::AUX_WARPS > 0 ? CF::AUX_WARPS : 1));
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&ctrl->tfull[b], 1);
            ptx::mbar_init(&ctrl->tempty[b], 2 * CF::EPI_WARPS);
        }
        ptx::mbar_init(&ctrl->drain, 1);
        ctrl->abort = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&maps.a);
    }
    if (LORA && threadIdx.x >= 32 && threadIdx.x < 32 + ODD_WORDS) ctrl->odd[threadIdx.x - 32] = 0;
    if (warp == 1) {
        ptx::tmem_alloc_pair(&ctrl->tmem_base, TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    pdl_wait();
    if (warp == 0) {
        build_segments(&ctrl->seg, p.seg, BN, crank == 0 && cluster == 0 ? p.status : nullptr);
        __syncwarp();
        if (lane == 0) {
            const int nf = (p.F + CF::PAIR_F - 1) / CF::PAIR_F;
            ctrl->total = !ctrl->seg.good ? 0 : WGRAD ? p.seg.E * nf * ((p.C + BN - 1) / BN) : ctrl->seg.total * nf;
        }
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();
    ptx::tc_fence_after_sync();

    const uint32_t tmem_base = ctrl->tmem_base;
    const int total = ctrl->total;
    // this pair's share of a tile: blocks [kb0, kb1) of the reduction, slices [s0, s1) of the adapters
    struct Share {
        int kb0, kb1, s0, s1;
    };
    auto share = [&](const Tile& t) {
        const int slices = LORA ? tile_slices(p.lora, t.col_tile) : 0;
        if (!SPLIT) return Share{0, t.nkb, 0, slices};
        // (a block of adapter slices, which warps prepare by hand, takes the time of about two others)
        const long long all = t.nkb + 2 * ((slices + SLICES - 1) / SLICES);
        const int b0 = (int)(all * part / parts), b1 = (int)(all * (part + 1) / parts);
        return Share{min(b0, t.nkb), min(b1, t.nkb), min((max(b0 - t.nkb, 0) + 1) / 2 * SLICES, slices),
                     min((max(b1 - t.nkb, 0) + 1) / 2 * SLICES, slices)};
    };
    const ptx::WaitCtl wc{&ctrl->abort, p.status, (uint64_t)p.wait_ns};
    auto mark_odd = [&](int tile) {   // one lane
        const int i = SPLIT ? 0 : (tile - cluster) / nclusters;
        atomicOr(&ctrl->odd[i / 32 % ODD_WORDS], 1u << i % 32);
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        if (lane == 0) {
            const uint64_t pol = ptx::policy_evict_normal();
            // Weights that one tile alone reads leave L2 first (256 rows of 8 experts, 14336 x 4096, 199 -> 193 us);
            // shared ones must not (8192 rows: 809 -> 914 us), the tiles read them at different times.
            const uint64_t pol_once = ptx::policy_evict_first();
            int stage = 0;
            uint32_t phase = 0;
            uint32_t armed = 0, armed_phase = 0, tail = 0, tail_phase = 0;   // bits per stage
            bool aborted = false;
            for (int tile = cluster; tile < total && !aborted; tile += nclusters) {
                const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
                const int fa = t.f0 + (int)rank * BM;
                const int half = t.nn / 2;
                const int cb = t.c0 + (int)rank * half;
                const int box = WGRAD ? 0 : box_of(half);
                const int bboxes = WGRAD ? (half + BOX - 1) / BOX : 1;
                // (asked for now, needed behind the last of the other blocks)
                const int32_t* list = LORA ? p.lora.tile_list + (size_t)t.col_tile * BN : nullptr;
                const int per = LORA ? p.lora.per : 1;
                const Share sh = share(t);
                int z[SLICES];
                if (LORA) {
#pragma unroll
                    for (int i = 0; i < SLICES; ++i) z[i] = list[(sh.s0 + i) / per];
                }
                const uint64_t polw = t.alone ? pol_once : pol;
                const uint32_t bytes = W * A_BYTES + (WGRAD ? bboxes * (int)MN_LBO : (16 << box) * BK * 2);
                for (int kb = sh.kb0; kb < sh.kb1; ++kb) {
                    if (!ptx::mbar_wait(&ctrl->empty[stage], phase ^ 1u, wc)) {
                        aborted = true;
                        break;
                    }
                    uint8_t* sa = smem + stage * STAGE;
                    uint8_t* sb = sa + W * A_BYTES;
                    const int k = kb * BK;
                    if (WGRAD && kb == t.nkb - 1 && (t.rows & 15) != 0) {
                        // the segment's last block: this CTA's own barrier, the clearing warp goes on from there
                        ptx::mbar_arrive_expect_tx(&ctrl->land[stage], bytes);
                        if (leader) ptx::mbar_arrive(&ctrl->full[stage]);
                        uint64_t* bar = &ctrl->land[stage];
#pragma unroll
                        for (int h = 0; h < 2 * W; ++h)
                            ptx::tma_load_2d(sa + h * MN_LBO, &maps.a, bar, fa + (h >> 1) * 2 * BM + (h & 1) * BOX,
                                             t.row0 + k, pol);
                        for (int h = 0; h < bboxes; ++h)
                            ptx::tma_load_2d(sb + h * MN_LBO, &maps.b[0], bar, cb + h * BOX, t.row0 + k, pol);
                        tail |= 1u << stage;
                    } else {
                        const uint32_t bar = ptx::map_to_rank(ptx::smem_addr(&ctrl->full[stage]), lead);
                        if (leader) ptx::mbar_arrive_expect_tx(&ctrl->full[stage], 2 * bytes);
                        if (WGRAD) {
#pragma unroll
                            for (int h = 0; h < 2 * W; ++h)
                                ptx::tma_load_2d_pair(sa + h * MN_LBO, &maps.a, bar,
                                                      fa + (h >> 1) * 2 * BM + (h & 1) * BOX, t.row0 + k, pol);
                            for (int h = 0; h < bboxes; ++h)
                                ptx::tma_load_2d_pair(sb + h * MN_LBO, &maps.b[0], bar, cb + h * BOX, t.row0 + k, pol);
                        } else {
                            if (CF::A_MN) {
#pragma unroll
                                for (int h = 0; h < 2 * W; ++h)
                                    ptx::tma_load_3d_pair(sa + h * MN_LBO, &maps.a, bar,
                                                          fa + (h >> 1) * 2 * BM + (h & 1) * BOX, k, t.e,
                                                          polw);
                            } else {
#pragma unroll
                                for (int h = 0; h < W; ++h)
                                    ptx::tma_load_3d_pair(sa + h * A_BYTES, &maps.a, bar, k, fa + h * 2 * BM, t.e, polw);
                            }
                            ptx::tma_load_2d_pair(sb, &maps.b[box], bar, k, cb, pol);
                        }
                        tail &= ~(1u << stage);
                    }
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    if (tail >> stage & 1) tail_phase ^= 1u << stage;   // uses of land[stage] so far, mod 2
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (LORA && !aborted) {
                    for (int s0 = sh.s0; s0 < sh.s1; s0 += SLICES) {
                        const int n = min(SLICES, sh.s1 - s0);
                        if (!ptx::mbar_wait(&ctrl->empty[stage], phase ^ 1u, wc)) {
                            aborted = true;
                            break;
                        }
                        ptx::mbar_arrive(&ctrl->land[stage]);   // the stage is free: u's warps may write it
                        const uint32_t bar = ptx::map_to_rank(ptx::smem_addr(&ctrl->full[stage]), lead);
                        if (leader) ptx::mbar_arrive_expect_tx(&ctrl->full[stage], 2 * n * W * SLICE_BYTES);
                        const int step = p.lora.box / SLICE, ranks = p.lora.R16 / SLICE;
#pragma unroll
                        for (int i = 0; i < SLICES; ++i) {
                            if (i >= n) break;
                            if (i % step != 0) continue;
                            const int k = (s0 + i) % per % ranks * SLICE;
#pragma unroll
                            for (int h = 0; h < W; ++h)
                                ptx::tma_load_3d_pair(smem + stage * STAGE + h * A_BYTES + i * SLICE_BYTES, &maps.l, bar,
                                                      k, fa + h * 2 * BM, z[i] * p.seg.E + t.e, pol);
                        }
#pragma unroll
                        for (int i = 0; i < SLICES; ++i) z[i] = list[min(s0 + SLICES + i, sh.s1 - 1) / per];
                        armed |= 1u << stage;
                        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                        if (++stage == NST) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (aborted || ctrl->abort) {
                // let copies still in flight land before shared memory is released
                for (int s = 0; s < NST; ++s) {
                    if (!(armed >> s & 1)) continue;
                    if (tail >> s & 1)
                        ptx::mbar_wait_drain(&ctrl->land[s], (tail_phase >> s & 1) ^ 1u, 100000000ull);
                    else if (leader)
                        ptx::mbar_wait_drain(&ctrl->full[s], armed_phase >> s & 1, 100000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer (leader)
        if (lane == 0 && leader) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            uint32_t hand_phase = 0;   // per stage: phase of ready[]
            bool issued = false, aborted = false;
            // Descriptors of the ring's first stage; others differ in the address field alone (16-byte units).
            // One thread issues every MMA: what it computes per MMA is kept to an addition.
            const uint32_t ring = ptx::smem_addr(smem);
            const uint64_t da0 = CF::A_MN ? ptx::desc_mnmajor_sw128(ring, MN_LBO, MN_SBO) : ptx::desc_kmajor_sw128(ring);
            const uint64_t db0 = CF::B_MN ? ptx::desc_mnmajor_sw128(ring + W * A_BYTES, MN_LBO, MN_SBO)
                                          : ptx::desc_kmajor_sw128(ring + W * A_BYTES);
            constexpr uint32_t A_STEP = (CF::A_MN ? 2048 : 32) / 16, B_STEP = (CF::B_MN ? 2048 : 32) / 16;
            // wait for block kb's accumulator (where it opens one) and operands
            uint32_t d_tmem = 0;
            auto open = [&](bool first) {
                if (first) {
                    if (!ptx::mbar_wait(&ctrl->tempty[acc], acc_phase ^ 1u, wc)) return false;
                    d_tmem = tmem_base + (uint32_t)(acc * BN);
                }
                return ptx::mbar_wait(&ctrl->full[stage], phase, wc);
            };
            auto by_hand = [&]() {   // the stage was also written by this pair's warps
                const bool ok = ptx::mbar_wait(&ctrl->ready[stage], hand_phase >> stage & 1, wc);
                hand_phase ^= 1u << stage;
                return ok;
            };
            auto close = [&](bool last) {
                ptx::tc_commit_pair_multicast(&ctrl->empty[stage], pair_mask);
                issued = true;
                if (++stage == NST) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (last) {
                    ptx::tc_commit_pair_multicast(&ctrl->tfull[acc], pair_mask);
                    if (++acc == CF::ACCS) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            };
            for (int tile = cluster; tile < total && !aborted; tile += nclusters) {
                const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
                const uint32_t idesc = ptx::idesc_bf16_f32(2 * BM, t.nn, CF::A_MN, CF::B_MN);
                const Share sh = share(t);
                const int kb0 = sh.kb0, nkb = sh.kb1 - kb0, aslices = sh.s1 - sh.s0;
                for (int i = 0; i < nkb; ++i) {
                    const int kb = kb0 + i;
                    const bool first = OUT16 ? i == 0 : i % CHUNK == 0;   // of an accumulator
                    bool ok = open(first);
                    int slices = BK / 16;
                    if (WGRAD && kb == t.nkb - 1) {
                        slices = (t.rows - kb * BK + 15) / 16;
                        if (ok && (t.rows & 15) != 0) ok = by_hand();
                    }
                    if (!ok) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const uint64_t da = da0 + (uint32_t)stage * (STAGE / 16), db = db0 + (uint32_t)stage * (STAGE / 16);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        if (WGRAD && kk >= slices) break;
#pragma unroll
                        for (int h = 0; h < W; ++h)
                            ptx::tc_mma_bf16_pair(d_tmem + h * BN, da + h * (A_BYTES / 16) + kk * A_STEP, db + kk * B_STEP,
                                                  idesc, kk > 0 || !first);
                    }
                    close((!OUT16 && i % CHUNK == CHUNK - 1) || (i == nkb - 1 && (!LORA || aslices == 0)));
                }
                if (!LORA || aborted) continue;
                const int box = p.lora.box, step = box / SLICE;
                const uint64_t la0 = ptx::desc_kmajor(ring, box * 2), lb0 = ptx::desc_kmajor(ring + W * A_BYTES, box * 2);
                int kb = nkb;
                for (int s0 = 0; s0 < aslices; s0 += SLICES, ++kb) {
                    const bool first = !OUT16 && kb % CHUNK == 0;
                    if (!open(first) || !by_hand()) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const int n = min(SLICES, aslices - s0);
                    const uint64_t la = la0 + (uint32_t)stage * (STAGE / 16), lb = lb0 + (uint32_t)stage * (STAGE / 16);
                    for (int i = 0; i < n; ++i) {
                        // box i / step, 32 bytes into its rows for every slice before this one
                        const uint32_t at = (uint32_t)(i / step * step * SLICE_BYTES + i % step * 32) / 16;
#pragma unroll
                        for (int h = 0; h < W; ++h)
                            ptx::tc_mma_bf16_pair(d_tmem + h * BN, la + h * (A_BYTES / 16) + at, lb + at, idesc,
                                                  i > 0 || !first);
                    }
                    close((!OUT16 && kb % CHUNK == CHUNK - 1) || s0 + SLICES >= aslices);
                }
            }
            if ((aborted || ctrl->abort) && issued) {
                ptx::tc_commit_pair(&ctrl->drain);
                ptx::mbar_wait_drain(&ctrl->drain, 0, 100000000ull);
            }
        }
    } else if (warp < 2 + CF::EPI_WARPS) {
        // ---------------------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3;   // TMEM lane quarter this warp may access
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int tile = cluster; tile < total && ok; tile += nclusters) {
            // groups of four warps: block of features, then part of the columns
            constexpr int PARTS = BN / CF::COLS;
            const int blk = (warp - 2) / 4 / PARTS, c0 = (warp - 2) / 4 % PARTS * CF::COLS;
            const Tile t0 = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
            const int ncol = min(CF::COLS, t0.nn - c0);   // a multiple of 32, or none (<= 0)
            if (WGRAD && !SPLIT && t0.nkb == 0) {
                // a segment without rows: nothing was accumulated, the gradient is zero
                const int f = t0.f0 + blk * 2 * BM + (int)rank * BM + q * 32 + lane;
                const size_t row0 = (size_t)t0.e * p.C + t0.c0 + c0;
                for (int i = 0; f < p.F && i < min(ncol, t0.valid - c0); ++i) {
                    if (OUT16) static_cast<__nv_bfloat16*>(p.out)[(row0 + i) * p.F + f] = __float2bfloat16_rn(0.f);
                    else static_cast<float*>(p.out)[(row0 + i) * p.F + f] = 0.f;
                }
                continue;
            }
            if (OUT16) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(&ctrl->tfull[acc], acc_phase, wc));
                if (!ok) break;
                ptx::tc_fence_after_sync();
                // The tile goes to registers first, rounded and packed by column pairs, so that the next
                // one's MMAs do not wait for the stores.
                uint32_t v[CF::COLS / 2];
                const uint32_t taddr = tmem_base + (uint32_t)((acc + blk) * BN + c0) + ((uint32_t)(q * 32) << 16);
#pragma unroll
                for (int c = 0; c < CF::COLS; c += 16) {
                    if (c >= ncol) break;
                    uint32_t r[16];
                    ptx::tmem_ld_32x32b_x16(taddr + c, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        v[(c + i) / 2] = pack_bf16x2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                }
                // the accumulator is free once every lane's tcgen05.ld has completed
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(ptx::smem_addr(&ctrl->tempty[acc]), lead));
                if (++acc == CF::ACCS) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
                // where it goes is worked out only now: the registers were needed
                asm volatile("" : "+r"(tile));
                const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
                const int aslices = LORA ? tile_slices(p.lora, t.col_tile) : 0;
                const size_t row0 = (WGRAD ? (size_t)t.e * p.C : (size_t)0) + t.c0 + c0;
                if (LORA && aslices > 0 && ncol > 0) {
                    // the smallest magnitude of the lane's feature, NaN aside: infinite (or NaN) if none is finite
                    uint32_t least = 0x7f807f80u;
#pragma unroll
                    for (int i = 0; i < CF::COLS; i += 2)
                        if (i < ncol) least = min_magnitude(least, v[i / 2]);
                    const bool odd = not_finite(least << 16) && not_finite(least);
                    if (__any_sync(0xffffffffu, odd) && lane == 0) mark_odd(tile);
                }
                // Neighbouring lanes swap halves: of columns i and i + 1 the even lane stores features f, f + 1 of
                // the first, the odd one f - 1, f of the second.  F is a multiple of 8: pairs are whole.
                const int hi = lane & 1;
                const int fp = t.f0 + blk * 2 * BM + (int)rank * BM + q * 32 + (lane & ~1);
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (row0 + hi) * p.F + fp;
                const uint32_t sel = hi ? 0x3276u : 0x5410u;
                const int cols = (fp < p.F ? t.valid - c0 : 0) - hi;
#pragma unroll
                for (int c = 0; c < CF::COLS; c += 16) {
                    if (c >= ncol) break;
#pragma unroll
                    for (int i = c; i < c + 16; i += 2) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, v[i / 2], 1);
                        if (i < cols)
                            *reinterpret_cast<uint32_t*>(out + (size_t)(i - c) * p.F) = __byte_perm(v[i / 2], got, sel);
                    }
                    out += 16 * (size_t)p.F;
                    asm volatile("" : "+l"(out));   // one pointer, not one per column, in registers
                }
            } else {
                float sum[CF::COLS];
#pragma unroll
                for (int i = 0; i < CF::COLS; ++i) sum[i] = 0.f;
                const Share sh = share(t0);
                const int aslices = sh.s1 - sh.s0;
                const int nblk = sh.kb1 - sh.kb0 + (aslices + SLICES - 1) / SLICES;
                for (int kb = 0; kb < nblk && ok; kb += CHUNK) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&ctrl->tfull[acc], acc_phase, wc));
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint32_t taddr = tmem_base + (uint32_t)(acc * BN + c0) + ((uint32_t)(q * 32) << 16);
#pragma unroll
                    for (int c = 0; c < CF::COLS; c += 16) {
                        if (c >= ncol) break;
                        uint32_t r[16];
                        ptx::tmem_ld_32x32b_x16(taddr + c, r);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(r[i]);
                    }
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(ptx::smem_addr(&ctrl->tempty[acc]), lead));
                    if (++acc == CF::ACCS) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (SPLIT) {
                    // one tile per cluster: the ring is idle, every copy and MMA of this pair is done
                    float* mine = reinterpret_cast<float*>(smem) + c0 * BM + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < CF::COLS; ++i)
                        if (i < ncol) mine[i * BM] = sum[i];
                    continue;
                }
                asm volatile("" : "+r"(tile));
                const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
                const int f = t.f0 + blk * 2 * BM + (int)rank * BM + q * 32 + lane;
                const size_t row0 = (WGRAD ? (size_t)t.e * p.C : (size_t)0) + t.c0 + c0;
                float* out = static_cast<float*>(p.out) + row0 * p.F + f;
                const int valid = f < p.F ? t.valid - c0 : 0;
#pragma unroll
                for (int c = 0; c < CF::COLS; c += 16) {
                    if (c >= ncol) break;
#pragma unroll
                    for (int i = c; i < c + 16; ++i)
                        if (i < valid) out[(size_t)(i - c) * p.F] = sum[i];
                    out += 16 * (size_t)p.F;
                    asm volatile("" : "+l"(out));
                }
                if (LORA && aslices > 0 && ncol > 0) {
                    float least = __uint_as_float(0x7f800000u);
#pragma unroll
                    for (int i = 0; i < CF::COLS; ++i)
                        if (i < ncol) least = fminf(least, fabsf(sum[i]));
                    if (__any_sync(0xffffffffu, not_finite(__float_as_uint(least))) && lane == 0) mark_odd(tile);
                }
            }
        }
    } else if (WGRAD) {
        // ---------------------------------------------------------------- ends of segments (both CTAs)
        unsigned block = 0;        // blocks through the ring so far
        uint32_t land_phase = 0;   // per stage
        for (int tile = cluster; tile < total; tile += nclusters) {
            const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
            const Share sh = share(t);
            block += sh.kb1 - sh.kb0;
            if ((t.rows & 15) == 0 || sh.kb1 != t.nkb || sh.kb0 == sh.kb1) continue;
            const int stage = (block - 1) % NST;
            bool ok = ptx::mbar_wait(&ctrl->land[stage], land_phase >> stage & 1, wc);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            land_phase ^= 1u << stage;
            // rows of the block that lie in its last 16-row slice behind the segment: 128 bytes a row and box
            const int r0 = (t.rows - 1) % BK + 1, r1 = (r0 + 15) / 16 * 16;
            uint8_t* base = smem + stage * STAGE;
            constexpr int BOXES = 2 * W + 2;
            for (int i = lane; i < (r1 - r0) * BOXES * 8; i += 32) {
                const int v = i & 7, box = (i >> 3) % BOXES, r = r0 + (i >> 3) / BOXES;
                *reinterpret_cast<uint4*>(base + box * (int)MN_LBO + r * 128 + v * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_operands(ptx::map_to_rank(ptx::smem_addr(&ctrl->ready[stage]), lead));
        }
    } else if (LORA) {
        // ---------------------------------------------------------------- rows of u (both CTAs)
        // They follow the producer's word (land), not the ring's own barriers: a parity can neither tell a
        // phase from the one before last nor from the one after next, and the MMAs run through a tile's other
        // blocks without these warps.
        unsigned block = 0;        // blocks through the ring so far
        uint32_t land_phase = 0;   // per stage
        bool ok = true;
        const int per = p.lora.per, box = p.lora.box, step = box / SLICE;
        const int t0 = (warp - 2 - CF::EPI_WARPS) * 32 + lane;   // this thread's rows of the half: t0, t0 + 64
        for (int tile = cluster; tile < total && ok; tile += nclusters) {
            const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
            const Share sh = share(t);
            const int slices = sh.s1;
            const int32_t* list = p.lora.tile_list + (size_t)t.col_tile * BN;
            const int32_t head = lane * per < slices ? list[lane] : -1;   // the list's first 32 adapters
            int id[2];
            const uint4* u[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = t0 + 64 * j, col = (int)rank * (t.nn / 2) + r;
                const bool live = r < t.nn / 2 && col < t.valid;
                id[j] = live ? p.lora.adapter[(size_t)t.c0 + col] : -1;
                u[j] = reinterpret_cast<const uint4*>(
                    p.lora.u + ((size_t)t.c0 + (live ? col : 0)) * p.lora.terms * p.lora.R16);
            }
            // copies of a stage go out as soon as it is free; the stage before is then waited for and handed over
            block += sh.kb1 - sh.kb0;
            auto hand_over = [&](unsigned blk) {
                ptx::fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive_operands(ptx::map_to_rank(ptx::smem_addr(&ctrl->ready[blk % NST]), lead));
            };
            for (int s0 = sh.s0; s0 < slices; s0 += SLICES, ++block) {
                const int stage = block % NST, n = min(SLICES, slices - s0);
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(&ctrl->land[stage], land_phase >> stage & 1, wc));
                if (!ok) break;
                land_phase ^= 1u << stage;
                const uint32_t sb = ptx::smem_addr(smem + stage * STAGE + W * A_BYTES);
#pragma unroll
                for (int i = 0; i < SLICES; ++i) {
                    if (i >= n) break;
                    const int k = (s0 + i) / per, part16 = (s0 + i) % per;
                    const int h = __shfl_sync(0xffffffffu, head, k & 31);
                    const int a = k < 32 ? h : list[k];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = t0 + 64 * j;
                        if (r >= t.nn / 2) continue;
                        // box i / step, rows of 2 box bytes whose 16-byte chunks are permuted by row as TMA does
                        const int chunk = i % step * 2, x = swizzle(r, box);
                        const uint32_t row = sb + i / step * step * SLICE_BYTES + r * 2 * box;
                        ptx::cp_async16(row + (chunk ^ x) * 16, u[j] + 2 * part16, id[j] == a);
                        ptx::cp_async16(row + ((chunk + 1) ^ x) * 16, u[j] + 2 * part16 + 1, id[j] == a);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (s0 > sh.s0) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    hand_over(block - 1);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (ok && sh.s0 < slices) hand_over(block - 1);
        }
    }

    if (SPLIT) {
        ptx::tc_fence_before_sync();
        __syncwarp();
        ptx::cluster_sync();
        if (cluster < total) {
            // the columns of this CTA's features: part, part + parts, ... in turn, a warp a column, four
            // features a lane
            const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, cluster);
            const size_t row0 = (WGRAD ? (size_t)t.e * p.C : (size_t)0) + t.c0;
            const int f = t.f0 + (int)rank * BM + 4 * lane;
            const uint32_t mine = ptx::smem_addr(smem) + 16 * lane;
            for (int c = part + parts * warp; c < t.valid; c += parts * (CF::THREADS / 32)) {
                float4 v[MAX_SPLIT];
#pragma unroll
                for (int i = 0; i < MAX_SPLIT; ++i)
                    if (i < parts) v[i] = ptx::ld_cluster4(ptx::map_to_rank(mine + c * BM * 4, 2 * i + rank));
                float s[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int i = 1; i < MAX_SPLIT; ++i)
                    if (i < parts) {
                        s[0] += v[i].x;
                        s[1] += v[i].y;
                        s[2] += v[i].z;
                        s[3] += v[i].w;
                    }
                if (f >= p.F) continue;   // F is a multiple of 8
                if (LORA && not_finite(__float_as_uint(s[0] + s[1] + s[2] + s[3]))) mark_odd(cluster);
                if (p.out16)
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (row0 + c) * p.F + f) =
                        make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + (row0 + c) * p.F + f) =
                        make_float4(s[0], s[1], s[2], s[3]);
            }
        }
    }
    ptx::tc_fence_before_sync();
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
    if (LORA) {
        // Outputs that another request's adapter took with it, where nothing waits for this CTA any more.  Each
        // sees to what it has stored itself.
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < ODD_WORDS; ++i) any |= ctrl->odd[i];
        int turn = 0;
        for (int tile = cluster; any != 0 && tile < total; tile += nclusters, ++turn) {
            if (!(ctrl->odd[turn / 32 % ODD_WORDS] >> turn % 32 & 1)) continue;
            const Tile t = decode<WGRAD, CF::PAIR_F>(ctrl, p, tile);
            const int mine = SPLIT ? (t.valid - part + parts - 1) / parts : t.valid;   // rows
            const int blocks = (mine + 31) / 32;
            for (int i = warp; i < W * BM / 16 * blocks; i += CF::THREADS / 32) {
                const int fg = i / blocks, c = i % blocks * 32;
                const int f0 = t.f0 + fg / (BM / 16) * 2 * BM + (int)rank * BM + fg % (BM / 16) * 16;
                if (f0 < p.F) repair(p, t.e, (size_t)t.c0 + part + (size_t)c * parts, min(32, mine - c), parts, f0);
            }
        }
    }
}

// Wide tiles (512 features) move a quarter fewer operand bytes per MMA through shared memory, which
// bounds the narrow ones (8192 rows of 8 experts, 14336 x 4096, us narrow and wide in loops of 2 s: mm 854, 765; dgrad 848,
// 794; wgrad to bf16 992, 814; 1024 rows 231, 229), but have one accumulator: for outputs of at least two waves of
// them, and where they waste no more than an eighth of the features.
bool wide(const Params& p, long long cols, int pairs) {
    const long long nf = (p.F + 511) / 512;
    return cols * nf >= 2LL * pairs && nf * 512 * 8 <= (long long)p.F * 9;
}

template <int OP, bool OUT16, int W, bool LORA = false, bool SPLIT = false>
cudaError_t launch(const GroupedArgs& a, const Maps& maps, const Params& p, long long col_tiles, cudaStream_t s) {
    using CF = Cfg<OP, OUT16, W, LORA, SPLIT>;
    static PerDeviceOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(grouped_tc_kernel<OP, OUT16, W, LORA, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    CF::SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = SPLIT ? 2 * p.split : 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(CF::THREADS);
    cfg.dynamicSmemBytes = CF::SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    const int most = SPLIT ? 0 : [&] {
        static PerDeviceInt clusters;
        return clusters.get([&] {
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(2 * 74);
            q.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, grouped_tc_kernel<OP, OUT16, W, LORA, SPLIT>, &q) != cudaSuccess ||
                n <= 0) {
                cudaGetLastError();
                n = (a.num_sms > 0 ? a.num_sms : 148) / 2;
            }
            return n;
        });
    }();

    const long long tiles = col_tiles * ((p.F + CF::PAIR_F - 1) / CF::PAIR_F);
    const long long pairs = SPLIT ? tiles * p.split : tiles < most ? tiles : most;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, grouped_tc_kernel<OP, OUT16, W, LORA, SPLIT>, maps, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Clusters of 2 * split CTAs that run at once (a cluster stays within a GPC, so large ones leave SMs over).
template <int OP, bool LORA>
int split_clusters(int split) {
    using CF = Cfg<OP, false, 1, LORA, true>;
    static PerDeviceInt known[MAX_SPLIT + 1];
    return known[split].get([&] {
        cudaLaunchConfig_t q = {};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2 * split;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        q.gridDim = dim3(2 * 72);
        q.blockDim = dim3(CF::THREADS);
        q.dynamicSmemBytes = CF::SMEM;
        q.attrs = at;
        q.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(grouped_tc_kernel<OP, false, 1, LORA, true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, CF::SMEM) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, grouped_tc_kernel<OP, false, 1, LORA, true>, &q) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        return n;
    });
}

// Pairs that split a tile's reduction: as many as run at once and keep at least four blocks each.
template <int OP, bool LORA>
int split_of(const Params& p, const GroupedArgs& a, long long cols) {
    const long long tiles = cols * ((p.F + 2 * BM - 1) / (2 * BM));
    // wgrad: the reduction is the segments' rows, on average
    const int blocks = (OP == kGroupedWgrad ? a.seg.M / a.seg.E : p.red) / BK;
    int s = 1;
    for (int t = 2; t <= MAX_SPLIT; ++t)
        if (blocks >= 4 * t && tiles <= split_clusters<OP, LORA>(t)) s = t;
    return s;
}

// [L * E][N][R] bf16: boxes of `width` ranks x 128 features, swizzled over the box's rows
bool map_adapters(CUtensorMap* m, const GroupedArgs& a, int width) {
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.R, (cuuint64_t)a.N, (cuuint64_t)a.L * a.seg.E};
    cuuint64_t strides[2] = {(cuuint64_t)a.R * 2, (cuuint64_t)a.R * a.N * 2};
    cuuint32_t box[3] = {(cuuint32_t)width, BM, 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.B), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              width == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
              : width == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                            : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OP>
cudaError_t launch_op(const GroupedArgs& a, cudaStream_t s) {
    const int M = a.seg.M, E = a.seg.E, N = a.N, K = a.K;
    Params p{};
    p.seg = a.seg;
    p.F = OP == kGroupedMm ? N : K;
    p.C = N;
    p.red = OP == kGroupedMm ? K : N;
    p.out = a.out;
    p.status = a.status;
    p.wait_ns = a.wait_ns;
    p.f_fast = K <= N;
    Maps m;
    bool ok;
    long long cols;   // upper bound of the tiles along the columns
    if (OP == kGroupedWgrad) {
        ok = map_matrix(&m.a, a.other, M, K, BOX, BK) && map_matrix(&m.b[0], a.rows, M, N, BOX, BK);
        for (int i = 1; i < 4; ++i) m.b[i] = m.b[0];
        cols = (long long)E * ((N + BN - 1) / BN);
    } else {
        ok = OP == kGroupedMm ? map_expert_weights(&m.a, a.other, E, N, K, BK, BM)
                              : map_expert_weights(&m.a, a.other, E, N, K, BOX, BK);
        for (int i = 0; i < 4; ++i) ok = ok && map_matrix(&m.b[i], a.rows, M, p.red, BK, 16 << i);
        cols = (long long)M / BN + E;
        if (cols > M) cols = M;   // a segment with rows has at least one
    }
    if (!ok) return cudaErrorInvalidValue;
    p.out16 = a.out16;
    if (OP == kGroupedMm && a.A) {
        p.split = split_of<kGroupedMm, true>(p, a, cols);
        p.lora = lora_view(a);
        p.x = static_cast<const __nv_bfloat16*>(a.rows);
        p.W = static_cast<const __nv_bfloat16*>(a.other);
        if (!map_adapters(&m.l, a, p.lora.box)) return cudaErrorInvalidValue;
        if (p.split > 1) return launch<kGroupedMm, false, 1, true, true>(a, m, p, cols, s);
        if (!a.out16) return launch<kGroupedMm, false, 1, true>(a, m, p, cols, s);
        return wide(p, cols, (a.num_sms > 0 ? a.num_sms : 148) / 2) ? launch<kGroupedMm, true, 2, true>(a, m, p, cols, s)
                             : launch<kGroupedMm, true, 1, true>(a, m, p, cols, s);
    }
    m.l = m.a;
    p.split = split_of<OP, false>(p, a, cols);
    if (p.split > 1) return launch<OP, false, 1, false, true>(a, m, p, cols, s);
    if (!a.out16) return launch<OP, false, 1>(a, m, p, cols, s);
    return wide(p, cols, (a.num_sms > 0 ? a.num_sms : 148) / 2) ? launch<OP, true, 2>(a, m, p, cols, s) : launch<OP, true, 1>(a, m, p, cols, s);
}

}  // namespace

cudaError_t launch_grouped_tc(const GroupedArgs& a, cudaStream_t s) {
    switch (a.op) {
        case kGroupedMm: return launch_op<kGroupedMm>(a, s);
        case kGroupedDgrad: return launch_op<kGroupedDgrad>(a, s);
        default: return launch_op<kGroupedWgrad>(a, s);
    }
}

}  // namespace moe
