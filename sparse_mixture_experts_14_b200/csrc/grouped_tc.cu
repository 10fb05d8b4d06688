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
// instruction field: a segment of n rows is cut into ceil(n / 256) tiles of equal
// height, rounded up to 32, so that no more than 31 rows a tile are computed in
// vain (a 256-row M side would round every segment up to 256).
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
// (in the pair's leader), 4 or 8 epilogue warps for the CTA's 128 features out of two
// alternating accumulators, a further warp for the ends of wgrad's segments.
//
// fp32 outputs: the tensor cores truncate when they add to the accumulator, which
// costs 1.8e-8 of the result per 16-deep step, all in one direction (1.6e-5 at a
// reduction of 14336, where a blocked fp32 sum has 3e-7).  So the accumulator takes
// 512 of the reduction at a time, and the epilogue adds these partial sums in
// registers with rounding, while the MMAs go on in the other accumulator.  bf16
// outputs, whose own rounding is 2^-9, take the whole reduction in one.
//
// wgrad: the last 64-row block of a segment also holds rows of the next one, which
// must not count, whatever they hold (NaN times zero is NaN).  The MMA stops at the
// 16-row slice of the segment's last row, and an extra warp in each CTA clears
// the rest of that slice in shared memory, in both operands, before the MMA may
// read it.
#include <cuda.h>

#include "grouped.cuh"
#include "ptx_grouped.cuh"
#include "tma_map.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                    // features per CTA (256 per pair)
constexpr int BN = 256;                    // columns of a tile at most
constexpr int BK = 64;                     // reduction per stage
constexpr int NST = 6;
constexpr int A_BYTES = BM * BK * 2;       // 16 KiB
constexpr int B_BYTES = BN / 2 * BK * 2;   // 16 KiB
constexpr int STAGE = A_BYTES + B_BYTES;
constexpr int BOX = 64;                    // MN-major operands: 64-wide boxes
constexpr uint32_t MN_LBO = BOX * BK * 2;
constexpr uint32_t MN_SBO = 1024;
constexpr int TMEM_COLS = 2 * BN;
constexpr int CHUNK = 512 / BK;            // blocks per accumulator, fp32 outputs

struct Maps {
    CUtensorMap a;
    CUtensorMap b[4];   // boxes of 16, 32, 64 and 128 rows (mm, dgrad); wgrad: b[0] only
};

struct Params {
    Segments seg;
    int F;            // features: the output's contiguous dimension
    int C;            // wgrad: columns (N)
    int red;          // mm, dgrad: length of the reduction
    void* out;
    int* status;
    long long wait_ns;
};

struct Ctrl {
    uint64_t full[NST];     // leader: both CTAs' bytes of a stage landed
    uint64_t empty[NST];    // each CTA: the MMAs that read a stage are done
    uint64_t land[NST];     // wgrad: this CTA's bytes of a segment's last block landed
    uint64_t ready[NST];    // leader: both CTAs prepared the stage by hand
    uint64_t tfull[2];      // each CTA: accumulator b holds a finished tile
    uint64_t tempty[2];     // leader: both CTAs' epilogues released accumulator b
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int total;
    SegTable seg;
};

template <int OP, bool OUT16>
struct Cfg {
    static constexpr bool WGRAD = OP == kGroupedWgrad;
    static constexpr bool A_MN = OP != kGroupedMm;
    static constexpr bool B_MN = WGRAD;
    static constexpr int AUX_WARPS = WGRAD ? 1 : 0;
    static constexpr int EPI_WARPS = OUT16 ? 4 : 8;
    static constexpr int THREADS = 32 * (2 + EPI_WARPS + AUX_WARPS);
    static constexpr int SMEM = NST * STAGE + (int)sizeof(Ctrl) + 1024;
};

// One tile: expert, first feature of the pair, first column (row of the row buffers, or n of dW),
// columns of the MMA and those that count, 64-deep blocks.
struct Tile {
    int e, f0, c0, nn, valid, nkb, rows, row0;
};

__host__ __device__ inline int tile_height(int n) {   // rows of a token tile of a segment of n rows
    const int tt = (n + BN - 1) / BN;
    return tt > 0 ? ((n + tt - 1) / tt + 31) / 32 * 32 : 32;
}

template <bool WGRAD>
__device__ __forceinline__ Tile decode(const Ctrl* c, const Params& p, int tile) {
    Tile t;
    const int nf = (p.F + 2 * BM - 1) / (2 * BM);
    if (WGRAD) {
        // columns fastest: the pairs at work share blocks of x
        const int nc = (p.C + BN - 1) / BN;
        t.e = tile / (nf * nc);
        const int local = tile - t.e * nf * nc;
        const int fi = local / nc;
        t.f0 = fi * 2 * BM;
        t.c0 = (local - fi * nc) * BN;
        t.rows = c->seg.rows[t.e];
        t.row0 = c->seg.row0[t.e];
        t.valid = min(BN, p.C - t.c0);
        t.nn = (t.valid + 31) / 32 * 32;
        t.nkb = (t.rows + BK - 1) / BK;
    } else {
        // token tiles fastest: the pairs at work share blocks of the weights
        const int tok = tile / nf;   // any tile of the expert's group
        t.e = segment_of(&c->seg, p.seg.E, tok);
        const int tt = c->seg.base[t.e + 1] - c->seg.base[t.e];
        const int local = tile - c->seg.base[t.e] * nf;
        const int fi = local / tt;
        t.rows = c->seg.rows[t.e];
        const int h = tile_height(t.rows);
        const int r = (local - fi * tt) * h;
        t.f0 = fi * 2 * BM;
        t.row0 = c->seg.row0[t.e];
        t.c0 = t.row0 + r;
        t.valid = min(h, t.rows - r);
        t.nn = h;
        t.nkb = (p.red + BK - 1) / BK;
    }
    return t;
}

// Index of the row box that holds n rows (n a multiple of 16, at most 128).
__device__ __forceinline__ int box_of(int n) { return n <= 16 ? 0 : n <= 32 ? 1 : n <= 64 ? 2 : 3; }

template <int OP, bool OUT16>
__global__ void __launch_bounds__(Cfg<OP, OUT16>::THREADS, 1)
    grouped_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
    using CF = Cfg<OP, OUT16>;
    constexpr bool WGRAD = CF::WGRAD;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + NST * STAGE);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1;
    const int nclusters = gridDim.x >> 1;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(&ctrl->full[s], 1);
            ptx::mbar_init(&ctrl->empty[s], 1);
            ptx::mbar_init(&ctrl->land[s], 1);
            ptx::mbar_init(&ctrl->ready[s], 2);
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
    if (warp == 1) {
        ptx::tmem_alloc_pair(&ctrl->tmem_base, TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    pdl_wait();
    if (warp == 0) {
        build_segments(&ctrl->seg, p.seg, BN, leader && cluster == 0 ? p.status : nullptr);
        __syncwarp();
        if (lane == 0) {
            const int nf = (p.F + 2 * BM - 1) / (2 * BM);
            const bool ok = ctrl->seg.total == ctrl->seg.base[p.seg.E];
            ctrl->total = !ok ? 0 : WGRAD ? p.seg.E * nf * ((p.C + BN - 1) / BN) : ctrl->seg.total * nf;
        }
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();
    ptx::tc_fence_after_sync();

    const uint32_t tmem_base = ctrl->tmem_base;
    const int total = ctrl->total;
    const ptx::WaitCtl wc{&ctrl->abort, p.status, (uint64_t)p.wait_ns};

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        if (lane == 0) {
            const uint64_t pol = ptx::policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            uint32_t armed = 0, armed_phase = 0, tail = 0, tail_phase = 0;   // bits per stage
            bool aborted = false;
            for (int tile = cluster; tile < total && !aborted; tile += nclusters) {
                const Tile t = decode<WGRAD>(ctrl, p, tile);
                const int fa = t.f0 + (int)rank * BM;
                const int half = t.nn / 2;
                const int cb = t.c0 + (int)rank * half;
                const int box = WGRAD ? 0 : box_of(half);
                const int bboxes = WGRAD ? (half + BOX - 1) / BOX : 1;
                const uint32_t bytes = A_BYTES + (WGRAD ? bboxes * (int)MN_LBO : (16 << box) * BK * 2);
                for (int kb = 0; kb < t.nkb; ++kb) {
                    if (!ptx::mbar_wait(&ctrl->empty[stage], phase ^ 1u, wc)) {
                        aborted = true;
                        break;
                    }
                    uint8_t* sa = smem + stage * STAGE;
                    uint8_t* sb = sa + A_BYTES;
                    const int k = kb * BK;
                    if (WGRAD && kb == t.nkb - 1 && (t.rows & 15) != 0) {
                        // the segment's last block: this CTA's own barrier, the clearing warp goes on from there
                        ptx::mbar_arrive_expect_tx(&ctrl->land[stage], bytes);
                        if (leader) ptx::mbar_arrive(&ctrl->full[stage]);
                        uint64_t* bar = &ctrl->land[stage];
                        ptx::tma_load_2d(sa, &maps.a, bar, fa, t.row0 + k, pol);
                        ptx::tma_load_2d(sa + MN_LBO, &maps.a, bar, fa + BOX, t.row0 + k, pol);
                        for (int h = 0; h < bboxes; ++h)
                            ptx::tma_load_2d(sb + h * MN_LBO, &maps.b[0], bar, cb + h * BOX, t.row0 + k, pol);
                        tail |= 1u << stage;
                    } else {
                        const uint32_t bar = ptx::map_to_rank(ptx::smem_addr(&ctrl->full[stage]), 0);
                        if (leader) ptx::mbar_arrive_expect_tx(&ctrl->full[stage], 2 * bytes);
                        if (WGRAD) {
                            ptx::tma_load_2d_pair(sa, &maps.a, bar, fa, t.row0 + k, pol);
                            ptx::tma_load_2d_pair(sa + MN_LBO, &maps.a, bar, fa + BOX, t.row0 + k, pol);
                            for (int h = 0; h < bboxes; ++h)
                                ptx::tma_load_2d_pair(sb + h * MN_LBO, &maps.b[0], bar, cb + h * BOX, t.row0 + k, pol);
                        } else {
                            if (CF::A_MN) {
                                ptx::tma_load_3d_pair(sa, &maps.a, bar, fa, k, t.e, pol);
                                ptx::tma_load_3d_pair(sa + MN_LBO, &maps.a, bar, fa + BOX, k, t.e, pol);
                            } else {
                                ptx::tma_load_3d_pair(sa, &maps.a, bar, k, fa, t.e, pol);
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
            for (int tile = cluster; tile < total && !aborted; tile += nclusters) {
                const Tile t = decode<WGRAD>(ctrl, p, tile);
                const uint32_t idesc = ptx::idesc_bf16_f32(2 * BM, t.nn, CF::A_MN, CF::B_MN);
                uint32_t d_tmem = 0;
                for (int kb = 0; kb < t.nkb; ++kb) {
                    const bool first = OUT16 ? kb == 0 : kb % CHUNK == 0;   // of an accumulator
                    bool ok = true;
                    if (first) {
                        ok = ptx::mbar_wait(&ctrl->tempty[acc], acc_phase ^ 1u, wc);
                        ptx::tc_fence_after_sync();
                        d_tmem = tmem_base + (uint32_t)(acc * BN);
                    }
                    ok = ok && ptx::mbar_wait(&ctrl->full[stage], phase, wc);
                    int slices = BK / 16;
                    if (WGRAD && kb == t.nkb - 1) {
                        slices = (t.rows - kb * BK + 15) / 16;
                        if (ok && (t.rows & 15) != 0) {
                            ok = ptx::mbar_wait_cluster(&ctrl->ready[stage], hand_phase >> stage & 1, wc);
                            hand_phase ^= 1u << stage;
                        }
                    }
                    if (!ok) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const uint32_t a0 = ptx::smem_addr(smem + stage * STAGE);
                    const uint32_t b0 = a0 + A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        if (WGRAD && kk >= slices) break;
                        const uint64_t da = CF::A_MN ? ptx::desc_mnmajor_sw128(a0 + kk * 2048, MN_LBO, MN_SBO)
                                                     : ptx::desc_kmajor_sw128(a0 + kk * 32);
                        const uint64_t db = CF::B_MN ? ptx::desc_mnmajor_sw128(b0 + kk * 2048, MN_LBO, MN_SBO)
                                                     : ptx::desc_kmajor_sw128(b0 + kk * 32);
                        ptx::tc_mma_bf16_pair(d_tmem, da, db, idesc, !(first && kk == 0));
                    }
                    ptx::tc_commit_pair_multicast(&ctrl->empty[stage], 0x3);
                    issued = true;
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (kb == t.nkb - 1 || (!OUT16 && kb % CHUNK == CHUNK - 1)) {
                        ptx::tc_commit_pair_multicast(&ctrl->tfull[acc], 0x3);
                        acc ^= 1;
                        if (acc == 0) acc_phase ^= 1u;
                    }
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
            const Tile t = decode<WGRAD>(ctrl, p, tile);
            const int f = t.f0 + (int)rank * BM + q * 32 + lane;
            const size_t row0 = WGRAD ? (size_t)t.e * p.C + t.c0 : (size_t)t.c0;
            if (OUT16) {
                // (no rows in the segment: nothing was accumulated, the sum is zero)
                if (t.nkb > 0) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&ctrl->tfull[acc], acc_phase, wc));
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint32_t taddr = tmem_base + (uint32_t)(acc * BN) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
                for (int c = 0; c < t.nn; c += 32) {
                    uint32_t r[32];
                    if (t.nkb > 0) {
                        ptx::tmem_ld_32x32b_x32(taddr + c, r);
                        ptx::tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0u;
                    }
                    // neighbouring lanes swap one of two columns: the even lane stores features f, f + 1 of
                    // column i, the odd one features f - 1, f of column i + 1 (F is a multiple of 8)
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (f & ~1);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float mine = __uint_as_float(lane & 1 ? r[i + 1] : r[i]);
                        const float send = __uint_as_float(lane & 1 ? r[i] : r[i + 1]);
                        const float got = __shfl_xor_sync(0xffffffffu, send, 1);
                        const uint32_t v = lane & 1 ? pack_bf16x2(got, mine) : pack_bf16x2(mine, got);
                        const int col = c + i + (lane & 1);
                        if (col < t.valid && f < p.F)
                            *reinterpret_cast<uint32_t*>(out + (row0 + col) * (size_t)p.F) = v;
                    }
                }
                if (t.nkb == 0) continue;
                // the accumulator is free once every lane's tcgen05.ld has completed
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(ptx::smem_addr(&ctrl->tempty[acc]), 0));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            } else {
                // two warps per lane quarter, each with half of the columns (a multiple of 16)
                const int half = t.nn / 2, c0 = (warp - 2) / 4 * half;
                float sum[BN / 2];
#pragma unroll
                for (int i = 0; i < BN / 2; ++i) sum[i] = 0.f;
                for (int kb = 0; kb < t.nkb && ok; kb += CHUNK) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&ctrl->tfull[acc], acc_phase, wc));
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint32_t taddr = tmem_base + (uint32_t)(acc * BN + c0) + ((uint32_t)(q * 32) << 16);
#pragma unroll
                    for (int c = 0; c < BN / 2; c += 16) {
                        if (c < half) {
                            uint32_t r[16];
                            ptx::tmem_ld_32x32b_x16(taddr + c, r);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(r[i]);
                        }
                    }
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(ptx::smem_addr(&ctrl->tempty[acc]), 0));
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
                if (!ok) break;
                float* out = static_cast<float*>(p.out) + (row0 + c0) * (size_t)p.F + f;
#pragma unroll
                for (int i = 0; i < BN / 2; ++i)
                    if (i < half && c0 + i < t.valid && f < p.F) out[i * (size_t)p.F] = sum[i];
            }
        }
    } else if (WGRAD) {
        // ---------------------------------------------------------------- ends of segments (both CTAs)
        int block = 0;             // blocks through the ring so far
        uint32_t land_phase = 0;   // per stage
        for (int tile = cluster; tile < total; tile += nclusters) {
            const Tile t = decode<WGRAD>(ctrl, p, tile);
            block += t.nkb;
            if ((t.rows & 15) == 0) continue;
            const int stage = (block - 1) % NST;
            bool ok = ptx::mbar_wait(&ctrl->land[stage], land_phase >> stage & 1, wc);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            land_phase ^= 1u << stage;
            // rows of the block that lie in its last 16-row slice behind the segment: 128 bytes a row and box
            const int r0 = (t.rows - 1) % BK + 1, r1 = (r0 + 15) / 16 * 16;
            uint8_t* base = smem + stage * STAGE;
            for (int i = lane; i < (r1 - r0) * 4 * 8; i += 32) {
                const int v = i & 7, box = (i >> 3) & 3, r = r0 + (i >> 5);
                *reinterpret_cast<uint4*>(base + box * (int)MN_LBO + r * 128 + v * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_addr(&ctrl->ready[stage]), 0));
        }
    }

    ptx::tc_fence_before_sync();
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

template <int OP, bool OUT16>
cudaError_t launch(const GroupedArgs& a, const Maps& maps, const Params& p, long long tiles, cudaStream_t s) {
    using CF = Cfg<OP, OUT16>;
    static PerDeviceOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(grouped_tc_kernel<OP, OUT16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    CF::SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(CF::THREADS);
    cfg.dynamicSmemBytes = CF::SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    static PerDeviceInt clusters;
    const int most = clusters.get([&] {
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3(2 * 74);
        q.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, grouped_tc_kernel<OP, OUT16>, &q) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = (a.num_sms > 0 ? a.num_sms : 148) / 2;
        }
        return n;
    });
    cfg.gridDim = dim3((unsigned)(2 * (tiles < most ? (tiles > 0 ? tiles : 1) : most)));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, grouped_tc_kernel<OP, OUT16>, maps, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int OP>
cudaError_t launch_op(const GroupedArgs& a, cudaStream_t s) {
    const int M = a.seg.M, E = a.seg.E, N = a.N, K = a.K;
    Params p{a.seg, OP == kGroupedMm ? N : K, N, OP == kGroupedMm ? K : N, a.out, a.status, a.wait_ns};
    Maps m;
    bool ok;
    long long tiles = (p.F + 2 * BM - 1) / (2 * BM);
    if (OP == kGroupedWgrad) {
        ok = map_matrix(&m.a, a.other, M, K, BOX, BK) && map_matrix(&m.b[0], a.rows, M, N, BOX, BK);
        for (int i = 1; i < 4; ++i) m.b[i] = m.b[0];
        tiles *= (long long)E * ((N + BN - 1) / BN);
    } else {
        ok = OP == kGroupedMm ? map_expert_weights(&m.a, a.other, E, N, K, BK, BM)
                              : map_expert_weights(&m.a, a.other, E, N, K, BOX, BK);
        for (int i = 0; i < 4; ++i) ok = ok && map_matrix(&m.b[i], a.rows, M, p.red, BK, 16 << i);
        const long long tok = (long long)M / BN + E;
        tiles *= tok < M ? tok : M;   // a segment with rows has at least one
    }
    if (!ok) return cudaErrorInvalidValue;
    return a.out16 ? launch<OP, true>(a, m, p, tiles, s) : launch<OP, false>(a, m, p, tiles, s);
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
