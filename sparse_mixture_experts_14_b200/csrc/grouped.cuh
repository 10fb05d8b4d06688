// Shared by the ragged grouped products (grouped_*.cu, lora.cu): the segments of
// the rows, their tile table, and the launcher declarations.
//
// Segment e holds rows [offsets[e], offsets[e] + n_e) of the row buffers, with
// n_e = counts[e], or offsets[e + 1] - offsets[e] when no counts are given.
// Segments need no alignment and may leave gaps; rows outside every segment are
// neither used nor written.
#pragma once

#include "moe_common.cuh"

namespace moe {

constexpr int kMaxGroups = 256;   // experts of a grouped product (the tile table is in shared memory)

struct Segments {
    const int32_t* offsets;   // [E + 1] device
    const int32_t* counts;    // [E] device or null
    int E;
    int M;                    // rows of the row buffers
    int least = 0, most = 0x7fffffff;   // segments with fewer or more rows are left to another kernel
};

// Tiles of `tile` rows: expert e owns tiles [base[e], base[e + 1]).
struct SegTable {
    int row0[kMaxGroups];
    int rows[kMaxGroups];
    int base[kMaxGroups + 1];
    int total;
    bool good;   // (a table of which no segment has rows may be good or bad)
};

// Built by one whole warp.  A segment outside the row buffers, or one that runs
// into the next, records MOE_ERR_DEVICE and leaves the table without tiles.
__device__ __forceinline__ void build_segments(SegTable* t, const Segments& s, int tile, int* status) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    bool ok = true;
    for (int e0 = 0; e0 < s.E; e0 += 32) {
        const int e = e0 + lane;
        int tiles = 0;
        if (e < s.E) {
            const int o0 = s.offsets[e], o1 = s.offsets[e + 1];
            const int n = s.counts ? s.counts[e] : o1 - o0;
            const bool good = o0 >= 0 && o1 >= o0 && o1 <= s.M && n >= 0 && n <= o1 - o0;
            ok = ok && good;
            tiles = good && n >= s.least && n <= s.most ? (n + tile - 1) / tile : 0;
            t->row0[e] = good ? o0 : 0;
            t->rows[e] = good ? n : 0;
        }
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        if (e < s.E) t->base[e] = carry + inc - tiles;
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
        if (!ok) record_status(status, MOE_ERR_DEVICE);
        t->base[s.E] = carry;
        t->total = ok ? carry : 0;
        t->good = ok;
    }
    if (!ok) {
        __syncwarp();
        for (int e = lane; e < s.E; e += 32) t->rows[e] = 0;
    }
}

// The expert that owns a tile: the last e with base[e] <= tile (tile < base[E]).
__device__ __forceinline__ int segment_of(const SegTable* t, int E, int tile) {
    int lo = 0, hi = E;   // base[lo] <= tile < base[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t->base[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

enum GroupedOp : int {
    kGroupedMm = 0,     // y_r  = W_e x_r
    kGroupedDgrad = 1,  // dx_r = W_e^T dy_r
    kGroupedWgrad = 2,  // dW_e = sum_r dy_r x_r^T
};

struct GroupedArgs {
    GroupedOp op;
    const void* rows;   // mm: x [M][K]; dgrad, wgrad: dy [M][N]
    const void* other;  // mm, dgrad: W [E][N][K]; wgrad: x [M][K]
    void* out;          // mm [M][N], dgrad [M][K], wgrad [E][N][K]
    Segments seg;
    int N, K;
    bool in16, out16;   // bfloat16 instead of float
    // adapters (mm only; A == null: none)
    const void* A;      // [L][E][R][K]
    const void* B;      // [L][E][N][R]
    const float* scale; // [L]
    const int32_t* adapter;   // [M], -1: none
    int L, R;
    uint8_t* ws;        // adapters: the shrunken rows u and the lists of the tiles
    int num_sms;
    int* status;
    long long wait_ns;
};

// Column tiles of a segment of n rows: ceil(n / 256) of them, their heights multiples of 32 that differ by 32 at
// most, `first` of `height` rows and then lower ones, so that at most 31 rows of a segment are computed in vain
// and neighbouring CTAs have equal work.  (Tiles of 256 rows and a rest computed as little, but beside an even
// number of CTA pairs every other pair then got the rests: 4096 rows with adapters 537 -> 573 us.)
constexpr int kColumnTile = 256;
struct ColumnTiles {
    int height, first;
    __host__ __device__ int start(int i) const { return i * height - 32 * (i > first ? i - first : 0); }
    __host__ __device__ int rows(int i) const { return i < first ? height : height - 32; }
};
__host__ __device__ inline ColumnTiles column_tiles(int n) {
    const int tt = (n + kColumnTile - 1) / kColumnTile;
    if (tt == 0) return {32, 0};
    const int h = ((n + tt - 1) / tt + 31) / 32 * 32;
    return {h, (n - tt * (h - 32) + 31) / 32};
}

// The adapters as the products' kernels see them.  u is a workspace buffer [M][terms][R16], R16 = R
// rounded up to 16 (zeros behind R); rows without an adapter hold nothing.  u is the sum of `terms` bf16 values:
// three beside an fp32 output, which hold fp32's 24 bits (one alone, off by up to 2^-8 of u, would be the largest error by
// far); for a bf16 output one where grouped_tc multiplies it, rounded like any of its operands, and two where
// grouped_few alone does, on the CUDA cores.  (Two in grouped_tc: error 1.81e-3 -> 1.66e-3 of the result, which is
// the output's own rounding, but 205 rows of 40 adapters of rank 32 take 47.1 us instead of 40.7, 4096 rows of 12 of
// rank 64 549 instead of 508; in grouped_few, 32 rows, 167.8 and 167.4.)
struct LoraView {
    const __nv_bfloat16* B;        // [L][E][N][R]
    const int32_t* adapter;        // [M]
    __nv_bfloat16* u;              // [M][terms][R16]
    int32_t* tile_list;            // [column tiles][256]: the adapters that occur in the tile, each once
    int32_t* tile_count;           // [column tiles]
    int L, R, R16;
    int terms;                     // 1, 2 or 3
    int per;                       // 16-wide slices of an adapter's part of a row of u
    int box;                       // ranks of a box of B: the widest of 64, 32, 16 that divides R16
};

// One output's own adapter term, u_r B^T[f], for adapter-expert pair ae; N features.
template <int TERMS>
__device__ __forceinline__ float adapter_term(const LoraView& l, size_t ae, int N, size_t row, int f) {
    const uint4* bl = reinterpret_cast<const uint4*>(l.B + (ae * N + f) * l.R);
    const uint4* ul = reinterpret_cast<const uint4*>(l.u + row * TERMS * l.R16);
    float d = 0.f;
#pragma unroll 2
    for (int j = 0; j < l.R / 8; ++j) {
        const uint4 m = __ldg(bl + j);
        const uint32_t mw[4] = {m.x, m.y, m.z, m.w};
        uint4 n[TERMS];
#pragma unroll
        for (int t = 0; t < TERMS; ++t) n[t] = ul[t * (l.R16 / 8) + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t) {   // (exact)
                const uint32_t nw = i == 0 ? n[t].x : i == 1 ? n[t].y : i == 2 ? n[t].z : n[t].w;
                lo += bf16_lo(nw);
                hi += bf16_hi(nw);
            }
            d = fmaf(bf16_lo(mw[i]), lo, d);
            d = fmaf(bf16_hi(mw[i]), hi, d);
        }
    }
    return d;
}

inline size_t lora_tiles(int M, int E) { return (size_t)M / kColumnTile + E; }
inline size_t lora_u_bytes(int M, int R) { return align_up((size_t)M * 3 * ((R + 15) / 16 * 16) * 2, 256); }
inline size_t lora_workspace_bytes(int M, int E, int R) {
    return lora_u_bytes(M, R) + align_up(lora_tiles(M, E) * (kColumnTile + 1) * 4, 256);
}
cudaError_t launch_grouped_simt(const GroupedArgs& a, cudaStream_t s);   // float
cudaError_t launch_grouped_tc(const GroupedArgs& a, cudaStream_t s);     // bfloat16, M > 0
cudaError_t launch_grouped_few(const GroupedArgs& a, cudaStream_t s);    // bfloat16 mm with few rows

// Which of the two takes a bf16 mm: the segments with at most `few` rows go to grouped_few, the others to
// grouped_tc; `both`: the host cannot tell which there are.
struct Choice {
    bool few, tc;
    int limit;
};
Choice grouped_choice(const GroupedArgs& a);
inline LoraView lora_view(const GroupedArgs& a) {
    LoraView v;
    v.B = static_cast<const __nv_bfloat16*>(a.B);
    v.adapter = a.adapter;
    v.u = reinterpret_cast<__nv_bfloat16*>(a.ws);
    v.tile_list = reinterpret_cast<int32_t*>(a.ws + lora_u_bytes(a.seg.M, a.R));
    v.tile_count = v.tile_list + lora_tiles(a.seg.M, a.seg.E) * kColumnTile;
    v.L = a.L;
    v.R = a.R;
    v.R16 = (a.R + 15) / 16 * 16;
    v.terms = !a.out16 ? 3 : grouped_choice(a).tc ? 1 : 2;
    v.per = v.terms * v.R16 / 16;
    v.box = v.R16 % 64 == 0 ? 64 : v.R16 % 32 == 0 ? 32 : 16;
    return v;
}
cudaError_t launch_lora_shrink(const GroupedArgs& a, cudaStream_t s);    // u and the tiles' lists

}  // namespace moe
