// C ABI of the ragged grouped products and the adapters beside them: argument
// checks and launches.  See include/moe.h for the contract of each call.
#include <climits>

#include "grouped.cuh"

namespace moe {
int* status_word(int dev);
cudaMemPool_t library_pool(int dev);
int device_sms(int dev);
long long pipeline_wait_ns();

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status check(const GroupedArgs& a, int M, int dtype, int out_dtype) {
    if (M < 0 || a.N <= 0 || a.K <= 0 || a.seg.E <= 0) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DTYPE_F32 && (out_dtype != MOE_DTYPE_BF16 || dtype != MOE_DTYPE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (a.seg.E > kMaxGroups) return MOE_ERR_UNSUPPORTED;
    const int step = dtype == MOE_DTYPE_BF16 ? 8 : 4;
    if (a.N % step != 0 || a.K % step != 0) return MOE_ERR_UNSUPPORTED;
    // tile counts and row coordinates are 32-bit
    const long long cols = a.N > a.K ? a.N : a.K;
    if (M > INT_MAX - 512 || ((long long)M / 32 + a.seg.E + 1) * (cols / 64 + 1) > INT_MAX ||
        (long long)a.seg.E * (a.N / 64 + 1) * (a.K / 64 + 1) > INT_MAX)
        return MOE_ERR_UNSUPPORTED;
    if (!a.seg.offsets || !aligned(a.seg.offsets, 4) || !aligned(a.seg.counts, 4)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a.rows, 16) || !aligned(a.other, 16) || !aligned(a.out, 16)) return MOE_ERR_INVALID_ARG;
    const bool wgrad = a.op == kGroupedWgrad;
    if (wgrad ? !a.out || (M > 0 && (!a.rows || !a.other)) : M > 0 && (!a.rows || !a.other || !a.out))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

bool on_device(GroupedArgs* a, int dev) {
    a->status = dev >= 0 ? status_word(dev) : nullptr;
    a->num_sms = device_sms(dev);
    a->wait_ns = pipeline_wait_ns();
    return a->status != nullptr;
}

cudaError_t launch_product(const GroupedArgs& a, cudaStream_t s) {
    if (!a.in16) return launch_grouped_simt(a, s);
    const Choice c = grouped_choice(a);
    GroupedArgs part = a;
    if (c.few) {
        if (c.tc) part.seg.most = c.limit;
        const cudaError_t e = launch_grouped_few(part, s);
        if (e != cudaSuccess || !c.tc) return e;
        part.seg.least = c.limit + 1;
        part.seg.most = a.seg.most;
    }
    return launch_grouped_tc(part, s);
}

moe_status run(GroupedOp op, const void* rows, const void* other, const int32_t* offsets, const int32_t* counts,
               void* out, int M, int N, int K, int E, int dtype, int out_dtype, cudaStream_t s) {
    GroupedArgs a{};
    a.op = op;
    a.rows = rows;
    a.other = other;
    a.out = out;
    a.seg.offsets = offsets;
    a.seg.counts = counts;
    a.seg.E = E;
    a.seg.M = M;
    a.N = N;
    a.K = K;
    a.in16 = dtype == MOE_DTYPE_BF16;
    a.out16 = out_dtype == MOE_DTYPE_BF16;
    const moe_status st = check(a, M, dtype, out_dtype);
    if (st != MOE_OK || (M == 0 && op != kGroupedWgrad)) return st;
    const DeviceScope scope(out, false);
    if (!on_device(&a, scope.device())) return MOE_ERR_CUDA;
    cudaError_t e;
    if (M == 0)   // no rows: every weight gradient is zero
        e = cudaMemsetAsync(out, 0, (size_t)E * N * K * (a.out16 ? 2 : 4), s);
    else
        e = launch_product(a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grouped_mm(const void* x, const void* W, const int32_t* offsets, const int32_t* counts, void* y, int M,
                          int N, int K, int E, int dtype, int out_dtype, cudaStream_t stream) {
    return run(kGroupedMm, x, W, offsets, counts, y, M, N, K, E, dtype, out_dtype, stream);
}

moe_status moe_grouped_dgrad(const void* dy, const void* W, const int32_t* offsets, const int32_t* counts, void* dx,
                             int M, int N, int K, int E, int dtype, int out_dtype, cudaStream_t stream) {
    return run(kGroupedDgrad, dy, W, offsets, counts, dx, M, N, K, E, dtype, out_dtype, stream);
}

moe_status moe_grouped_wgrad(const void* dy, const void* x, const int32_t* offsets, const int32_t* counts, void* dW,
                             int M, int N, int K, int E, int dtype, int out_dtype, cudaStream_t stream) {
    return run(kGroupedWgrad, dy, x, offsets, counts, dW, M, N, K, E, dtype, out_dtype, stream);
}

size_t moe_grouped_lora_workspace_size(int M, int E, int L, int R) {
    if (M < 0 || E <= 0 || L <= 0 || R <= 0 || E > kMaxGroups || R > MOE_LORA_MAX_RANK || R % 8 != 0) return 0;
    return lora_workspace_bytes(M, E, R);
}

moe_status moe_grouped_lora(const void* x, const void* W, const int32_t* offsets, const int32_t* counts, const void* A,
                            const void* B, const float* scale, const int32_t* adapter, void* y, int M, int N, int K,
                            int E, int L, int R, int out_dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
    GroupedArgs a{};
    a.op = kGroupedMm;
    a.rows = x;
    a.other = W;
    a.out = y;
    a.seg.offsets = offsets;
    a.seg.counts = counts;
    a.seg.E = E;
    a.seg.M = M;
    a.N = N;
    a.K = K;
    a.in16 = true;
    a.out16 = out_dtype == MOE_DTYPE_BF16;
    a.A = A;
    a.B = B;
    a.scale = scale;
    a.adapter = adapter;
    a.L = L;
    a.R = R;
    const moe_status st = check(a, M, MOE_DTYPE_BF16, out_dtype);
    if (st != MOE_OK) return st;
    if (L <= 0 || R <= 0) return MOE_ERR_INVALID_ARG;
    if (R % 8 != 0 || R > MOE_LORA_MAX_RANK || (long long)L * E > INT_MAX / 256) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    if (!A || !B || !scale || !adapter || !aligned(A, 16) || !aligned(B, 16) || !aligned(scale, 4) ||
        !aligned(adapter, 4))
        return MOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < lora_workspace_bytes(M, E, R))
        return MOE_ERR_WORKSPACE;
    a.ws = static_cast<uint8_t*>(workspace);
    const DeviceScope scope(y, false);
    if (!on_device(&a, scope.device())) return MOE_ERR_CUDA;
    if (launch_lora_shrink(a, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_product(a, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
