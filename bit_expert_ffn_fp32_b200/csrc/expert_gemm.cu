// Unquantised matrix products grouped by expert and their gradients, over the
// sorted pairs of a routed batch:
//   forward  out[s] = W[e] a_s,   dgrad  da[s] = W[e]^T dy[s],
//   wgrad    dW[e]  = base[e] + sum_s dy[s] a_s^T.
//
// One 16 x 16 output tile per block, operands staged through shared memory.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

enum Pass { kForward = 0, kDgrad = 1, kWgrad = 2 };
constexpr int kT = 16;

struct GemmParams {
    const void *a, *w, *dy;
    const int32_t *offsets, *sorted_tok;
    const void *base;
    void *out;
    int T, P, E, N, K;
    int32_t *status;
};

// Rows of expert e, empty (and flagged) where the table is out of bounds.
__device__ __forceinline__ int2 expert_range(const GemmParams &p, int e) {
    const int r0 = p.offsets[e], r1 = p.offsets[e + 1];
    if (r0 < 0 || r1 < r0 || r1 > p.P) {
        flag(p.status, MOE_DEV_BAD_INDEX);
        return make_int2(0, 0);
    }
    return make_int2(r0, r1);
}

// Row of a for sorted pair s, -1 if its token is out of bounds.
__device__ __forceinline__ int row_of(const GemmParams &p, int s) {
    if (!p.sorted_tok) return s;
    const int t = p.sorted_tok[s];
    if (t >= 0 && t < p.T) return t;
    flag(p.status, MOE_DEV_BAD_INDEX);
    return -1;
}

// Forward and dgrad: block (x: column tile, y: expert), walking its row tiles.
// Forward: columns n, inner k, weight W[n][k]; dgrad: columns k, inner n.
template <typename I, typename O, int PASS>
__global__ void __launch_bounds__(kT *kT) rows_kernel(const GemmParams p) {
    __shared__ float sa[kT][kT + 1], sw[kT][kT + 1];
    const int e = blockIdx.y, tx = threadIdx.x, ty = threadIdx.y;
    const int cols = PASS == kForward ? p.N : p.K, inner = PASS == kForward ? p.K : p.N;
    const int c0 = blockIdx.x * kT;
    const I *W = static_cast<const I *>(p.w) + int64_t(e) * p.N * p.K;
    const I *A = static_cast<const I *>(PASS == kForward ? p.a : p.dy);
    const int2 r = expert_range(p, e);
    for (int s0 = r.x; s0 < r.y; s0 += kT) {
        const int row = s0 + ty < r.y ? (PASS == kForward ? row_of(p, s0 + ty) : s0 + ty) : -1;
        float acc = 0.f;
        for (int i0 = 0; i0 < inner; i0 += kT) {
            sa[ty][tx] = row >= 0 && i0 + tx < inner ? to_f32(A[int64_t(row) * inner + i0 + tx]) : 0.f;
            if (PASS == kForward)  // sw[column][inner]
                sw[ty][tx] = c0 + ty < cols && i0 + tx < inner ? to_f32(W[int64_t(c0 + ty) * p.K + i0 + tx]) : 0.f;
            else                   // W[n][k]: inner n is the slow index
                sw[tx][ty] = c0 + tx < cols && i0 + ty < inner ? to_f32(W[int64_t(i0 + ty) * p.K + c0 + tx]) : 0.f;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kT; ++i) acc = fmaf(sa[ty][i], sw[tx][i], acc);
            __syncthreads();
        }
        if (s0 + ty < r.y && c0 + tx < cols)
            static_cast<O *>(p.out)[int64_t(s0 + ty) * cols + c0 + tx] = from_f32<O>(acc);
    }
}

template <typename I, typename O>
__global__ void __launch_bounds__(kT *kT) wgrad_kernel(const GemmParams p) {
    __shared__ float sa[kT][kT + 1], sd[kT][kT + 1];
    const int e = blockIdx.z, tx = threadIdx.x, ty = threadIdx.y;
    const int k = blockIdx.x * kT + tx, n0 = blockIdx.y * kT;
    const int2 r = expert_range(p, e);
    float acc = 0.f;
    for (int s0 = r.x; s0 < r.y; s0 += kT) {
        const int row = s0 + ty < r.y ? row_of(p, s0 + ty) : -1;
        sa[ty][tx] = row >= 0 && k < p.K ? to_f32(static_cast<const I *>(p.a)[int64_t(row) * p.K + k]) : 0.f;
        sd[ty][tx] = s0 + ty < r.y && n0 + tx < p.N
                         ? to_f32(static_cast<const I *>(p.dy)[int64_t(s0 + ty) * p.N + n0 + tx]) : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kT; ++i) acc = fmaf(sd[i][ty], sa[i][tx], acc);
        __syncthreads();
    }
    if (k < p.K && n0 + ty < p.N) {
        const int64_t at = (int64_t(e) * p.N + n0 + ty) * p.K + k;
        if (p.base) acc += to_f32(static_cast<const O *>(p.base)[at]);
        static_cast<O *>(p.out)[at] = from_f32<O>(acc);
    }
}

template <typename I, typename O>
void launch(int pass, const GemmParams &p, cudaStream_t stream) {
    const dim3 block(kT, kT);
    if (pass == kForward)
        rows_kernel<I, O, kForward><<<dim3((p.N + kT - 1) / kT, p.E), block, 0, stream>>>(p);
    else if (pass == kDgrad)
        rows_kernel<I, O, kDgrad><<<dim3((p.K + kT - 1) / kT, p.E), block, 0, stream>>>(p);
    else
        wgrad_kernel<I, O><<<dim3((p.K + kT - 1) / kT, (p.N + kT - 1) / kT, p.E), block, 0, stream>>>(p);
}

moe_status run_gemm(int pass, const GemmParams &p, int dtype, int out_dtype, cudaStream_t stream) {
    if (dtype == MOE_BF16) {
        if (out_dtype == MOE_FP32) launch<__nv_bfloat16, float>(pass, p, stream);
        else launch<__nv_bfloat16, __nv_bfloat16>(pass, p, stream);
    } else {
        if (out_dtype == MOE_FP32) launch<__half, float>(pass, p, stream);
        else launch<__half, __half>(pass, p, stream);
    }
    return launch_status();
}

moe_status check_gemm(int dtype, int T, int E, int k, int N, int K, int out_dtype) {
    if (T < 0 || E <= 0 || k <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (!half_type(dtype) || !out_type_ok(dtype, out_dtype)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED;
    if (N % 8 || K % 8 || N > 2 * kMaxDim || K > 2 * kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (int64_t(T) * k >= (int64_t(1) << 31)) return MOE_ERR_OVERFLOW;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_expert_gemm(const void *a, const void *W, int dtype, int T, int E, int k, int N, int K,
                                   const int32_t *offsets, const int32_t *sorted_tok, void *out, int out_dtype,
                                   int32_t *dev_status, moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK || T == 0) return st;
    if (!a || !W || !offsets || !out || !aligned16(a) || !aligned16(W) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    const GemmParams p = {a, W, nullptr, offsets, sorted_tok, nullptr, out, T, T * k, E, N, K, dev_status};
    return run_gemm(kForward, p, dtype, out_dtype, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_dgrad(const void *dy, const void *W, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, void *da, int out_dtype, int32_t *dev_status,
                                         moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK || T == 0) return st;
    if (!dy || !W || !offsets || !da || !aligned16(dy) || !aligned16(W) || !aligned16(da)) return MOE_ERR_INVALID_ARG;
    const GemmParams p = {nullptr, W, dy, offsets, nullptr, nullptr, da, T, T * k, E, N, K, dev_status};
    return run_gemm(kDgrad, p, dtype, out_dtype, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_wgrad(const void *dy, const void *a, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, const int32_t *sorted_tok, const void *base,
                                         void *dW, int out_dtype, int32_t *dev_status, moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK) return st;
    if (!offsets || !dW || !aligned16(dW) || !aligned16(base)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !a || !aligned16(dy) || !aligned16(a))) return MOE_ERR_INVALID_ARG;
    const GemmParams p = {a, nullptr, dy, offsets, sorted_tok, base, dW, T, T * k, E, N, K, dev_status};
    return run_gemm(kWgrad, p, dtype, out_dtype, as_cuda(stream));
}
