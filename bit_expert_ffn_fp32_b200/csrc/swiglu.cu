// The activation between the gate/up and the down product of an unquantised
// expert, and its gradient:
//   h = silu(g) * u,  dg = dh * u * sig(g) * (1 + g * (1 - sig(g))),  du = dh * silu(g)
// elementwise in fp32 from 16-bit tensors, rounded once.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

template <typename E>
__global__ void swiglu_kernel(const E *__restrict__ gu, int64_t n, int f, E *__restrict__ h) {
    for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / f, c = i - r * f;
        const float g = to_f32(gu[r * 2 * f + c]), u = to_f32(gu[r * 2 * f + f + c]);
        h[i] = from_f32<E>(g / (1.0f + expf(-g)) * u);
    }
}

template <typename E>
__global__ void swiglu_backward_kernel(const E *gu, const E *__restrict__ dh, int64_t n, int f, E *dgu) {
    for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / f, c = i - r * f;
        const float g = to_f32(gu[r * 2 * f + c]), u = to_f32(gu[r * 2 * f + f + c]), d = to_f32(dh[i]);
        const float sig = 1.0f / (1.0f + expf(-g));
        dgu[r * 2 * f + c] = from_f32<E>(d * u * sig * (1.0f + g * (1.0f - sig)));
        dgu[r * 2 * f + f + c] = from_f32<E>(d * g * sig);
    }
}

moe_status check_swiglu(int dtype, int64_t rows, int f) {
    if (rows < 0 || f <= 0 || !half_type(dtype)) return MOE_ERR_INVALID_ARG;
    if (f % 8 || f > 2 * kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (rows >= (int64_t(1) << 31)) return MOE_ERR_OVERFLOW;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_swiglu(const void *gu, int dtype, int64_t rows, int f, void *h, moe_stream_t stream) {
    const moe_status st = check_swiglu(dtype, rows, f);
    if (st != MOE_OK || rows == 0) return st;
    if (!gu || !h || !aligned16(gu) || !aligned16(h)) return MOE_ERR_INVALID_ARG;
    const int64_t n = rows * f;
    const int grid = int(std::min<int64_t>((n + 255) / 256, 148 * 16));
    if (dtype == MOE_BF16)
        swiglu_kernel<<<grid, 256, 0, as_cuda(stream)>>>(static_cast<const __nv_bfloat16 *>(gu), n, f,
                                                         static_cast<__nv_bfloat16 *>(h));
    else
        swiglu_kernel<<<grid, 256, 0, as_cuda(stream)>>>(static_cast<const __half *>(gu), n, f,
                                                         static_cast<__half *>(h));
    return launch_status();
}

MOE_API moe_status moe_swiglu_backward(const void *gu, const void *dh, int dtype, int64_t rows, int f, void *dgu,
                                       moe_stream_t stream) {
    const moe_status st = check_swiglu(dtype, rows, f);
    if (st != MOE_OK || rows == 0) return st;
    if (!gu || !dh || !dgu || !aligned16(gu) || !aligned16(dh) || !aligned16(dgu)) return MOE_ERR_INVALID_ARG;
    const int64_t n = rows * f;
    const int grid = int(std::min<int64_t>((n + 255) / 256, 148 * 16));
    if (dtype == MOE_BF16)
        swiglu_backward_kernel<<<grid, 256, 0, as_cuda(stream)>>>(
            static_cast<const __nv_bfloat16 *>(gu), static_cast<const __nv_bfloat16 *>(dh), n, f,
            static_cast<__nv_bfloat16 *>(dgu));
    else
        swiglu_backward_kernel<<<grid, 256, 0, as_cuda(stream)>>>(static_cast<const __half *>(gu),
                                                                  static_cast<const __half *>(dh), n, f,
                                                                  static_cast<__half *>(dgu));
    return launch_status();
}
