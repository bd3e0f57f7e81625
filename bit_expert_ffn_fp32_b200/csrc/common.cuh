// Internal helpers shared by the libmoe CUDA sources.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

constexpr int kMaxE = 4096;
constexpr int kMaxK = 16;
constexpr int kMaxDim = 8192;
// Pairs of the 4-bit and the unquantised products: row numbers rounded up to a tile stay in 32 bits.
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - 4096;

inline cudaStream_t as_cuda(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Reports a rejected launch without clearing sticky errors of other work.
inline moe_status launch_status() {
    cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

// A launch that may be set up while the work before it on the stream still runs
// (kernels that begin with after_previous()); shared by the calls that follow
// one another in decoding, where a launch is a good part of the time.
inline cudaError_t launch_early(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attrs)[2], int clusters, const void *fn,
                                void **args) {
    int n = 0;
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n++].val.programmaticStreamSerializationAllowed = 1;
    if (clusters > 1) {
        attrs[n].id = cudaLaunchAttributeClusterDimension;
        attrs[n].val.clusterDim.x = clusters;
        attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelExC(&cfg, fn, args);
}
// Dynamic shared memory a launch of fn may ask for: always the template's
// largest amount, so that calls of several host threads set the same value and
// none lowers it between another's set and launch. Set on every call, as it
// belongs to the current device's context.
template <typename F>
inline bool allow_smem(F *fn, int most) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}
constexpr int kMaxSmem = 232448;  // of a block, its static shared memory included
// First thing in such a kernel, by every thread: from here on everything before
// it on the stream is done and visible; what follows it may be set up as well.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void flag(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// The two 16-bit element types and fp32 behind one name.
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

inline bool half_type(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16; }
inline bool out_type_ok(int dtype, int out_dtype) { return out_dtype == dtype || out_dtype == MOE_FP32; }
inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline bool dims_ok(int d, int f) {
    return d > 0 && f > 0 && d % 256 == 0 && f % 256 == 0 && d <= kMaxDim && f <= kMaxDim;
}

// Prefill path (ffn_tc05.cu): grouped tcgen05 GEMMs for Q2 or Q3 experts. Used
// by moe_expert_ffn_q2/q3 when T*k >= kTcMinPairs; the caller has validated
// arguments.
constexpr int kTcMinPairs = 512;
constexpr int kTcMaxE = 1024;
// Byte offset of the permuted fp16 activations (fp16 [T*k][d]) inside the
// tensor-core path's workspace (after h, fp16 [T*k][f], rounded up to 256 B).
inline size_t tc05_xperm_offset(int T, int k, int f) {
    return (size_t(T) * size_t(k) * size_t(f) * 2 + 255) & ~size_t(255);
}
moe_status tc05_ffn(int fmt, const moe_qpool *W, const int32_t *slot_of, const uint16_t *x, int T, int d, int f, int E,
                    int k, const int32_t *offsets, const int32_t *sorted_tok, const int32_t *sorted_j,
                    const int32_t *active, const float *topk_w, float *out, void *ws, int32_t *dev_status,
                    cudaStream_t stream);

}  // namespace moe
