// Products with 4-bit weights and group scales: out[s] = W[slot] x_s, dense or
// grouped by expert, w = s*q + m or s*(q-8).
//
// One warp per weight row (with SwiGLU: a gate row and its up row) and expert,
// the expert's rows one after another.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

struct Q4Params {
    const uint8_t *codes;
    const __half *scale, *min;
    int num_slots, N, K, group;
    const int32_t *slot_of;  // NULL: one matrix, slot `slot`, rows 0..T
    int slot;
    const void *x;
    int T, E, P;
    const int32_t *offsets, *sorted_tok, *active;
    void *out;
    int32_t *status;
};

template <typename X>
__device__ float row_dot(const Q4Params &p, int64_t row, const X *x, int lane) {
    const uint8_t *c = p.codes + row * (p.K / 2);
    const __half *sc = p.scale + row * (p.K / p.group);
    const __half *mn = p.min ? p.min + row * (p.K / p.group) : nullptr;
    float acc = 0.f;
    for (int b = lane; b < p.K / 2; b += 32) {
        const int g = 2 * b / p.group;
        const float s = __half2float(sc[g]), m = mn ? __half2float(mn[g]) : -8.0f * s;
        acc = fmaf(fmaf(s, float(c[b] & 15), m), to_f32(x[2 * b]), acc);
        acc = fmaf(fmaf(s, float(c[b] >> 4), m), to_f32(x[2 * b + 1]), acc);
    }
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

// grid.y: active experts (or 1); 8 warps of a block: 8 output columns.
template <typename X, typename O, bool SWIGLU>
__global__ void __launch_bounds__(256) q4_kernel(const Q4Params p) {
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int cols = SWIGLU ? p.N / 2 : p.N;
    int slot = p.slot, r0 = 0, r1 = p.T;
    if (p.slot_of) {
        const int na = p.active[0];
        if (blockIdx.x == 0 && blockIdx.y == 0 && (na < 0 || na > p.E)) flag(p.status, MOE_DEV_BAD_INDEX);
        if (int(blockIdx.y) >= na) return;
        const int e = p.active[1 + blockIdx.y];
        if (e < 0 || e >= p.E) return flag(p.status, MOE_DEV_BAD_INDEX);
        slot = p.slot_of[e];
        if (slot < 0 || slot >= p.num_slots) {
            if (slot != -1) flag(p.status, MOE_DEV_BAD_SLOT);
            return;
        }
        r0 = p.offsets[e], r1 = p.offsets[e + 1];
        if (r0 < 0 || r1 < r0 || r1 > p.P) return flag(p.status, MOE_DEV_BAD_INDEX);
    }
    if (n >= cols) return;
    for (int s = r0; s < r1; ++s) {
        int t = s;
        if (p.slot_of && p.sorted_tok) t = p.sorted_tok[s];
        const bool ok = !(p.slot_of && p.sorted_tok) || (t >= 0 && t < p.T);
        float y = 0.f, u = 0.f;
        if (ok) {
            const X *x = static_cast<const X *>(p.x) + int64_t(t) * p.K;
            y = row_dot(p, int64_t(slot) * p.N + n, x, lane);
            if (SWIGLU) u = row_dot(p, int64_t(slot) * p.N + cols + n, x, lane);
        } else {
            flag(p.status, MOE_DEV_BAD_INDEX);
        }
        if (SWIGLU) y = y / (1.0f + expf(-y)) * u;
        if (lane == 0) static_cast<O *>(p.out)[int64_t(s) * cols + n] = from_f32<O>(y);
    }
}

template <typename X, typename O>
void launch(const Q4Params &p, int act, dim3 grid, cudaStream_t stream) {
    if (act == MOE_ACT_SWIGLU)
        q4_kernel<X, O, true><<<grid, 256, 0, stream>>>(p);
    else
        q4_kernel<X, O, false><<<grid, 256, 0, stream>>>(p);
}

moe_status run_q4(const moe_q4weights *W, Q4Params &p, const void *x, int dtype, int act, void *out, int out_dtype,
                  int experts, cudaStream_t stream) {
    p.codes = W->codes;
    p.scale = reinterpret_cast<const __half *>(W->scale);
    p.min = reinterpret_cast<const __half *>(W->min);
    p.num_slots = W->num_slots;
    p.N = W->N;
    p.K = W->K;
    p.group = W->group;
    p.x = x;
    p.out = out;
    const dim3 grid((p.N / (act == MOE_ACT_SWIGLU ? 2 : 1) + 7) / 8, experts);
    if (dtype == MOE_BF16) {
        if (out_dtype == MOE_FP32) launch<__nv_bfloat16, float>(p, act, grid, stream);
        else launch<__nv_bfloat16, __nv_bfloat16>(p, act, grid, stream);
    } else {
        if (out_dtype == MOE_FP32) launch<__half, float>(p, act, grid, stream);
        else launch<__half, __half>(p, act, grid, stream);
    }
    return launch_status();
}

moe_status check_q4(const moe_q4weights *W, int dtype, int act, int out_dtype) {
    if (!W || !half_type(dtype) || !out_type_ok(dtype, out_dtype)) return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
    if (W->num_slots <= 0 || W->N <= 0 || W->K <= 0) return MOE_ERR_INVALID_ARG;
    if (W->group != 32 && W->group != 64 && W->group != 128) return MOE_ERR_UNSUPPORTED;
    if (W->N % 32 || W->K % W->group || W->N > 2 * kMaxDim || W->K > 2 * kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (!W->codes || !W->scale || !aligned16(W->codes)) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(W->scale) % 2 || reinterpret_cast<uintptr_t>(W->min) % 2)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_linear_q4(const moe_q4weights *W, int32_t slot, const void *x, int dtype, int T, int act,
                                 void *out, int out_dtype, moe_stream_t stream) {
    const moe_status st = check_q4(W, dtype, act, out_dtype);
    if (st != MOE_OK) return st;
    if (T < 0 || slot < 0 || slot >= W->num_slots) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !out || !aligned16(x) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    Q4Params p = {};
    p.slot = slot;
    p.T = p.P = T;
    p.E = 1;
    return run_q4(W, p, x, dtype, act, out, out_dtype, 1, as_cuda(stream));
}

MOE_API moe_status moe_expert_linear_q4(const moe_q4weights *W, const int32_t *slot_of, const void *x, int dtype,
                                        int T, int E, int k, const int32_t *offsets, const int32_t *sorted_tok,
                                        const int32_t *active, int act, void *out, int out_dtype, int32_t *dev_status,
                                        moe_stream_t stream) {
    const moe_status st = check_q4(W, dtype, act, out_dtype);
    if (st != MOE_OK) return st;
    if (T < 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED;
    if (int64_t(T) * k >= (int64_t(1) << 31)) return MOE_ERR_OVERFLOW;
    if (T == 0) return MOE_OK;
    if (!slot_of || !x || !offsets || !active || !out || !aligned16(x) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    Q4Params p = {};
    p.slot_of = slot_of;
    p.T = T;
    p.E = E;
    p.P = T * k;
    p.offsets = offsets;
    p.sorted_tok = sorted_tok;
    p.active = active;
    p.status = dev_status;
    return run_q4(W, p, x, dtype, act, out, out_dtype, int(std::min<int64_t>(E, int64_t(T) * k)), as_cuda(stream));
}
