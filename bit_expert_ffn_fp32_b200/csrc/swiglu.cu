// The activation between the gate/up and the down product of an unquantised
// expert, and its gradient:
//   h = silu(g) * u,  dg = dh * u * sig(g) * (1 + g * (1 - sig(g))),  du = dh * silu(g)
// elementwise in fp32 from 16-bit tensors, rounded once.
//
// Bound by memory: 6 bytes an element forward, 10 backward. A thread takes two
// chunks of 8 elements (16-byte loads of every operand, all issued before the
// first is used), a block 512 chunks in a row; blocks are not persistent, so
// the loads of one cover the stores of another. sig(g) is formed with the
// hardware's exp2 and reciprocal: off by about 2^-19 + |g| 2^-23, at most 2^-16,
// against half a step of 2^-11 (fp16, whose products vanish long before) or 2^-8
// in the result; backward, gates below -87.3 add a subnormal's 2^-150 to sig(g).
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kChunks = 2, kTile = kThreads * kChunks;

template <typename E>
struct Pack2;
template <>
struct Pack2<__nv_bfloat16> {
    static __device__ float2 load(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
    static __device__ uint32_t store(float a, float b) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};
template <>
struct Pack2<__half> {
    static __device__ float2 load(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
    static __device__ uint32_t store(float a, float b) {
        const __half2 r = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// The hardware's exp2 and reciprocal, results below 2^-126 as zeros.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// sig(g) = 1 / (1 + exp(-g)) without an overflow on the way, so that a far gate
// keeps its share of a large product down to g = -103.97, where sig(g) passes
// below fp32's smallest subnormal (2^-149) and the result is zero.
// Forward: g sig(g) u as ((u 2^-16) (2^16 sig(g))) g, with
//   2^16 sig(g) = 2^-8 (1 / (2^-24 + 2^(-g log2 e - 24))).
// The reciprocal stays above 2^-126 as long as the result is not zero, 2^16
// sig(g) keeps 15 bits at the far end, and u 2^-16 is exact, for subnormal u too
// (0.45 us more at 81,920 x 768 than g sig(g) u unscaled).
__device__ __forceinline__ float gated(float g, float u) {
    const float r = rcp_approx(0x1p-24f + exp2_approx(fmaf(g, -1.4426950408889634f, -24.f)));
    return u * 0x1p-16f * (r * 0x1p-8f) * g;
}
// Backward: for g < 0 as exp(g) / (1 + exp(g)). Below g = -87.3 exp(g) is a
// subnormal, off by up to 2^-150.
__device__ __forceinline__ float sigmoid(float g) {
    const float e = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
    return g < 0.f ? e * r : r;
}

// Chunk i of this block's tile: its row, and its first element in the row.
// chunks_of_row = f / 8; div = ceil(2^32 / chunks_of_row) divides the small
// numbers that are left inside a tile exactly.
struct Where {
    int64_t row;
    int col;
    bool in;
};
__device__ __forceinline__ Where where(int64_t row0, uint32_t chunk0, uint32_t i, uint32_t chunks_of_row, uint32_t div,
                                       int64_t left) {
    const uint32_t c = chunk0 + i;
    const uint32_t q = chunks_of_row == 1 ? c : __umulhi(c, div);
    return {row0 + q, int(c - q * chunks_of_row) * 8, int64_t(i) < left};
}

// Blocks an SM are held to what the loads in flight need: forward 8 (32 registers;
// with 37, hence 6 blocks, 1.0 us more at 81,920 x 768), backward 5.
template <typename E, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, BACKWARD ? 5 : 8)
    swiglu_kernel(const E *gu, const E *__restrict__ dh, int64_t chunks, int f, uint32_t div, E *out) {
    after_previous();
    const uint32_t cr = uint32_t(f) / 8;
    const int64_t first = int64_t(blockIdx.x) * kTile, row0 = first / cr;
    const uint32_t chunk0 = uint32_t(first - row0 * cr);
    uint4 g[kChunks], u[kChunks], d[kChunks];
    Where w[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        w[j] = where(row0, chunk0, j * kThreads + threadIdx.x, cr, div, chunks - first);
        if (w[j].in) {
            const E *r = gu + w[j].row * 2 * f + w[j].col;
            g[j] = *reinterpret_cast<const uint4 *>(r);
            u[j] = *reinterpret_cast<const uint4 *>(r + f);
            if (BACKWARD) d[j] = __ldg(reinterpret_cast<const uint4 *>(dh + w[j].row * f + w[j].col));
        }
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        if (!w[j].in) continue;
        const uint32_t gv[4] = {g[j].x, g[j].y, g[j].z, g[j].w}, uv[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        uint32_t a[4], b[4];
        if (!BACKWARD) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 gf = Pack2<E>::load(gv[i]), uf = Pack2<E>::load(uv[i]);
                a[i] = Pack2<E>::store(gated(gf.x, uf.x), gated(gf.y, uf.y));
            }
            *reinterpret_cast<uint4 *>(out + w[j].row * f + w[j].col) = make_uint4(a[0], a[1], a[2], a[3]);
        } else {
            const uint32_t dv[4] = {d[j].x, d[j].y, d[j].z, d[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 gf = Pack2<E>::load(gv[i]), uf = Pack2<E>::load(uv[i]), df = Pack2<E>::load(dv[i]);
                const float sx = sigmoid(gf.x), sy = sigmoid(gf.y);
                a[i] = Pack2<E>::store(df.x * uf.x * sx * (1.0f + gf.x * (1.0f - sx)),
                                       df.y * uf.y * sy * (1.0f + gf.y * (1.0f - sy)));
                b[i] = Pack2<E>::store(df.x * gf.x * sx, df.y * gf.y * sy);
            }
            E *r = out + w[j].row * 2 * f + w[j].col;
            *reinterpret_cast<uint4 *>(r) = make_uint4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint4 *>(r + f) = make_uint4(b[0], b[1], b[2], b[3]);
        }
    }
}

template <typename E, bool BACKWARD>
moe_status launch(const void *gu, const void *dh, int64_t rows, int f, void *out, cudaStream_t stream) {
    const int64_t chunks = rows * (f / 8), blocks = (chunks + kTile - 1) / kTile;
    if (blocks >= (int64_t(1) << 31)) return MOE_ERR_OVERFLOW;
    const uint64_t cr = uint64_t(f) / 8;
    uint32_t div = uint32_t(((uint64_t(1) << 32) + cr - 1) / cr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    int64_t n = chunks;
    void *args[] = {&gu, &dh, &n, &f, &div, &out};
    if (launch_early(cfg, attrs, 1, reinterpret_cast<const void *>(swiglu_kernel<E, BACKWARD>), args) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
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
    return dtype == MOE_BF16 ? launch<__nv_bfloat16, false>(gu, nullptr, rows, f, h, as_cuda(stream))
                             : launch<__half, false>(gu, nullptr, rows, f, h, as_cuda(stream));
}

MOE_API moe_status moe_swiglu_backward(const void *gu, const void *dh, int dtype, int64_t rows, int f, void *dgu,
                                       moe_stream_t stream) {
    const moe_status st = check_swiglu(dtype, rows, f);
    if (st != MOE_OK || rows == 0) return st;
    if (!gu || !dh || !dgu || !aligned16(gu) || !aligned16(dh) || !aligned16(dgu)) return MOE_ERR_INVALID_ARG;
    return dtype == MOE_BF16 ? launch<__nv_bfloat16, true>(gu, dh, rows, f, dgu, as_cuda(stream))
                             : launch<__half, true>(gu, dh, rows, f, dgu, as_cuda(stream));
}
