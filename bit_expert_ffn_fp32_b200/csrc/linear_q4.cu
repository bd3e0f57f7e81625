// Products with 4-bit weights and group scales: out[s] = W[slot] x_s, dense or
// grouped by expert, w = s*q + m or s*(q-8), for few rows a matrix.
//
// Bound by the weights' bytes, so every warp streams codes through its own
// ring in shared memory (cp.async, kDepth steps of 128 k in flight) and nothing
// else waits on memory: a warp owns 16 or 32 weight rows and every KS-th step
// of k, the KS warps of the same rows add their sums in a fixed order at the
// end. Products run on the tensor cores (mma.m16n8k16, weights as the 16 rows,
// 8 tokens as the columns): a code q becomes the 16-bit float 16 + q by one
// shift and one logic operation (q in the top mantissa bits of 16.0), exact in
// bf16 and fp16, so no weight is rounded and x needs no conversion. The shift
// comes off a group at a time in fp32:
//   sum_k w x = s * sum (16 + q) x + (m - 16 s) * sum x      (m = -8 s without min)
// with sum x from one more mma whose weights are all 1.
#include <algorithm>

#include "common.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 128;   // k of one ring step: 64 bytes of codes a row
constexpr int kDepth = 4;    // steps in flight

struct Q4Params {
    const uint8_t *codes;
    const __half *scale, *min;
    int num_slots, N, K;
    const int32_t *slot_of;  // NULL: one matrix, slot `slot`, rows 0..T
    int slot;
    const void *x;
    int T, E, P;
    const int32_t *offsets, *sorted_tok, *active;
    void *out;
    int out_fp32, swiglu;
    int ks_log2;             // warps that share the same rows, log2
    int scales_in_words;     // a step's scales of a row can be read as one aligned word
    int32_t *status;
};

template <typename X>
struct Codes16;  // 16 + q as X, two at a time: nibbles j and j + 4 of a code word
template <>
struct Codes16<__nv_bfloat16> {
    template <int J>
    static __device__ __forceinline__ uint32_t at(uint32_t w) {
        constexpr int sh = 4 * J - 3;  // nibble j to bits 3..6
        return ((sh < 0 ? w << (sh < 0 ? -sh : 0) : w >> (sh < 0 ? 0 : sh)) & 0x00780078u) | 0x41804180u;
    }
    static constexpr uint32_t kOnes = 0x3F803F80u;
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <>
struct Codes16<__half> {
    template <int J>
    static __device__ __forceinline__ uint32_t at(uint32_t w) {
        constexpr int sh = 4 * J - 6;  // nibble j to bits 6..9
        return ((sh < 0 ? w << (sh < 0 ? -sh : 0) : w >> (sh < 0 ? 0 : sh)) & 0x03C003C0u) | 0x4C004C00u;
    }
    static constexpr uint32_t kOnes = 0x3C003C00u;
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Bytes from one weight row to the next in a ring step: 64 of codes, padded so
// that the fragment reads (4, 8 or 16 bytes a lane) fall into different banks.
template <int G>
constexpr int kRowStride = G == 32 ? 80 : G == 64 ? 96 : 64;

template <int G, int RG>
constexpr int ring_bytes() { return kDepth * 16 * RG * kRowStride<G>; }
constexpr int kPartStride = 36;  // floats from one token's 32 partial sums to the next
template <int G, int RG, int NB>
constexpr int warp_smem() {
    return ring_bytes<G, RG>() > NB * 8 * kPartStride * 4 ? ring_bytes<G, RG>() : NB * 8 * kPartStride * 4;
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// The scales (or mins) of one row in one step, 128 / G of them, low first.
template <int G>
__device__ __forceinline__ uint2 load_scales(const __half *row, int first, int count, bool words) {
    uint2 v = make_uint2(0, 0);
    const __half *p = row + first;
    if (words) {
        if (G == 32) v = __ldg(reinterpret_cast<const uint2 *>(p));
        else if (G == 64) v.x = __ldg(reinterpret_cast<const uint32_t *>(p));
        else v.x = __ldg(reinterpret_cast<const unsigned short *>(p));
        return v;
    }
    const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
    if (first < count) v.x = __ldg(h);
    if (G <= 64 && first + 1 < count) v.x |= uint32_t(__ldg(h + 1)) << 16;
    if (G == 32 && first + 2 < count) v.y = __ldg(h + 2);
    if (G == 32 && first + 3 < count) v.y |= uint32_t(__ldg(h + 3)) << 16;
    return v;
}

__device__ __forceinline__ float half_at(uint2 v, int j) {
    const uint32_t w = j < 2 ? v.x : v.y;
    return __half2float(__ushort_as_half(static_cast<unsigned short>(j & 1 ? w >> 16 : w & 0xFFFF)));
}

// Grid: (row blocks, active experts or 1). X: type of x; G: group; RG: 16-row
// groups a warp owns (2: 32 rows, or with SwiGLU 16 gate rows and their 16 up
// rows); NB: tiles of 8 tokens whose sums a warp keeps.
template <typename X, int G, int RG, int NB>
__global__ void __launch_bounds__(32 * kWarps, NB == 1 ? 3 : 2) q4_kernel(const __grid_constant__ Q4Params p) {
    constexpr int R = 16 * RG, RS = kRowStride<G>, W = G / 32, J = kStep / G;
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = 1 << p.ks_log2, ks = warp & (KS - 1);
    const int units = (p.swiglu ? p.N / 2 : p.N) / (p.swiglu ? 16 : R);
    const int unit0 = blockIdx.x * (kWarps >> p.ks_log2), unit = unit0 + (warp >> p.ks_log2);

    int slot = p.slot, r0 = 0, r1 = p.T;
    if (p.slot_of) {
        const int na = p.active[0];
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && (na < 0 || na > p.E))
            flag(p.status, MOE_DEV_BAD_INDEX);
        if (int(blockIdx.y) >= na) return;
        const int e = p.active[1 + blockIdx.y];
        if (e < 0 || e >= p.E) {
            if (threadIdx.x == 0) flag(p.status, MOE_DEV_BAD_INDEX);
            return;
        }
        slot = p.slot_of[e];
        r0 = p.offsets[e];
        r1 = p.offsets[e + 1];
        if (slot < 0 || slot >= p.num_slots) {
            if (slot != -1 && threadIdx.x == 0) flag(p.status, MOE_DEV_BAD_SLOT);
            return;
        }
        if (r0 < 0 || r1 < r0 || r1 > p.P) {
            if (threadIdx.x == 0) flag(p.status, MOE_DEV_BAD_INDEX);
            return;
        }
    }
    // weight row i of this warp's unit
    auto weight_row = [&](int i) {
        return p.swiglu ? (i < 16 ? unit * 16 + i : p.N / 2 + unit * 16 + i - 16) : unit * R + i;
    };
    const bool busy = unit < units;
    const int steps = (p.K + kStep - 1) / kStep, groups = p.K / G;
    const int64_t slot_row = int64_t(slot) * p.N;
    const uint32_t ring = tc::smem_u32(smem) + warp * warp_smem<G, RG, NB>();
    const unsigned char *ring_ptr = smem + warp * warp_smem<G, RG, NB>();
    // this lane's 16-byte parts of a step: part t of rows g + 8i
    const uint8_t *src = p.codes + (slot_row + (busy ? weight_row(g) : 0)) * (p.K / 2) + 16 * t;
    const int64_t up8 = int64_t(8) * (p.K / 2), up16 = p.swiglu ? int64_t(p.N / 2) * (p.K / 2) : 2 * up8;
    const uint32_t dst = ring + g * RS + 16 * t;
    const __half *srow = nullptr, *mrow = nullptr;  // scales of row `lane`
    {
        const int64_t row = slot_row + (busy ? weight_row(lane & (R - 1)) : 0);
        srow = p.scale + row * groups;
        mrow = p.min ? p.min + row * groups : nullptr;
    }
    auto issue = [&](int step, int stage) {
        if (busy && step < steps) {
            const bool in = step * kStep + 32 * t < p.K;
            const uint8_t *s = src + int64_t(step) * (kStep / 2);
            const uint32_t d = dst + stage * (R * RS);
#pragma unroll
            for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t *from = s + (rg ? up16 : 0) + (i ? up8 : 0);
                    cp_async16_or_zero(d + (16 * rg + 8 * i) * RS, in ? from : p.codes, in);
                }
        }
        tc::cp_async_commit();
    };
    uint2 sc[kDepth], mn[kDepth];
    auto issue_scales = [&](int step, uint2 &s, uint2 &m) {
        if (busy && step < steps) {
            s = load_scales<G>(srow, step * J, groups, p.scales_in_words);
            if (mrow) m = load_scales<G>(mrow, step * J, groups, p.scales_in_words);
        }
    };

    const uint32_t ones[4] = {Codes16<X>::kOnes, Codes16<X>::kOnes, Codes16<X>::kOnes, Codes16<X>::kOnes};
    for (int pass = r0; pass < r1; pass += 8 * NB) {
        const int n = min(8 * NB, r1 - pass);
        // columns (tokens) of this lane's B fragments: token 8 nb + g
        const X *xrow[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            xrow[nb] = nullptr;
            if (8 * nb + g < n) {
                int row = pass + 8 * nb + g;
                if (p.sorted_tok) {
                    row = p.sorted_tok[row];
                    if (row < 0 || row >= p.T) {
                        if (blockIdx.x == 0 && warp == 0 && t == 0) flag(p.status, MOE_DEV_BAD_INDEX);
                        row = -1;
                    }
                }
                if (row >= 0) xrow[nb] = static_cast<const X *>(p.x) + int64_t(row) * p.K + (G / 4) * t;
            }
        }
        float sum[NB][RG][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[nb][rg][i] = 0.f;
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            sc[d] = mn[d] = make_uint2(0, 0);
            issue(ks + d * KS, d);
            issue_scales(ks + d * KS, sc[d], mn[d]);
        }
        for (int step0 = ks; step0 < steps; step0 += kDepth * KS) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                const int step = step0 + d * KS;
                if (step < steps && busy) {
                    tc::cp_async_wait<kDepth - 1>();
                    __syncwarp();
                    const unsigned char *st = ring_ptr + d * (R * RS) + g * RS + (G / 8) * t;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (step * J + j >= groups) break;
                        uint32_t w[RG][2][W];
#pragma unroll
                        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const unsigned char *from = st + (16 * rg + 8 * i) * RS + j * (G / 2);
                                if (W == 1) w[rg][i][0] = *reinterpret_cast<const uint32_t *>(from);
                                if (W == 2) {
                                    const uint2 v = *reinterpret_cast<const uint2 *>(from);
                                    w[rg][i][0] = v.x;
                                    w[rg][i][W - 1] = v.y;
                                }
                                if (W == 4) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(from);
                                    w[rg][i][0] = v.x;
                                    w[rg][i][W > 1 ? 1 : 0] = v.y;
                                    w[rg][i][W > 2 ? 2 : 0] = v.z;
                                    w[rg][i][W - 1] = v.w;
                                }
                            }
                        float acc[NB][RG + 1][4];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int rg = 0; rg <= RG; ++rg)
#pragma unroll
                                for (int i = 0; i < 4; ++i) acc[nb][rg][i] = 0.f;
#pragma unroll
                        for (int wi = 0; wi < W; ++wi) {
                            uint32_t a[RG][2][4];
#pragma unroll
                            for (int rg = 0; rg < RG; ++rg) {
                                const uint32_t lo = w[rg][0][wi], hi = w[rg][1][wi];
                                a[rg][0][0] = Codes16<X>::template at<0>(lo);
                                a[rg][0][1] = Codes16<X>::template at<0>(hi);
                                a[rg][0][2] = Codes16<X>::template at<1>(lo);
                                a[rg][0][3] = Codes16<X>::template at<1>(hi);
                                a[rg][1][0] = Codes16<X>::template at<2>(lo);
                                a[rg][1][1] = Codes16<X>::template at<2>(hi);
                                a[rg][1][2] = Codes16<X>::template at<3>(lo);
                                a[rg][1][3] = Codes16<X>::template at<3>(hi);
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                if (NB > 1 && 8 * nb >= n) break;
                                uint4 xv = make_uint4(0, 0, 0, 0);  // 8 consecutive k of token g
                                if (xrow[nb])
                                    xv = __ldg(reinterpret_cast<const uint4 *>(xrow[nb] + step * kStep + j * G +
                                                                               8 * wi));
                                // nibbles j and j + 4 share a register of a, so k j and k j + 4 one of b
                                const uint32_t b00 = __byte_perm(xv.x, xv.z, 0x5410),
                                               b01 = __byte_perm(xv.x, xv.z, 0x7632),
                                               b10 = __byte_perm(xv.y, xv.w, 0x5410),
                                               b11 = __byte_perm(xv.y, xv.w, 0x7632);
#pragma unroll
                                for (int rg = 0; rg < RG; ++rg) {
                                    Codes16<X>::mma(acc[nb][rg], a[rg][0], b00, b01);
                                    Codes16<X>::mma(acc[nb][rg], a[rg][1], b10, b11);
                                }
                                Codes16<X>::mma(acc[nb][RG], ones, b00, b01);
                                Codes16<X>::mma(acc[nb][RG], ones, b10, b11);
                            }
                        }
                        // scale of this lane's row, then those of the rows this lane has sums of
                        const float s_own = half_at(sc[d], j);
                        const float c_own = p.min ? fmaf(-16.f, s_own, half_at(mn[d], j)) : -24.f * s_own;
#pragma unroll
                        for (int rg = 0; rg < RG; ++rg) {
                            const float s_lo = __shfl_sync(0xffffffffu, s_own, 16 * rg + g);
                            const float s_hi = __shfl_sync(0xffffffffu, s_own, 16 * rg + 8 + g);
                            const float c_lo = __shfl_sync(0xffffffffu, c_own, 16 * rg + g);
                            const float c_hi = __shfl_sync(0xffffffffu, c_own, 16 * rg + 8 + g);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                if (NB > 1 && 8 * nb >= n) break;
                                float(&y)[4] = sum[nb][rg];
                                const float(&v)[4] = acc[nb][rg];
                                const float x0 = acc[nb][RG][0], x1 = acc[nb][RG][1];
                                y[0] = fmaf(s_lo, v[0], fmaf(c_lo, x0, y[0]));
                                y[1] = fmaf(s_lo, v[1], fmaf(c_lo, x1, y[1]));
                                y[2] = fmaf(s_hi, v[2], fmaf(c_hi, x0, y[2]));
                                y[3] = fmaf(s_hi, v[3], fmaf(c_hi, x1, y[3]));
                            }
                        }
                    }
                    __syncwarp();  // every lane has read the stage before it is refilled
                    issue(step + kDepth * KS, d);
                    issue_scales(step + kDepth * KS, sc[d], mn[d]);
                }
            }
        }
        tc::cp_async_wait<0>();
        __syncthreads();  // the rings are free: partial sums [token][row] take their place
        if (busy) {
            float *part = reinterpret_cast<float *>(smem + warp * warp_smem<G, RG, NB>());
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part[(8 * nb + 2 * t + (i & 1)) * kPartStride + 16 * rg + g + 8 * (i >> 1)] =
                            sum[nb][rg][i];
        }
        __syncthreads();
        // outputs of the block: [token][unit][row of the unit]
        const int per_unit = p.swiglu ? 16 : R, in_block = min(kWarps >> p.ks_log2, units - unit0) * per_unit;
        const int cols = p.swiglu ? p.N / 2 : p.N;
        for (int i = threadIdx.x; i < n * in_block; i += 32 * kWarps) {
            const int tok = i / in_block, c = i - tok * in_block, u = c / per_unit, row = c - u * per_unit;
            const unsigned char *from = smem + (u << p.ks_log2) * warp_smem<G, RG, NB>();
            float y = 0.f, up = 0.f;
            for (int k = 0; k < KS; ++k, from += warp_smem<G, RG, NB>()) {
                const float *part = reinterpret_cast<const float *>(from) + tok * kPartStride;
                y += part[row];
                if (RG == 2 && p.swiglu) up += part[16 + row];
            }
            if (RG == 2 && p.swiglu) y = y / (1.0f + expf(-y)) * up;
            const int64_t at = int64_t(pass + tok) * cols + unit0 * per_unit + c;
            if (p.out_fp32) static_cast<float *>(p.out)[at] = y;
            else static_cast<X *>(p.out)[at] = from_f32<X>(y);
        }
        __syncthreads();  // read before the next pass refills the rings
    }
}

template <typename X, int G, int RG, int NB>
moe_status launch(Q4Params &p, int experts, cudaStream_t stream) {
    constexpr int smem = kWarps * warp_smem<G, RG, NB>();
    static_assert(smem <= 100 * 1024, "two blocks of an SM do not fit");
    // set on every call: the attribute belongs to the current device's context
    if (smem > 48 * 1024 && cudaFuncSetAttribute(q4_kernel<X, G, RG, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int units = p.swiglu ? p.N / 32 : p.N / (16 * RG), per_block = kWarps >> p.ks_log2;
    q4_kernel<X, G, RG, NB><<<dim3((units + per_block - 1) / per_block, experts), 32 * kWarps, smem, stream>>>(p);
    return launch_status();
}

template <typename X, int G>
moe_status launch_g(Q4Params &p, int rg, int nb, int experts, cudaStream_t stream) {
    if (rg == 1)
        return nb == 1 ? launch<X, G, 1, 1>(p, experts, stream)
                       : nb == 2 ? launch<X, G, 1, 2>(p, experts, stream) : launch<X, G, 1, 4>(p, experts, stream);
    return nb == 1 ? launch<X, G, 2, 1>(p, experts, stream)
                   : nb == 2 ? launch<X, G, 2, 2>(p, experts, stream) : launch<X, G, 2, 4>(p, experts, stream);
}

template <typename X>
moe_status launch_x(Q4Params &p, int group, int rg, int nb, int experts, cudaStream_t stream) {
    return group == 32 ? launch_g<X, 32>(p, rg, nb, experts, stream)
                       : group == 64 ? launch_g<X, 64>(p, rg, nb, experts, stream)
                                     : launch_g<X, 128>(p, rg, nb, experts, stream);
}

moe_status run_q4(const moe_q4weights *W, Q4Params &p, const void *x, int dtype, int act, void *out, int out_dtype,
                  int experts, cudaStream_t stream) {
    p.codes = W->codes;
    p.scale = reinterpret_cast<const __half *>(W->scale);
    p.min = reinterpret_cast<const __half *>(W->min);
    p.num_slots = W->num_slots;
    p.N = W->N;
    p.K = W->K;
    p.x = x;
    p.out = out;
    p.out_fp32 = out_dtype == MOE_FP32;
    p.swiglu = act == MOE_ACT_SWIGLU;
    p.scales_in_words = W->K % kStep == 0 && reinterpret_cast<uintptr_t>(W->scale) % 8 == 0 &&
                        reinterpret_cast<uintptr_t>(W->min) % 8 == 0;
    // Enough warps to keep every SM's memory pipe full (16 each): split k over
    // up to the 8 warps of a block, then halve the rows a warp owns.
    constexpr int64_t kWant = 148 * 16;
    const int steps = (p.K + kStep - 1) / kStep;
    int rg = 2, ks = 0;
    const int64_t warps = int64_t(p.N / 32) * experts;
    while (ks < 3 && (warps << ks) < kWant && (2 << ks) <= steps) ++ks;
    if (!p.swiglu && (warps << ks) < kWant) rg = 1;
    p.ks_log2 = ks;
    // Token tiles: as many as the rows a matrix has on average (at most T) fill.
    const int rows = std::min(p.T, 2 * ((p.P + experts - 1) / experts));
    const int nb = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    return dtype == MOE_BF16 ? launch_x<__nv_bfloat16>(p, W->group, rg, nb, experts, stream)
                             : launch_x<__half>(p, W->group, rg, nb, experts, stream);
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
