// Products with 4-bit weights and group scales: out[s] = W[slot] x_s, dense or
// grouped by expert, w = s*q + m or s*(q-8), for few rows a matrix.
//
// Bound by the weights' bytes, so every warp streams codes through its own
// ring in shared memory (cp.async, kDepth steps of 256 k in flight) and nothing
// in the loop waits on global memory: a warp owns 16 or 32 weight rows and every
// KS-th step of k, the KS warps of the same rows add their sums in a fixed order
// at the end; x is staged once a block, in the order the products read it.
// Products run on the tensor cores (mma.m16n8k16, weights as the 16 rows, 8
// tokens as the columns), and what limits them is instructions: 8 codes of a
// word must take few. A code masked where it stands is the fp16 subnormal
// q * 2^-24 (bits 0-3 of a half) or q * 2^-20 (bits 4-7), exactly, so a word
// costs four masks and one shift. Without min the operand is q - 8 itself: one
// half-pair FMA, exact too, makes (q - 8) * 2^-9 or 2^-5 of it. Four instructions
// more a word (8192 x 8192, one token: 12.1 -> 12.6 us; four tokens' down rows
// 18.1 -> 19.2; with 1024 + q and 64 + q and a subtraction 15.0 and 19.5), but q x
// and 8 x apart would cancel: an outlier on a zero weight would take the digits
// of every other product. x enters as fp16: 128 k of a token are scaled
// by a power of two that brings their largest to [2^14, 2^15), and the k of the
// codes at 2^-20 by another 2^-4, to [2^10, 2^11) at most. bf16 and fp16 values
// stay exact down to 2^-24 of the largest (2^-14 of 2^10); below that they are
// off by half a subnormal, 2^-25 of 2^10, under the 2^-24 of the fp32 sums they
// join. No weight is rounded; in fp32, by group and then
// by 128 k:
//   sum_k w x = 2^-e * (s * 2^24 * sum (q 2^-24) (x 2^e) + m * sum x 2^e)   with min
//             = 2^-e * s * 2^9 * sum ((q - 8) 2^-9) (x 2^e)                 without
// An infinity or a NaN in x makes its row's results non-finite, all of them.
#include <algorithm>

#include "common.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 256;   // k of one ring step: 128 bytes of codes a row
constexpr int kDepth = 2;    // steps in flight

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
    int ts_log2;             // tokens a tile of staged x holds, log2 (3 unless a single tile is never full)
    int chunk;               // steps of x staged at a time, a multiple of kDepth << ks_log2
    int scales_in_words;     // a step's scales of a row can be read as one aligned word
    int32_t *status;
};

__device__ __forceinline__ uint32_t fma_halves(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// The four half pairs of a code word as fp16: codes (0, 4) and (2, 6) times
// 2^-24, codes (1, 5) and (3, 7) times 2^-20; without min, the codes less 8,
// times 2^-9 and 2^-5.
template <bool MIN>
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t v = w >> 8;
    h[0] = w & 0x000F000Fu;
    h[1] = w & 0x00F000F0u;
    h[2] = v & 0x000F000Fu;
    h[3] = v & 0x00F000F0u;
    if constexpr (!MIN) {  // times 2^15, less 8
        h[0] = fma_halves(h[0], 0x78007800u, 0xA400A400u);  // -8 * 2^-9
        h[1] = fma_halves(h[1], 0x78007800u, 0xB400B400u);  // -8 * 2^-5
        h[2] = fma_halves(h[2], 0x78007800u, 0xA400A400u);
        h[3] = fma_halves(h[3], 0x78007800u, 0xB400B400u);
    }
}
__device__ __forceinline__ void mma_fp16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A ring step holds 128 bytes of codes a row, 16-byte chunks swizzled so that
// the fragment reads (4, 8 or 16 bytes a lane) fall into different banks.
template <int G>
__device__ __forceinline__ int swizzle(int row) {
    return G == 32 ? row & 7 : G == 64 ? (row & 3) * 2 : (row & 1) * 4;
}
constexpr int kPartStride = 36;  // floats from one token's 32 partial sums to the next
// Per warp: the ring, later the partial sums; then the step's scale pairs.
template <int RG, int NB>
constexpr int kRingBytes = kDepth * 16 * RG * 128 > NB * 8 * kPartStride * 4 ? kDepth * 16 * RG * 128
                                                                           : NB * 8 * kPartStride * 4;
template <int G, int RG, int NB>
constexpr int kWarpBytes = kRingBytes<RG, NB> + (kStep / G) * 16 * RG * 8;

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The scales (or mins) of one row in one step, 256 / G of them, low first.
template <int G>
__device__ __forceinline__ uint4 load_scales(const __half *row, int first, int count, bool words) {
    uint4 v = make_uint4(0, 0, 0, 0);
    const __half *p = row + first;
    if (words) {
        if constexpr (G == 32) v = __ldg(reinterpret_cast<const uint4 *>(p));
        if constexpr (G == 64) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            v.x = u.x, v.y = u.y;
        }
        if constexpr (G == 128) v.x = __ldg(reinterpret_cast<const uint32_t *>(p));
        return v;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kStep / G; ++j)
        if (first + j < count) w[j / 2] |= uint32_t(__ldg(reinterpret_cast<const unsigned short *>(p) + j)) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float half_at(const uint4 &v, int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return __half2float(__ushort_as_half(static_cast<unsigned short>(j & 1 ? w >> 16 : w & 0xFFFF)));
}

// Grid: (row blocks, active experts or 1). X: type of x; G: group; RG: 16-row
// groups a warp owns (2: 32 rows, or with SwiGLU 16 gate rows and their 16 up
// rows); NB: tiles of 8 tokens whose sums a warp keeps; MIN: weights have
// an offset.
template <typename X, int G, int RG, int NB, bool MIN>
__global__ void __launch_bounds__(32 * kWarps, NB == 4 ? 1 : 2) q4_kernel(const __grid_constant__ Q4Params p) {
    after_previous();
    constexpr int R = 16 * RG, W = G / 32, J = kStep / G;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = 1 << p.ks_log2, ks = warp & (KS - 1);
    const int units = (p.swiglu ? p.N / 2 : p.N) / (p.swiglu ? 16 : R);
    const int unit0 = blockIdx.x * (kWarps >> p.ks_log2), unit = unit0 + (warp >> p.ks_log2);

    int slot = p.slot, r0 = 0, r1 = p.T;
    if (p.slot_of) {
        const int na = p.active[0], e = p.active[1 + blockIdx.y];  // E + 1 entries: blockIdx.y < E
        // more experts than there are pairs (or experts at all): entries that no block looks at
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && (na < 0 || na > int(gridDim.y)))
            flag(p.status, MOE_DEV_BAD_INDEX);
        if (int(blockIdx.y) >= na) return;
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
    unsigned char *mine = smem + warp * kWarpBytes<G, RG, NB>;
    const uint32_t ring = tc::smem_u32(mine);
    float4 *pairs = reinterpret_cast<float4 *>(mine + kRingBytes<RG, NB>);  // [J][RG][8]: {s, c} of rows g and g + 8
    // x of a chunk of k, 16 bytes (8 k) of one token each: [tile][step][32 units][tokens], a step's units in the order
    // (group, code word of a lane, lane t); then, with min, the sums of the scaled x:
    // [tile][group][8 tokens]
    const int tile_units = p.chunk * (kStep / 8) << p.ts_log2;
    uint4 *xs = reinterpret_cast<uint4 *>(smem + kWarps * kWarpBytes<G, RG, NB>);
    float *xsum = reinterpret_cast<float *>(xs + NB * tile_units);
    float *xdown = xsum + (MIN ? NB * p.chunk * J * 8 : 0);  // 2^-e: [tile][128 k][8 tokens]
    // this lane's 16-byte parts of a step: parts t and t + 4 of rows g + 8i
    const uint8_t *src[2 * RG];
#pragma unroll
    for (int i = 0; i < 2 * RG; ++i)
        src[i] = p.codes + (slot_row + (busy ? weight_row(g + 8 * i) : 0)) * (p.K / 2) + 16 * t;
    const uint32_t dst = ring + g * 128 + ((t ^ swizzle<G>(g)) << 4);  // rows 8 apart have the same swizzle
    const __half *srow = nullptr, *mrow = nullptr;  // scales of row `lane`
    {
        const int64_t row = slot_row + (busy ? weight_row(lane & (R - 1)) : 0);
        srow = p.scale + row * groups;
        if constexpr (MIN) mrow = p.min + row * groups;
    }
    auto issue = [&](int step, int stage) {
        if (busy && step < steps) {
            const uint32_t d = dst + stage * (R * 128);
            const int64_t at = int64_t(step) * (kStep / 2);
            const int left = p.K - step * kStep;
            if (left >= kStep) {
#pragma unroll
                for (int i = 0; i < 2 * RG; ++i) {
                    cp_async16(d + i * 1024, src[i] + at);
                    cp_async16((d + i * 1024) ^ 64, src[i] + at + 64);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 * RG; ++i) {
                    cp_async16_or_zero(d + i * 1024, 32 * t < left ? src[i] + at : p.codes, 32 * t < left);
                    cp_async16_or_zero((d + i * 1024) ^ 64, 128 + 32 * t < left ? src[i] + at + 64 : p.codes,
                                       128 + 32 * t < left);
                }
            }
        }
        tc::cp_async_commit();
    };
    uint4 sc[kDepth], mn[kDepth];
    auto issue_scales = [&](int step, uint4 &s, uint4 &m) {
        if (busy && step < steps) {
            s = load_scales<G>(srow, step * J, groups, p.scales_in_words);
            if constexpr (MIN) m = load_scales<G>(mrow, step * J, groups, p.scales_in_words);
        }
    };

    const int per_pass = NB == 1 ? 1 << p.ts_log2 : 8 * NB;
    for (int pass = r0; pass < r1; pass += per_pass) {
        const int n = min(per_pass, r1 - pass), tiles = (n + 7) / 8;
        const int ts = n > 4 ? 3 : n > 2 ? 2 : n > 1 ? 1 : 0, TS = 1 << ts;  // tokens a tile of x holds here
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            sc[d] = mn[d] = make_uint4(0, 0, 0, 0);
            issue(ks + d * KS, d);
            issue_scales(ks + d * KS, sc[d], mn[d]);
        }
        float sum[NB][RG][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[nb][rg][i] = 0.f;
        for (int c0 = 0; c0 < steps; c0 += p.chunk) {
            // stage x: a code word's halves hold codes j and j + 4, so k j and k j + 4 share a register of x; those of
            // odd j scaled down by the 2^4 that their codes are high
            const int quads = min(p.chunk * (kStep / 32), p.K / 32 - c0 * (kStep / 32)), cgroups = quads * 32 / G;  // of 32 k
            const int quads4 = (quads + 3) & ~3;  // of whole 128 k, so that the four of one stay together
            if (c0) __syncthreads();
            // one token's 32 k: lanes of one token are TS apart, so the sums and the largest of 128 k are a shuffle away
            const int all = (tiles * quads4 << ts) + 31 & ~31;
            auto load = [&](int i, uint4(&v)[4]) {
                const int tq = i >> ts, nb = tq / quads4, quad = tq - nb * quads4, tok = 8 * nb + (i & (TS - 1));
                int row = -1;
                if (nb < tiles && quad < quads && tok < n) {
                    row = pass + tok;
                    if (p.sorted_tok) {
                        row = p.sorted_tok[row];
                        if (row < 0 || row >= p.T) {
                            if (blockIdx.x == 0 && quad == 0) flag(p.status, MOE_DEV_BAD_INDEX);
                            row = -1;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = make_uint4(0, 0, 0, 0);
                if (row >= 0) {
                    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const X *>(p.x) + int64_t(row) * p.K) +
                                        (c0 * (kStep / 32) + quad) * 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = __ldg(from + k);
                }
            };
            uint4 next[4];
            if (int(threadIdx.x) < all) load(threadIdx.x, next);
            for (int i = threadIdx.x; i < all; i += 32 * kWarps) {
                const int tq = i >> ts, nb = tq / quads4, quad = tq - nb * quads4;
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = next[k];
                if (i + 32 * kWarps < all) load(i + 32 * kWarps, next);  // on its way while these are scaled
                // the power of two of these 128 k: 14 less the exponent of their largest
                float x[4][8], most = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const X *h = reinterpret_cast<const X *>(&v[k]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[k][j] = to_f32(h[j]);
                        most = fmaxf(most, fabsf(x[k][j]));
                    }
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, TS));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2 * TS));
                const int e = min(14 - (int(__float_as_uint(most) >> 23) - 127), 100);
                const float up = __uint_as_float(uint32_t(127 + e) << 23);
                float part = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float eight = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[k][j] *= up;
                        eight += x[k][j];
                    }
                    part += eight;
                }
                if (MIN && G >= 64) part += __shfl_xor_sync(0xffffffffu, part, TS);
                if (MIN && G >= 128) part += __shfl_xor_sync(0xffffffffu, part, 2 * TS);
                if (nb < tiles && quad < quads) {
                    const int slot8 = i & (TS - 1);
                    if (MIN && (quad & (G / 32 - 1)) == 0) xsum[(nb * cgroups + quad / (G / 32)) * 8 + slot8] = part;
                    if ((quad & 3) == 0)
                        xdown[(nb * p.chunk * 2 + quad / 4) * 8 + slot8] = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int unit8 = quad * 4 + k, q = unit8 & (G / 8 - 1);
                        const int at = (unit8 & ~(G / 8 - 1)) + (q % W) * 4 + q / W;
                        uint32_t h[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float f = j & 1 ? 0.0625f : 1.f;
                            const __half2 two = __floats2half2_rn(x[k][j] * f, x[k][j + 4] * f);
                            h[j] = *reinterpret_cast<const uint32_t *>(&two);
                        }
                        xs[nb * tile_units + (at << ts) + slot8] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
            }
            __syncthreads();
            for (int step0 = c0 + ks; step0 < min(steps, c0 + p.chunk); step0 += kDepth * KS) {
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    const int step = step0 + d * KS;
                    if (step < steps && busy) {
                        tc::cp_async_wait<kDepth - 1>();
                        if (RG == 2 || lane < 16) {  // scale pairs of this lane's row
                            float2 *own = reinterpret_cast<float2 *>(pairs) + (lane >> 4) * 16 + 2 * (lane & 7) +
                                          ((lane >> 3) & 1);
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                const float s = half_at(sc[d], j);
                                own[j * R] = MIN ? make_float2(s * 16777216.f, half_at(mn[d], j)) : make_float2(s * 512.f, 0.f);
                            }
                        }
                        __syncwarp();
                        const unsigned char *st = mine + d * (R * 128) + g * 128;
                        const uint4 *xstep = xs + (((step - c0) * (kStep / 8) + t) << ts) + (g & (TS - 1));
                        // adds group j to y, in the scale of its 128 k
                        auto group = [&](int j, float(&y)[NB][RG][4]) {
                            uint32_t w[RG][2][W];
#pragma unroll
                            for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    // bytes (G / 8) t of the group's G / 2, in swizzled 16-byte chunks
                                    const int byte = j * (G / 2) + (G / 8) * t;
                                    const unsigned char *from = st + (16 * rg + 8 * i) * 128 +
                                                                (((byte >> 4) ^ swizzle<G>(g)) << 4) + (byte & 15);
                                    if constexpr (W == 1) {
                                        w[rg][i][0] = *reinterpret_cast<const uint32_t *>(from);
                                    } else if constexpr (W == 2) {
                                        const uint2 v = *reinterpret_cast<const uint2 *>(from);
                                        w[rg][i][0] = v.x, w[rg][i][1] = v.y;
                                    } else {
                                        const uint4 v = *reinterpret_cast<const uint4 *>(from);
                                        w[rg][i][0] = v.x, w[rg][i][1] = v.y, w[rg][i][2] = v.z, w[rg][i][3] = v.w;
                                    }
                                }
                            float acc[NB][RG][4];
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) acc[nb][rg][i] = 0.f;
#pragma unroll
                            for (int wi = 0; wi < W; ++wi) {
                                uint32_t lo[RG][4], hi[RG][4];
#pragma unroll
                                for (int rg = 0; rg < RG; ++rg) {
                                    halves_of<MIN>(w[rg][0][wi], lo[rg]);
                                    halves_of<MIN>(w[rg][1][wi], hi[rg]);
                                }
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    if (NB > 1 && nb >= tiles) break;
                                    const uint4 xv = xstep[nb * tile_units + ((j * W + wi) * 4 << ts)];
#pragma unroll
                                    for (int rg = 0; rg < RG; ++rg) {
                                        mma_fp16(acc[nb][rg], lo[rg][0], hi[rg][0], lo[rg][1], hi[rg][1], xv.x, xv.y);
                                        mma_fp16(acc[nb][rg], lo[rg][2], hi[rg][2], lo[rg][3], hi[rg][3], xv.z, xv.w);
                                    }
                                }
                            }
                            float2 x01[NB];
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                if (MIN && (NB == 1 || nb < tiles))
                                    x01[nb] = *reinterpret_cast<const float2 *>(
                                        xsum + (nb * cgroups + (step - c0) * J + j) * 8 + 2 * t);
#pragma unroll
                            for (int rg = 0; rg < RG; ++rg) {
                                const float4 f = pairs[(j * RG + rg) * 8 + g];  // s 2^24, m (s 2^9, 0) of row g, then of row g + 8
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    if (NB > 1 && nb >= tiles) break;
                                    float(&o)[4] = y[nb][rg];
                                    const float(&v)[4] = acc[nb][rg];
                                    if constexpr (MIN) {
                                        o[0] = fmaf(f.y, x01[nb].x, o[0]);
                                        o[1] = fmaf(f.y, x01[nb].y, o[1]);
                                        o[2] = fmaf(f.w, x01[nb].x, o[2]);
                                        o[3] = fmaf(f.w, x01[nb].y, o[3]);
                                    }
                                    o[0] = fmaf(f.x, v[0], o[0]);
                                    o[1] = fmaf(f.x, v[1], o[1]);
                                    o[2] = fmaf(f.z, v[2], o[2]);
                                    o[3] = fmaf(f.z, v[3], o[3]);
                                }
                            }
                        };
                        // `count` groups of 128 k, then out of their scale
                        auto half_step = [&](int h, int count, bool whole) {
                            float y[NB][RG][4];
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) y[nb][rg][i] = 0.f;
                            if (whole) {
#pragma unroll
                                for (int j = 0; j < J / 2; ++j) group(h * (J / 2) + j, y);
                            } else {
#pragma unroll 1
                                for (int j = 0; j < count; ++j) group(h * (J / 2) + j, y);
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                if (NB > 1 && nb >= tiles) break;
                                const float2 down = *reinterpret_cast<const float2 *>(
                                    xdown + ((nb * p.chunk + step - c0) * 2 + h) * 8 + 2 * t);
#pragma unroll
                                for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        sum[nb][rg][i] = fmaf(i & 1 ? down.y : down.x, y[nb][rg][i], sum[nb][rg][i]);
                            }
                        };
                        const int here = groups - step * J;
                        if (here >= J) {  // in one piece, so that the groups' products overlap
                            half_step(0, J / 2, true);
                            half_step(1, J / 2, true);
                        } else {
                            half_step(0, min(here, J / 2), false);
                            if (here > J / 2) half_step(1, here - J / 2, false);
                        }
                        __syncwarp();  // every lane has read the stage before it is refilled
                        issue(step + kDepth * KS, d);
                        issue_scales(step + kDepth * KS, sc[d], mn[d]);
                    }
                }
            }
        }
        tc::cp_async_wait<0>();
        __syncthreads();  // the rings are free: partial sums [token][row] take their place
        if (busy) {
            float *part = reinterpret_cast<float *>(mine);
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
            const unsigned char *from = smem + (u << p.ks_log2) * kWarpBytes<G, RG, NB>;
            float y = 0.f, up = 0.f;
            for (int k = 0; k < KS; ++k, from += kWarpBytes<G, RG, NB>) {
                const float *part = reinterpret_cast<const float *>(from) + tok * kPartStride;
                y += part[row];
                if (RG == 2 && p.swiglu) up += part[16 + row];
            }
            if (RG == 2 && p.swiglu) {
                // e^(-|y|/2), once for the gate and once for the up row: neither is a subnormal where their product
                // is not, so a far gate keeps its share of a large up row, and its digits
                const float e = expf(-0.5f * fabsf(y));
                if (y < 0.f) y *= e, up *= e;
                y = y / (1.0f + e * e) * up;
            }
            const int64_t at = int64_t(pass + tok) * cols + unit0 * per_unit + c;
            if (p.out_fp32) static_cast<float *>(p.out)[at] = y;
            else static_cast<X *>(p.out)[at] = from_f32<X>(y);
        }
        __syncthreads();  // read before the next pass refills the rings
    }
}

template <typename X, int G, int RG, int NB, bool MIN>
moe_status launch(Q4Params &p, int experts, cudaStream_t stream) {
    // x of the whole of k where two blocks of an SM still fit (one, with more
    // tiles of tokens), else in chunks
    const int steps = (p.K + kStep - 1) / kStep, unit = kDepth << p.ks_log2, per_step = NB * (kStep * 2 << p.ts_log2);
    const int whole = (steps + unit - 1) / unit, fit = (NB == 1 ? 36 : 128) * 1024 / (per_step * unit);
    p.chunk = std::max(1, std::min(whole, fit)) * unit;
    const size_t smem = size_t(kWarps) * kWarpBytes<G, RG, NB> +
                        size_t(p.chunk) * (per_step + (MIN ? NB * (kStep / G) * 32 : 0) + NB * 64);
    if (smem > kMaxSmem || !allow_smem(q4_kernel<X, G, RG, NB, MIN>, kMaxSmem)) return MOE_ERR_CUDA;
    const int units = p.swiglu ? p.N / 32 : p.N / (16 * RG), per_block = kWarps >> p.ks_log2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((units + per_block - 1) / per_block, experts);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    void *args[] = {&p};
    if (launch_early(cfg, attrs, 1, reinterpret_cast<const void *>(q4_kernel<X, G, RG, NB, MIN>), args) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

template <typename X, int G, bool MIN>
moe_status launch_g(Q4Params &p, int rg, int nb, int experts, cudaStream_t stream) {
    if (rg == 1)
        return nb == 1 ? launch<X, G, 1, 1, MIN>(p, experts, stream)
                       : nb == 2 ? launch<X, G, 1, 2, MIN>(p, experts, stream)
                                 : launch<X, G, 1, 4, MIN>(p, experts, stream);
    return nb == 1 ? launch<X, G, 2, 1, MIN>(p, experts, stream)
                   : nb == 2 ? launch<X, G, 2, 2, MIN>(p, experts, stream)
                             : launch<X, G, 2, 4, MIN>(p, experts, stream);
}

template <typename X, bool MIN>
moe_status launch_x(Q4Params &p, int group, int rg, int nb, int experts, cudaStream_t stream) {
    return group == 32 ? launch_g<X, 32, MIN>(p, rg, nb, experts, stream)
                       : group == 64 ? launch_g<X, 64, MIN>(p, rg, nb, experts, stream)
                                     : launch_g<X, 128, MIN>(p, rg, nb, experts, stream);
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
    p.scales_in_words = W->K % kStep == 0 && reinterpret_cast<uintptr_t>(W->scale) % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(W->min) % 16 == 0;
    // Token tiles: as many as a third more rows than a matrix has on average (at
    // most T) fill; two of four, if then 8 warps can share 16 rows in one turn of
    // an SM each. (64 experts with 5.8 rows: 48 us with one tile, 84 with two; 512
    // x 8192, 20 tokens: 31 us with two, 43 with four.)
    const int rows = int(std::min<int64_t>(p.T, (4 * int64_t(p.P) + 3 * experts - 1) / (3 * experts)));
    const int64_t units = int64_t(p.N / 32) * experts;
    const int nb = rows <= 8 ? 1 : rows <= 16 || (!p.swiglu && 2 * units <= 148) ? 2 : 4;
    p.ts_log2 = nb > 1 || p.T > 4 ? 3 : p.T > 2 ? 2 : p.T > 1 ? 1 : 0;
    // Warps that share rows: as many as leave all blocks running at once (two an
    // SM; one, where staging the x of several tokens weighs more than the codes),
    // up to 8 (4 with four token tiles, whose x would not fit); then 16 rows a
    // warp. Where the blocks take several turns anyway, pairs of warps, unless k
    // is too short to split. Measured (warps a row: us; those without min before
    // q - 8 was formed, which adds 4 to 6%): gate and up rows of one
    // token 1: 13.0, 2: 8.8, 4: 8.2, 8: 10.7 (480 blocks); 8192 x 8192, one token
    // 1: 32, 2: 19, 4: 12.8, 8: 12.1 (256 blocks), five tokens 4: 22, 8: 28; gate
    // and up rows of 37 tokens 1: 91, 2: 79, 4: 89; down rows (3 steps of k) of
    // four tokens 1: 17, 2: 20, 4: 24.
    const int64_t slots = 148 * kWarps * (rows > 2 ? 1 : 2);
    const int steps = (p.K + kStep - 1) / kStep, most = nb == 4 ? 2 : 3;
    int rg = 2, ks = 0;
    while (ks < most && (units << (ks + 1)) <= slots && (2 << ks) <= steps) ++ks;
    if (!p.swiglu && (units << (ks + 1)) <= slots) rg = 1;
    if (units > slots && steps >= 8) ks = 1;
    p.ks_log2 = ks;
    if (dtype == MOE_BF16)
        return W->min ? launch_x<__nv_bfloat16, true>(p, W->group, rg, nb, experts, stream)
                      : launch_x<__nv_bfloat16, false>(p, W->group, rg, nb, experts, stream);
    return W->min ? launch_x<__half, true>(p, W->group, rg, nb, experts, stream)
                  : launch_x<__half, false>(p, W->group, rg, nb, experts, stream);
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
    if (T > kMaxPairs) return MOE_ERR_OVERFLOW;
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
    if (int64_t(T) * k > kMaxPairs) return MOE_ERR_OVERFLOW;
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
