// Unquantised matrix products grouped by expert and their gradients, over the
// sorted pairs of a routed batch:
//   forward  out[s] = W[e] a_s,   dgrad  da[s] = W[e]^T dy[s],
//   wgrad    dW[e]  = base[e] + sum_s dy[s] a_s^T.
//
// One persistent tcgen05 kernel for the three. The index along which the
// output is contiguous is M (128 rows of tensor memory a CTA), so that a warp
// of the epilogue writes consecutive addresses; the other output index, tokens
// or n, is N (up to 256 columns, padded to 16, so that an expert with few rows
// costs few columns); 64 of the contracted index make a stage:
//   pass     M     N       contracted   A (M)                 B (N)
//   forward  n     pairs   k            W[e][n][k], K-major    a rows, K-major
//   dgrad    k     pairs   n            W[e][n][k], MN-major   dy rows, K-major
//   wgrad    k     n       pairs        a rows, MN-major       dy rows, MN-major
// The operands come by TMA in the 128-byte swizzle, rows picked by token with
// gathering loads (four rows each). Rows past an expert's end fall into columns
// that are never written; in wgrad, where they would be summed, the last stage
// is loaded row by row with an index past the tensor for them, which reads
// zeros. Warps: loads, MMA issue, eight for the epilogue; two accumulators, so
// that the epilogue of one tile runs beside the products of the next. Every
// wait is bounded and sets MOE_DEV_TIMEOUT.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

enum Pass { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kTileM = 128;      // rows of tensor memory
constexpr int kTileI = 64;       // contracted index a stage: 128 bytes, one swizzle row
constexpr int kLoadWarp = 0, kMmaWarp = 1, kEpiWarp0 = 2, kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kMaxStages = 10;
constexpr unsigned long long kWaitNs = 200ull * 1000 * 1000;

struct GemmParams {
    const int32_t *offsets, *sorted_tok;  // sorted_tok: rows of the gathered operand, or NULL
    const void *base;
    void *out;
    int rows_a;      // rows of the operand that sorted_tok picks from (T), or P
    int P, E;
    int M, I;        // extent of the output's contiguous index; of the contracted one (forward, dgrad)
    int N;           // wgrad: extent of the output's other index
    int bf16, out_fp32;
    int32_t *status;
};

// Tensor maps. w: weights [E][N][K]; rows, rows16: 64- and 16-row boxes of the
// 16-bit rows that are N (forward, dgrad) or M (wgrad); pick: single rows of
// the same; dy, dy_pick: wgrad's other operand.
struct GemmMaps {
    CUtensorMap w, rows, rows16, pick, dy, dy_pick;
};

struct GemmSmem {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
    uint32_t tmem_base;
    int abort;
    int warp_sum[kThreads / 32];
    int prefix[kMaxE + 1];  // tiles before expert e
};

template <int PASS, int TN>
struct Cfg {
    static constexpr int kA = kTileM * 128, kB = TN * 128, kStage = kA + kB;
    // what fits beside the tables in 227 KB
    static constexpr int kFit = (232448 - int(sizeof(GemmSmem)) - 1024) / kStage;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr int kSmem = kStages * kStage + 1024;
};

__device__ __forceinline__ void stop(GemmSmem &s, int32_t *status) {
    if (atomicExch(&s.abort, 1) == 0) flag(status, MOE_DEV_TIMEOUT);
}

// Rows of expert e; empty where the table is out of bounds.
__device__ __forceinline__ bool range_of(const GemmParams &p, int e, int &r0, int &r1) {
    r0 = p.offsets[e], r1 = p.offsets[e + 1];
    if (r0 >= 0 && r1 >= r0 && r1 <= p.P) return true;
    r0 = r1 = 0;
    return false;
}

template <int PASS, int TN>
__device__ __forceinline__ int tiles_of(const GemmParams &p, int e, int r0, int r1, int MT) {
    if (PASS != kWgrad) return MT * ((r1 - r0 + TN - 1) / TN);
    // an expert without rows: nothing to do where the sum so far is in place
    return r1 == r0 && p.base == p.out ? 0 : MT * ((p.N + TN - 1) / TN);
}

// Whole CTA: prefix sums of the experts' tiles; returns their total.
template <int PASS, int TN>
__device__ int build_prefix(const GemmParams &p, GemmSmem &s, int MT) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.E + kThreads - 1) / kThreads, e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int r0, r1;
        if (!range_of(p, e, r0, r1) && blockIdx.x == 0) flag(p.status, MOE_DEV_BAD_INDEX);
        const int n = tiles_of<PASS, TN>(p, e, r0, r1, MT);
        s.prefix[e] = sum;
        sum += n;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s.warp_sum[w];
        total += s.warp_sum[w];
    }
    for (int e = e0; e < e1; ++e) s.prefix[e] += before;
    if (tid == 0) s.prefix[p.E] = total;
    __syncthreads();
    return total;
}

struct Tile {
    int e, m0;       // expert; first M index
    int c0, n;       // forward, dgrad: first sorted pair and pairs; wgrad: first n and their number
    int r0, r1;      // the expert's rows
};

template <int PASS, int TN>
__device__ __forceinline__ Tile tile_at(const GemmParams &p, const GemmSmem &s, int tau, int MT) {
    int lo = 0, hi = p.E;  // last e with prefix[e] <= tau; experts without tiles share the next one's prefix
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.prefix[mid] <= tau) lo = mid; else hi = mid;
    }
    Tile t;
    t.e = lo;
    range_of(p, lo, t.r0, t.r1);
    const int local = tau - s.prefix[lo], j = local / MT;
    t.m0 = (local - j * MT) * kTileM;
    if (PASS == kWgrad) {
        t.c0 = j * TN;
        t.n = min(TN, p.N - t.c0);
    } else {  // the rows spread evenly over their tiles, in multiples of 16
        const int rows = t.r1 - t.r0, nt = (rows + TN - 1) / TN;
        const int per = ((rows + nt - 1) / nt + 15) & ~15;
        t.c0 = t.r0 + j * per;
        t.n = min(per, t.r1 - t.c0);
    }
    return t;
}

template <int PASS>
__device__ __forceinline__ int stages_of(const GemmParams &p, const Tile &t) {
    return ((PASS == kWgrad ? t.r1 - t.r0 : p.I) + kTileI - 1) / kTileI;
}

// MN-major operand, 128-byte swizzle: blocks of 64 along MN 8192 bytes apart
// (leading offset), groups of 8 along the contracted index 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFF) | (uint64_t(8192 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Token row of sorted pair `pair`, or a row past the tensor (which reads as
// zeros) where the token or the pair is out of bounds.
__device__ __forceinline__ int picked_row(const GemmParams &p, int pair, int end, int32_t *status) {
    if (pair >= end) return p.rows_a;
    if (!p.sorted_tok) return pair;
    const int t = p.sorted_tok[pair];
    if (t >= 0 && t < p.rows_a) return t;
    flag(status, MOE_DEV_BAD_INDEX);
    return p.rows_a;
}

// Load warp: fills stage after stage, all tiles of this CTA in a row.
template <int PASS, int TN>
__device__ void load_tiles(const GemmParams &p, GemmSmem &s, const GemmMaps &m, unsigned char *dyn, int total, int MT) {
    using C = Cfg<PASS, TN>;
    const int lane = threadIdx.x & 31;
    int it = 0;
    bool ok = true;
    for (int tau = blockIdx.x; tau < total && ok; tau += gridDim.x) {
        const Tile t = tile_at<PASS, TN>(p, s, tau, MT);
        const int KS = stages_of<PASS>(p, t);
        const int ablocks = min(2, (p.M - t.m0 + 63) / 64);  // 64-wide blocks of an MN-major A inside the tensor
        // forward by token: this lane's rows of N, four at a time (8 for 256 columns)
        int pick[TN / 128 > 0 ? TN / 128 : 1][4];
        if (PASS == kForward && p.sorted_tok) {
#pragma unroll
            for (int i = 0; i < (TN + 127) / 128; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    pick[i][r] = picked_row(p, t.c0 + 4 * (lane + 32 * i) + r, t.c0 + t.n, p.status);
        }
        for (int ks = 0; ks < KS; ++ks, ++it) {
            const int stage = it % C::kStages;
            if (!tc::mbar_wait(&s.empty[stage], ((it / C::kStages) & 1) ^ 1, kWaitNs) || s.abort) {
                ok = false;
                break;
            }
            unsigned char *a = dyn + stage * C::kStage, *b = a + C::kA;
            uint64_t *bar = &s.full[stage];
            if (PASS != kWgrad) {
                const bool small = t.n <= 48;
                const bool by_token = PASS == kForward && p.sorted_tok;
                const int picks = (t.n + 3) / 4, boxes = small ? (t.n + 15) / 16 : (t.n + 63) / 64;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(bar, uint32_t((PASS == kForward ? C::kA : ablocks * 8192) +
                                                            (by_token ? picks * 512 : boxes * (small ? 2048 : 8192))));
                    if (PASS == kForward) {
                        tc::tma_load_3d(a, &m.w, kTileI * ks, t.m0, t.e, bar);
                    } else {
                        for (int i = 0; i < ablocks; ++i)
                            tc::tma_load_3d(a + 8192 * i, &m.w, t.m0 + 64 * i, kTileI * ks, t.e, bar);
                    }
                    if (!by_token)
                        for (int i = 0; i < boxes; ++i)
                            tc::tma_load_2d(b + i * (small ? 2048 : 8192), small ? &m.rows16 : &m.rows, kTileI * ks,
                                            t.c0 + i * (small ? 16 : 64), bar);
                }
                __syncwarp();
                if (by_token) {
#pragma unroll
                    for (int i = 0; i < (TN + 127) / 128; ++i)
                        if (lane + 32 * i < picks)
                            tc::tma_gather4(b + (lane + 32 * i) * 512, &m.pick, kTileI * ks, pick[i][0], pick[i][1],
                                            pick[i][2], pick[i][3], bar);
                }
            } else {
                const int first = t.r0 + kTileI * ks, left = t.r1 - first;
                const bool tail = left < kTileI;
                const int bboxes = (t.n + 63) / 64;
                const int picks = (tail ? (left + 15) & ~15 : kTileI) / 4;  // groups of four rows
                const bool pick_a = tail || p.sorted_tok;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(bar, uint32_t(ablocks * (pick_a ? picks * 512 : 8192) +
                                                            (tail ? bboxes * picks * 512 : bboxes * 8192)));
                    if (!pick_a)
                        for (int i = 0; i < ablocks; ++i)
                            tc::tma_load_2d(a + 8192 * i, &m.rows, t.m0 + 64 * i, first, bar);
                    if (!tail)
                        for (int i = 0; i < bboxes; ++i)
                            tc::tma_load_2d(b + 8192 * i, &m.dy, t.c0 + 64 * i, first, bar);
                }
                __syncwarp();
                if (pick_a) {  // lane: 64-column block lane / 16, rows 4 (lane % 16) ..
                    const int g = lane & 15, blk = lane >> 4;
                    if (g < picks && blk < ablocks) {
                        int r[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[i] = picked_row(p, first + 4 * g + i, t.r1, p.status);
                        tc::tma_gather4(a + 8192 * blk + 512 * g, &m.pick, t.m0 + 64 * blk, r[0], r[1], r[2], r[3], bar);
                    }
                }
                if (tail)
                    for (int i = lane; i < bboxes * picks; i += 32) {
                        const int blk = i / picks, g = i - blk * picks;
                        int r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[j] = first + 4 * g + j < t.r1 ? first + 4 * g + j : p.P;
                        tc::tma_gather4(b + 8192 * blk + 512 * g, &m.dy_pick, t.c0 + 64 * blk, r[0], r[1], r[2], r[3],
                                        bar);
                    }
            }
        }
    }
    if (!ok) {
        stop(s, p.status);
        // no copy may land after this CTA's shared memory has another owner
        for (int i = max(0, it - C::kStages); i < it; ++i)
            tc::mbar_wait(&s.full[i % C::kStages], (i / C::kStages) & 1, kWaitNs);
    }
}

template <int PASS, int TN>
__device__ void issue_mma(const GemmParams &p, GemmSmem &s, unsigned char *dyn, int total, int MT, uint32_t tmem) {
    using C = Cfg<PASS, TN>;
    constexpr bool kMnA = PASS != kForward, kMnB = PASS == kWgrad;
    int it = 0, count = 0;
    bool ok = true;
    for (int tau = blockIdx.x; tau < total && ok && !s.abort; tau += gridDim.x) {
        const Tile t = tile_at<PASS, TN>(p, s, tau, MT);
        const int KS = stages_of<PASS>(p, t);
        if (KS == 0) continue;  // wgrad of an expert without rows
        const int buf = count & 1;
        if (!tc::mbar_wait(&s.tempty[buf], ((count >> 1) & 1) ^ 1, kWaitNs)) {
            ok = false;
            break;
        }
        tc::fence_after();
        ++count;
        const uint32_t fmt = p.bf16 ? 1u : 0u;
        const uint32_t idesc = tc::idesc_f16(kTileM, (t.n + 15) & ~15) | (fmt << 7) | (fmt << 10) |
                               (kMnA ? 1u << 15 : 0u) | (kMnB ? 1u << 16 : 0u);
        const uint32_t d = tmem + uint32_t(buf * TN);
        for (int ks = 0; ks < KS; ++ks, ++it) {
            const int stage = it % C::kStages;
            if (!tc::mbar_wait(&s.full[stage], (it / C::kStages) & 1, kWaitNs)) {
                ok = false;
                break;
            }
            tc::fence_after();
            const uint32_t a = tc::smem_u32(dyn + stage * C::kStage), b = a + C::kA;
            const int left = PASS == kWgrad ? t.r1 - t.r0 - kTileI * ks : p.I - kTileI * ks;
            const int steps = min(4, (left + 15) >> 4);  // of 16; the last one reads zeros past the end
            for (int kk = 0; kk < steps; ++kk)
                tc::mma_f16(d, kMnA ? desc_mn128(a + 2048 * kk) : tc::desc_sw128(a + 32 * kk),
                            kMnB ? desc_mn128(b + 2048 * kk) : tc::desc_sw128(b + 32 * kk), idesc, (ks | kk) ? 1u : 0u);
            tc::mma_commit(&s.empty[stage]);
        }
        if (ok) tc::mma_commit(&s.tfull[buf]);
    }
    if (!ok) stop(s, p.status);
}

// Output element types behind one store: O a column's 32 consecutive values,
// or, for 16-bit outputs, two columns at once (lane pairs swap halves so that
// each lane holds two neighbours of one column).
template <int PASS, int TN, typename O>
__device__ void store_tiles(const GemmParams &p, GemmSmem &s, int total, int MT, uint32_t tmem) {
    const int warp = (threadIdx.x >> 5) - kEpiWarp0, lane = threadIdx.x & 31;
    const int q = (warp + kEpiWarp0) & 3, half = warp >> 2;  // lane quadrant of tensor memory; column half
    int count = 0;
    for (int tau = blockIdx.x; tau < total && !s.abort; tau += gridDim.x) {
        const Tile t = tile_at<PASS, TN>(p, s, tau, MT);
        const bool sums = stages_of<PASS>(p, t) > 0;
        const int buf = count & 1;
        if (sums) {
            if (!tc::mbar_wait_sleep(&s.tfull[buf], (count >> 1) & 1, kWaitNs, 64)) {
                stop(s, p.status);
                break;
            }
            tc::fence_after();
            ++count;
        }
        const int m = t.m0 + 32 * q + lane;
        const int64_t row0 = PASS == kWgrad ? int64_t(t.e) * p.N + t.c0 : int64_t(t.c0);
        const uint32_t td = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf * TN);
        for (int c = 16 * half; c < t.n; c += 32) {
            float v[16];
            if (sums) {
                tc::tmem_ld16(td + c, v);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0.f;
            }
            if (sizeof(O) == 4) {
                if (m < p.M) {
                    float *o = static_cast<float *>(p.out) + (row0 + c) * p.M + m;
                    if (PASS == kWgrad && p.base) {
                        const float *b = static_cast<const float *>(p.base) + (row0 + c) * p.M + m;
                        float bv[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) bv[j] = c + j < t.n ? b[int64_t(j) * p.M] : 0.f;
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += bv[j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < t.n) o[int64_t(j) * p.M] = v[j];
                }
            } else {
                const int odd = lane & 1;
                const int64_t at = (row0 + c + odd) * p.M + (m & ~1);
                uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<O *>(p.out) + at);
                const uint32_t *b = reinterpret_cast<const uint32_t *>(static_cast<const O *>(p.base) + at);
                uint32_t bv[8];
                if (PASS == kWgrad && p.base) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        bv[j] = m < p.M && c + 2 * j + odd < t.n ? b[int64_t(j) * p.M] : 0u;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * j] : v[2 * j + 1], 1);
                    float lo = odd ? got : v[2 * j], hi = odd ? v[2 * j + 1] : got;
                    O pair[2];
                    if (PASS == kWgrad && p.base) {
                        const O *old = reinterpret_cast<const O *>(&bv[j]);
                        lo += to_f32(old[0]);
                        hi += to_f32(old[1]);
                    }
                    pair[0] = from_f32<O>(lo);
                    pair[1] = from_f32<O>(hi);
                    if (m < p.M && c + 2 * j + odd < t.n) o[int64_t(j) * p.M] = *reinterpret_cast<const uint32_t *>(pair);
                }
            }
        }
        if (sums) {
            tc::fence_before();
            tc::mbar_arrive(&s.tempty[buf]);
        }
    }
}

template <int PASS, int TN>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ GemmMaps maps) {
    using C = Cfg<PASS, TN>;
    extern __shared__ __align__(1024) unsigned char dyn_raw[];
    unsigned char *dyn =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    __shared__ GemmSmem s;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int MT = (p.M + kTileM - 1) / kTileM;
    constexpr int kCols = 2 * TN < 32 ? 32 : 2 * TN;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&s.full[i], 1);
            tc::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.tfull[i], 1);
            tc::mbar_init(&s.tempty[i], 32 * kEpiWarps);
        }
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem_base, kCols);
    const int total = build_prefix<PASS, TN>(p, s, MT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s.tmem_base;
    if (warp == kLoadWarp) {
        load_tiles<PASS, TN>(p, s, maps, dyn, total, MT);
    } else if (warp == kMmaWarp) {
        if ((tid & 31) == 0) issue_mma<PASS, TN>(p, s, dyn, total, MT, tmem);
    } else if (p.out_fp32) {
        store_tiles<PASS, TN, float>(p, s, total, MT, tmem);
    } else if (p.bf16) {
        store_tiles<PASS, TN, __nv_bfloat16>(p, s, total, MT, tmem);
    } else {
        store_tiles<PASS, TN, __half>(p, s, total, MT, tmem);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kCols);
    }
}

// ------------------------------------------------------------------- host side
std::mutex g_mu;
int g_sms[64] = {};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// The tensor-map encoder (looked up once) and the current device's SM count.
bool host_setup(int &sms) {
    int dev = 0;
    std::lock_guard<std::mutex> lock(g_mu);
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!g_sms[dev] && cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return false;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    sms = g_sms[dev];
    return true;
}

// 16-bit tensor [slabs][rows][inner] in boxes of box_rows x 64, 128-byte swizzle, zeros outside.
bool map16(CUtensorMap *m, bool bf16, const void *base, int64_t inner, int64_t rows, int64_t slabs, uint32_t box_rows) {
    const cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(slabs)};
    const cuuint64_t strides[2] = {cuuint64_t(inner) * 2, cuuint64_t(inner) * cuuint64_t(rows) * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, slabs ? 3 : 2,
                    const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PASS, int TN>
moe_status launch(const GemmParams &p, const GemmMaps &maps, int64_t most_tiles, int sms, cudaStream_t stream) {
    using C = Cfg<PASS, TN>;
    static_assert(C::kStages >= 4, "fewer than four stages fit");
    if (cudaFuncSetAttribute(expert_gemm_kernel<PASS, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int grid = int(std::min<int64_t>(sms, most_tiles));
    expert_gemm_kernel<PASS, TN><<<grid, kThreads, C::kSmem, stream>>>(p, maps);
    return launch_status();
}

// rows: a (forward, wgrad) or dy (dgrad); inner: its row length.
moe_status run_gemm(int pass, GemmParams &p, const void *w, const void *rows, const void *dy, int N, int K,
                    cudaStream_t stream) {
    int sms = 0;
    if (!host_setup(sms)) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    GemmMaps maps = {};
    const bool bf = p.bf16;
    const int inner = pass == kDgrad ? N : K;
    // an empty batch (wgrad) has no rows to describe; nothing is loaded then
    const int64_t nrows = std::max(p.rows_a, 1), npairs = std::max(p.P, 1);
    bool ok = true;
    if (p.P > 0) {
        ok = map16(&maps.rows, bf, rows, inner, nrows, 0, 64) && map16(&maps.pick, bf, rows, inner, nrows, 0, 1);
        if (pass != kWgrad)
            ok = ok && map16(&maps.rows16, bf, rows, inner, nrows, 0, 16) &&
                 map16(&maps.w, bf, w, K, N, p.E, pass == kForward ? 128 : 64);
        else
            ok = ok && map16(&maps.dy, bf, dy, N, npairs, 0, 64) && map16(&maps.dy_pick, bf, dy, N, npairs, 0, 1);
    }
    if (!ok) return MOE_ERR_CUDA;
    const int64_t MT = (p.M + kTileM - 1) / kTileM;
    if (pass == kWgrad)
        return launch<kWgrad, 256>(p, maps, MT * ((N + 255) / 256) * p.E, sms, stream);
    // Few rows an expert: narrow tiles, so that more stages of weights are in flight.
    const int64_t experts = std::min<int64_t>(p.E, p.P);
    const bool narrow = p.P <= 16 * experts;
    const int64_t most = MT * (experts + p.P / (narrow ? 32 : 256));
    if (pass == kForward)
        return narrow ? launch<kForward, 32>(p, maps, most, sms, stream)
                      : launch<kForward, 256>(p, maps, most, sms, stream);
    return narrow ? launch<kDgrad, 32>(p, maps, most, sms, stream) : launch<kDgrad, 256>(p, maps, most, sms, stream);
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
    GemmParams p = {offsets, sorted_tok, nullptr, out, sorted_tok ? T : T * k, T * k, E, N, K, 0,
                    dtype == MOE_BF16, out_dtype == MOE_FP32, dev_status};
    return run_gemm(kForward, p, W, a, nullptr, N, K, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_dgrad(const void *dy, const void *W, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, void *da, int out_dtype, int32_t *dev_status,
                                         moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK || T == 0) return st;
    if (!dy || !W || !offsets || !da || !aligned16(dy) || !aligned16(W) || !aligned16(da)) return MOE_ERR_INVALID_ARG;
    GemmParams p = {offsets, nullptr, nullptr, da, T * k, T * k, E, K, N, 0,
                    dtype == MOE_BF16, out_dtype == MOE_FP32, dev_status};
    return run_gemm(kDgrad, p, W, dy, nullptr, N, K, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_wgrad(const void *dy, const void *a, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, const int32_t *sorted_tok, const void *base,
                                         void *dW, int out_dtype, int32_t *dev_status, moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK) return st;
    if (!offsets || !dW || !aligned16(dW) || !aligned16(base)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !a || !aligned16(dy) || !aligned16(a))) return MOE_ERR_INVALID_ARG;
    GemmParams p = {offsets, sorted_tok, base, dW, sorted_tok ? T : T * k, T * k, E, K, 0, N,
                    dtype == MOE_BF16, out_dtype == MOE_FP32, dev_status};
    return run_gemm(kWgrad, p, nullptr, a, dy, N, K, as_cuda(stream));
}
