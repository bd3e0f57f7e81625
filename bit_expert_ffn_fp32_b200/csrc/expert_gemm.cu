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
// Wide tiles are computed by pairs of CTAs (cta_group::2, M = 256): each loads
// its own half of A and of B, which cuts the L2 traffic of a 160-row tile by a
// quarter. Operands come by TMA in the 128-byte swizzle, except rows picked by
// token and wgrad's last stage of an expert (rows past its end must read as
// zeros there, as they are summed): those are written by gathering warps with
// 16-byte cp.async in the same swizzle (gathering TMA loads of four rows took
// about 48 cycles each, ten bytes a cycle). Warps: TMA, MMA issue, eight for
// the epilogue, eight (wgrad: four) that gather and one that hands their stages
// on; two accumulators, so that the epilogue of one tile runs beside the
// products of the next. Every wait is bounded and sets MOE_DEV_TIMEOUT.
//
// Measured (device time of a call in a burst; back to back, at the sustained
// clock): 81,920 pairs by token, 512 experts, 1536 x 2048: 653-704 us, 76 to 82%
// of the copy bandwidth on its 3.5 GB (830 us); dgrad of 4096 tokens, top-10 of
// 128 experts, the same weights: 228-257 us (298), tensor pipe 69% active, DRAM
// 60%; wgrad of 2048 x 768 for them: 150 us (181), where MMA and epilogue take
// turns (5.6 stages a tile); four tokens through 2048 x 768 in fp32: 25-27 us,
// 69 to 74% of the copy bandwidth.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "row_tiles.h"
#include "tc05.cuh"

namespace moe {
namespace {

enum Pass { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kTileM = 128;      // rows of tensor memory of a CTA
constexpr int kTileI = 64;       // contracted index a stage: 128 bytes, one swizzle row
constexpr int kLoadWarp = 0, kMmaWarp = 1, kEpiWarp0 = 2, kEpiWarps = 8, kPickWarp0 = kEpiWarp0 + kEpiWarps;
constexpr int kPickThreads = 128;  // gathering threads that fill a stage
constexpr int kMaxStages = 10;
constexpr int kTurn = 2048;      // per epilogue warp: a box of results on its way out
constexpr int kMaxDynamic = kMaxSmem - 1024;  // 1 KB: GemmSmem
constexpr unsigned long long kWaitNs = 200ull * 1000 * 1000;

struct GemmParams {
    const int32_t *offsets, *sorted_tok;  // sorted_tok: rows of the gathered operand, or NULL
    const uint16_t *rows, *dy;            // a (forward, wgrad), as the gathering warps read it; wgrad's dy
    const void *base;
    void *out;
    int rows_a;      // rows of the operand that sorted_tok picks from (T), or P
    int P, E;
    int M, I;        // extent of the output's contiguous index; of the contracted one (forward, dgrad)
    int N;           // wgrad: extent of the output's other index
    int bf16, out_fp32;
    int stages;      // of the shared-memory ring
    int read_base;   // 1: wgrad's sum so far is read (0: there is none, or the results are added where it is)
    int blocks2;     // 1: MN-major operands are mapped in 64-wide blocks, two a box (extents multiples of 64)
    int32_t *status;
};

// Tensor maps. w: weights [E][N][K]; rows: the rows that are N (forward, dgrad)
// in boxes of 16, 32, 64, 96 and 128 rows, so that a tile's are one load; rows[0]
// of wgrad: the rows that are M; dy: wgrad's other operand; out, base: the
// result and wgrad's sum so far, in boxes of 32 M and 32 (16-bit) or 16 (fp32)
// columns.
constexpr int kBoxes = 5;
__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 16 : 32 * i; }
struct GemmMaps {
    CUtensorMap w, rows[kBoxes], dy, out, base;
};

// One expert that has tiles: its first tile, rows and id.
struct Entry {
    int tile, r0, rows, e;
};

struct GemmSmem {
    uint64_t full[kMaxStages], empty[kMaxStages], landed[kMaxStages], tfull[2], tempty[2], based[kEpiWarps];
    uint32_t tmem_base;
    int abort, entries;
    int warp_tiles[32], warp_entries[32];
};

// CG: CTAs that share a tile; TN: columns of a tile; PICK: groups of gathering
// warps, stages they fill at the same time (0: none).
template <int PASS_, int CG_, int TN_, int PICK_>
struct Cfg {
    static constexpr int PASS = PASS_, CG = CG_, TN = TN_, PICK = PICK_;
    static constexpr int kRelayWarp = kPickWarp0 + PICK * kPickThreads / 32;
    static constexpr int kThreads = 32 * (PICK ? kRelayWarp + 1 : kPickWarp0);
    static constexpr int kBRows = TN / CG;  // of B a CTA holds
    static constexpr int kA = kTileM * 128, kB = kBRows * 128, kStage = kA + kB;
    // shared memory: the ring, the epilogue's boxes (twice with a sum to read), the table of E + 1 entries
    static constexpr size_t fixed(int E, int read_base) {
        return kEpiWarps * kTurn * (1 + read_base) + (size_t(E) + 1) * sizeof(Entry) + 1024;
    }
    static constexpr int stages(int E, int read_base) {
        const size_t fit = (kMaxDynamic - fixed(E, read_base)) / kStage;
        return fit < size_t(kMaxStages) ? int(fit) : kMaxStages;
    }
    // Tensor memory: two buffers, so that the epilogue of one tile runs beside the
    // products of the next. The tensor cores cut instead of round, an error that
    // grows with the length of a chain: narrow tiles with fp32 results take the
    // stages of a buffer in turns to kAccs accumulators, added at the end, and a
    // tile whose sums are long takes both buffers (segments_of).
    static constexpr int kAccs = CG == 1 ? 4 : 1, kBuf = kAccs * TN, kCols = 2 * kBuf;
    static_assert(stages(kMaxE, PASS == kWgrad) >= 4 && sizeof(GemmSmem) <= 1024 && kCols >= 32 && kCols <= 512,
                  "tile does not fit");
};

__device__ __forceinline__ void stop(GemmSmem &s, int32_t *status) {
    if (atomicExch(&s.abort, 1) == 0) flag(status, MOE_DEV_TIMEOUT);
}

// Rows of expert e; empty where the table is out of bounds.
__device__ __forceinline__ bool range_of(const GemmParams &p, int e, int &r0, int &rows) {
    r0 = p.offsets[e];
    const int r1 = p.offsets[e + 1];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.P;
    rows = ok ? r1 - r0 : 0;
    return ok;
}

template <typename C>
__device__ __forceinline__ int tiles_of(const GemmParams &p, int rows, int MT) {
    if (C::PASS != kWgrad) return MT * row_tiles(rows, C::TN);
    // an expert without rows: nothing to do where the sum so far is in place
    return rows > 0 || p.base != p.out ? MT * ((p.N + C::TN - 1) / C::TN) : 0;
}

// Whole CTA: the experts that have tiles, in order, and a last entry with the
// number of all tiles, which is returned.
template <typename C>
__device__ int build_table(const GemmParams &p, GemmSmem &s, Entry *table, int MT) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.E + C::kThreads - 1) / C::kThreads, e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
    int tiles = 0, entries = 0, r0, rows;
    for (int e = e0; e < e1; ++e) {
        if (!range_of(p, e, r0, rows) && blockIdx.x == 0) flag(p.status, MOE_DEV_BAD_INDEX);
        const int n = tiles_of<C>(p, rows, MT);
        tiles += n;
        entries += n > 0;
    }
    int t_incl = tiles, n_incl = entries;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, t_incl, o), n = __shfl_up_sync(0xffffffffu, n_incl, o);
        if (lane >= o) t_incl += t, n_incl += n;
    }
    if (lane == 31) s.warp_tiles[warp] = t_incl, s.warp_entries[warp] = n_incl;
    __syncthreads();
    int tile = t_incl - tiles, at = n_incl - entries, total = 0, all = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
        const int t = s.warp_tiles[w], n = s.warp_entries[w];
        if (w < warp) tile += t, at += n;
        total += t, all += n;
    }
    for (int e = e0; e < e1; ++e) {
        range_of(p, e, r0, rows);
        const int n = tiles_of<C>(p, rows, MT);
        if (n > 0) table[at++] = {tile, r0, rows, e};
        tile += n;
    }
    if (tid == 0) {
        table[all] = {total, 0, 0, 0};
        s.entries = all;
    }
    return total;
}

struct Tile {
    int e, m0;       // expert; first M index of this CTA
    int c0, n;       // forward, dgrad: first sorted pair and pairs; wgrad: first n and their number
    int r0, rows;    // the expert's rows
    int npad, b0;    // n padded to the MMA's 16 a CTA; first of the npad / CG of them whose B rows this CTA loads
};

// A warp's way through this CTA's tiles.
template <typename C>
struct Walk {
    const Entry *table;
    int entries, MT, rank, at = 0;
    float inv_mt;
    __device__ Walk(const GemmSmem &s, const Entry *table, int MT, int rank)
        : table(table), entries(s.entries), MT(MT), rank(rank), inv_mt(1.0f / MT) {}
    // Tile tau, not before the last one asked for. All lanes together.
    __device__ __forceinline__ Tile tile(const GemmParams &p, int tau) {
        for (;;) {  // each lane looks at one of the next 32 entries
            const int ahead = at + 1 + (threadIdx.x & 31);
            const unsigned past = __ballot_sync(0xffffffffu, ahead < entries && table[min(ahead, entries)].tile <= tau);
            at += __popc(past);
            if (past != 0xffffffffu) break;
        }
        const Entry x = table[at];
        Tile t;
        t.e = x.e, t.r0 = x.r0, t.rows = x.rows;
        const int local = tau - x.tile;
        int j = local / (1 << 22) ? local / MT : int(float(local) * inv_mt);  // local / MT, off by one at most
        j += (j + 1) * MT <= local;
        j -= j * MT > local;
        t.m0 = ((local - j * MT) * C::CG + rank) * kTileM;
        if (C::PASS == kWgrad) {
            t.c0 = j * C::TN;
            t.n = min(C::TN, p.N - t.c0);
        } else {
            const int per = rows_per_tile(t.rows, row_tiles(t.rows, C::TN), C::TN);
            t.c0 = t.r0 + j * per;
            t.n = min(per, t.r0 + t.rows - t.c0);
        }
        // in 64-wide blocks, each CTA of a pair takes whole ones
        t.npad = C::PASS == kWgrad && p.blocks2 ? (t.n + 127) & ~127 : padded_columns(t.n, C::CG);
        t.b0 = rank * (t.npad / C::CG);
        return t;
    }
};

template <typename C>
__device__ __forceinline__ int stages_of(const GemmParams &p, const Tile &t) {
    return ((C::PASS == kWgrad ? t.rows : p.I) + kTileI - 1) / kTileI;
}

// A tile's stages fall into segments, so that no chain of an fp32 result is
// longer than 1024 products of the contracted index (relative error 1e-6 by
// norms; 9e-6 at 16384 in two chains; wide tiles keep to one of 768, 7e-7, or two
// up to 2048), none of a 16-bit one longer than 16384 (1.5e-5, against half a
// step of 4.9e-4 in fp16). One segment: a buffer, the
// tiles take them in turns. Several: the first is summed in the tile's buffer,
// the others in the other one, from where the epilogue adds them to the first;
// each costs the tensor cores a pause of the epilogue's two reads and a write
// (fp32 results of 8 x 512 rows, N = 2048, in a burst: K = 4096 60.2 -> 62.2 us,
// 16384 213 -> 226; 2048 34.6 -> 34.8).
struct Segments {
    int count, per;  // per: stages of each but the last
};
template <typename C>
__device__ __forceinline__ Segments segments_of(const GemmParams &p, int KS) {
    constexpr int kMost = 16 * C::kAccs, kFirst = C::kAccs == 1 ? 12 : kMost;  // stages: of a segment, of a single one
    if (KS <= (p.out_fp32 ? kFirst : 256)) return {1, KS};  // no division on the way of most tiles
    const int count = p.out_fp32 ? max(2, (KS + kMost - 1) / kMost) : (KS + 255) / 256;
    return {count, (KS + count - 1) / count};
}
// Accumulators of a buffer that a segment of `stages` fills.
template <typename C>
__device__ __forceinline__ int accs_of(const GemmParams &p, int stages) {
    return p.out_fp32 ? min(C::kAccs, stages) : min(1, stages);
}

// The buffers as a role goes through them: whose turn it is, and the phase of
// each buffer's barriers.
struct Buffers {
    int next = 0;
    uint32_t phases = 0;
    // The buffer of segment i of a tile, and its phase.
    __device__ __forceinline__ int take(int i, uint32_t &phase) {
        const int b = next ^ int(i > 0);
        phase = (phases >> b) & 1;
        phases ^= 1u << b;
        return b;
    }
    // After a tile: one with several segments leaves the other buffer last.
    __device__ __forceinline__ void turn(const Segments &g) { next ^= int(g.count == 1); }
};

// MN-major operand, 128-byte swizzle: blocks of 64 along MN 8192 bytes apart
// (leading offset), groups of 8 along the contracted index 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFF) | (uint64_t(8192 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Position in the ring of stages.
struct Ring {
    int stages, stage = 0;
    uint32_t phase = 0;
    __device__ explicit Ring(int stages) : stages(stages) {}
    __device__ __forceinline__ void next() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// TMA warp: fills stage after stage, all tiles of this CTA in a row. The bytes
// of both CTAs of a pair count on rank 0's barrier.
template <typename C>
__device__ void load_tiles(const GemmParams &p, GemmSmem &s, const GemmMaps &m, unsigned char *dyn, Walk<C> walk,
                           int total) {
    Ring at(p.stages);
    int it = 0;
    bool ok = true;
    const uint32_t full0 = C::CG == 2 ? tc::at_rank(tc::smem_u32(&s.full[0]), 0) : tc::smem_u32(&s.full[0]);
    const uint32_t dyn0 = tc::smem_u32(dyn);
    auto load2 = [](uint32_t dst, const void *map, int x, int y, uint32_t bar) {
        if (C::CG == 2) tc::tma_load_2d_pair(dst, map, x, y, bar);
        else tc::tma_load_2d_at(dst, map, x, y, bar);
    };
    auto load3 = [](uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
        if (C::CG == 2) tc::tma_load_3d_pair(dst, map, x, y, z, bar);
        else tc::tma_load_3d_at(dst, map, x, y, z, bar);
    };
    auto load4 = [](uint32_t dst, const void *map, int x, int y, int z, int w, uint32_t bar) {
        if (C::CG == 2) tc::tma_load_4d_pair(dst, map, x, y, z, w, bar);
        else tc::tma_load_4d_at(dst, map, x, y, z, w, bar);
    };
    for (int tau = blockIdx.x / C::CG; tau < total && ok; tau += gridDim.x / C::CG) {
        const Tile t = walk.tile(p, tau);
        const int KS = stages_of<C>(p, t);
        // 64-wide blocks of an MN-major A that lie inside the tensor (none for a
        // CTA whose rows all lie past it), and the same of both CTAs of a pair;
        // a box of two counts whole
        const int rank = walk.rank, mfirst = t.m0 - rank * kTileM;
        int ablocks = max(0, min(2, (p.M - t.m0 + 63) / 64)), ablocks_all = min(2 * C::CG, (p.M - mfirst + 63) / 64);
        if (p.blocks2) ablocks_all += ablocks_all & 1, ablocks += ablocks & 1;
        // rows of B in one box (the same in both CTAs); wgrad: 64-wide blocks of n
        const int brows = t.npad / C::CG, brow0 = t.c0 + t.b0;
        const int box = brows <= 16 ? 0 : (brows + 31) / 32;
        int bblocks = (brows + 63) / 64;
        if (p.blocks2) bblocks += bblocks & 1;
        // bytes of a stage of both CTAs
        const uint32_t bytes_a = C::PASS == kForward ? C::CG * C::kA : ablocks_all * 8192;
        const uint32_t bytes_b = C::PASS == kWgrad ? C::CG * bblocks * 8192
                                                   : C::PICK ? 0 : C::CG * box_rows(box) * 128;
        for (int ks = 0; ks < KS; ++ks, ++it, at.next()) {
            if (!tc::mbar_wait_warp(&s.empty[at.stage], at.phase ^ 1, kWaitNs)) {
                ok = false;
                break;
            }
            const uint32_t a = dyn0 + at.stage * C::kStage, b = a + C::kA, bar = full0 + at.stage * 8;
            const int i0 = kTileI * ks;
            // wgrad's last stage of an expert, and its rows by token, come from the gathering warps
            const bool load_b = C::PASS == kWgrad ? t.rows - i0 >= kTileI : !C::PICK;
            const bool load_a = C::PASS != kWgrad || (load_b && !p.sorted_tok);
            if (tc::elect_one()) {
                if (rank == 0)
                    tc::mbar_arrive_expect_tx(&s.full[at.stage], (load_a ? bytes_a : 0) + (load_b ? bytes_b : 0));
                if (C::PASS == kForward) {
                    load3(a, &m.w, i0, t.m0, t.e, bar);
                } else if (load_a && p.blocks2) {
                    if (ablocks) {
                        if (C::PASS == kDgrad) load4(a, &m.w, 0, i0, t.m0 / 64, t.e, bar);
                        else load3(a, &m.rows[0], 0, t.r0 + i0, t.m0 / 64, bar);
                    }
                } else if (load_a) {
                    for (int i = 0; i < ablocks; ++i) {
                        if (C::PASS == kDgrad) load3(a + 8192 * i, &m.w, t.m0 + 64 * i, i0, t.e, bar);
                        else load2(a + 8192 * i, &m.rows[0], t.m0 + 64 * i, t.r0 + i0, bar);
                    }
                }
                if (C::PASS == kWgrad && load_b) {
                    if (p.blocks2) load3(b, &m.dy, 0, t.r0 + i0, brow0 / 64, bar);
                    else
                        for (int i = 0; i < bblocks; ++i) load2(b + 8192 * i, &m.dy, brow0 + 64 * i, t.r0 + i0, bar);
                }
                if (C::PASS != kWgrad && !C::PICK) load2(b, &m.rows[box], i0, brow0, bar);
            }
            __syncwarp();
        }
    }
    if (!ok) {
        stop(s, p.status);
        // no copy may land after this CTA's shared memory has another owner
        if (walk.rank == 0)
            for (int i = max(0, it - p.stages); i < it; ++i)
                tc::mbar_wait(&s.full[i % p.stages], (i / p.stages) & 1, kWaitNs);
    }
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Token row of sorted pair `pair`, -1 (read as zeros) where the pair or its token is out of bounds.
__device__ __forceinline__ int picked_row(const GemmParams &p, int pair, int end) {
    if (pair >= end) return -1;
    if (!p.sorted_tok) return pair;
    const int t = p.sorted_tok[pair];
    if (t >= 0 && t < p.rows_a) return t;
    flag(p.status, MOE_DEV_BAD_INDEX);
    return -1;
}

// Gathering warps: forward's rows by token (K-major B); wgrad's rows by token
// (MN-major A) and, in an expert's last stage, the rows of both operands. Four
// warps fill a stage; two groups of four take every second one. They never wait
// for their copies: those arrive on `landed` by themselves, so that a whole ring
// of stages is in flight, and the relay warp hands the stage to the MMA.
template <typename C>
__device__ void gather_tiles(const GemmParams &p, GemmSmem &s, unsigned char *dyn, Walk<C> walk, int total) {
    const int tid = (threadIdx.x - 32 * kPickWarp0) % kPickThreads;
    const int group = (threadIdx.x - 32 * kPickWarp0) / kPickThreads;
    const uint32_t dyn0 = tc::smem_u32(dyn);
    Ring at(p.stages);
    int it = 0;
    bool ok = true;
    // this thread's chunk of 16 bytes in its rows, and its place in a stage: rows
    // 16 (forward) or 8 (wgrad) apart have the same swizzle
    constexpr int kCh = C::PASS == kForward ? 8 : 16, kApart = kPickThreads / kCh;
    constexpr int kRows = (C::PASS == kForward ? C::kBRows : kTileI) / kApart;
    const int ch = tid % kCh, row0 = tid / kCh;
    const uint32_t off = (ch >> 3) * 8192 + row0 * 128 + (((ch & 7) ^ (row0 & 7)) << 4);
    for (int tau = blockIdx.x / C::CG; tau < total && ok; tau += gridDim.x / C::CG) {
        const Tile t = walk.tile(p, tau);
        const int KS = stages_of<C>(p, t), brows = t.npad / C::CG;
        const uint16_t *from[kRows];  // this thread's chunk in each of its rows, NULL: zeros
        if (C::PASS == kForward) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = row0 + kApart * i;
                const int row = r < brows ? picked_row(p, t.c0 + t.b0 + r, t.c0 + t.n) : -1;
                from[i] = row >= 0 ? p.rows + int64_t(row) * p.I + 8 * ch : nullptr;
            }
        }
        const bool picks = C::PASS == kForward || p.sorted_tok;
        const int end = t.r0 + t.rows;
        const int m = t.m0 + 8 * ch;
        int row[kRows];  // wgrad: rows of the next stage this thread fills
        auto next_rows = [&](int ks) {
            const int first = t.r0 + kTileI * ks;
            if (ks < KS && (p.sorted_tok || end - first < kTileI))
#pragma unroll
                for (int i = 0; i < kRows; ++i) row[i] = picked_row(p, first + row0 + kApart * i, end);
        };
        if (C::PASS == kWgrad) next_rows(C::PICK == 2 ? (it + group) & 1 : 0);
        for (int ks = 0; ks < KS; ++ks, ++it, at.next()) {
            if (C::PICK == 2 && (it & 1) != group) continue;
            if (!tc::mbar_wait_warp(&s.empty[at.stage], at.phase ^ 1, kWaitNs)) {
                ok = false;
                break;
            }
            const uint32_t a = dyn0 + at.stage * C::kStage, b = a + C::kA;
            if (C::PASS == kForward) {
                const int k = kTileI * ks;
                const bool kin = k + 8 * ch < p.I;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    if (kApart * i >= brows) break;
                    const bool in = kin && from[i];
                    cp_async16_or_zero(b + off + i * (kApart * 128), in ? from[i] + k : p.rows, in);
                }
            } else {
                const int first = t.r0 + kTileI * ks, left = end - first;
                const bool tail = left < kTileI;
                const int rows = tail ? (left + 15) & ~15 : kTileI;
                if (tail || picks) {
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        if (kApart * i >= rows) break;
                        const bool in = row[i] >= 0 && m < p.M;
                        cp_async16_or_zero(a + off + i * (kApart * 128), in ? p.rows + int64_t(row[i]) * p.M + m : p.rows,
                                           in);
                    }
                }
                if (tail) {
                    static_assert(C::PASS != kWgrad || C::kBRows == 128, "16 chunks a row");
                    const int n = t.c0 + t.b0 + 8 * ch;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        const int r = row0 + kApart * i;
                        if (kApart * i >= rows) break;
                        const bool in = r < left && n < p.N;
                        cp_async16_or_zero(b + off + i * (kApart * 128), in ? p.dy + int64_t(first + r) * p.N + n : p.dy,
                                           in);
                    }
                }
                next_rows(ks + C::PICK);
            }
            tc::cp_async_arrive_noinc(&s.landed[at.stage]);
        }
    }
    tc::cp_async_wait_all();
    if (!ok) stop(s, p.status);
}

// Relay warp: a stage whose gathered rows have landed is made visible to the
// tensor cores and counted on rank 0's barrier.
template <typename C>
__device__ void relay_stages(const GemmParams &p, GemmSmem &s, Walk<C> walk, int total) {
    const uint32_t full0 = C::CG == 2 ? tc::at_rank(tc::smem_u32(&s.full[0]), 0) : tc::smem_u32(&s.full[0]);
    Ring at(p.stages);
    bool ok = true;
    for (int tau = blockIdx.x / C::CG; tau < total && ok; tau += gridDim.x / C::CG) {
        const int KS = stages_of<C>(p, walk.tile(p, tau));
        for (int ks = 0; ks < KS; ++ks, at.next()) {
            if (!tc::mbar_wait_warp(&s.landed[at.stage], at.phase, kWaitNs)) {
                ok = false;
                break;
            }
            tc::fence_proxy_async();
            if (tc::elect_one()) tc::mbar_arrive_cluster(full0 + at.stage * 8);
            __syncwarp();
        }
    }
    if (!ok) stop(s, p.status);
}

template <typename C>
__device__ void issue_mma(const GemmParams &p, GemmSmem &s, unsigned char *dyn, Walk<C> walk, int total,
                          uint32_t tmem) {
    constexpr bool kMnA = C::PASS != kForward, kMnB = C::PASS == kWgrad;
    // descriptors advance by 16 of the contracted index: 32 bytes in a K-major row, 16 rows of an MN-major block
    constexpr uint64_t kStepA = (kMnA ? 2048 : 32) >> 4, kStepB = (kMnB ? 2048 : 32) >> 4;
    const uint32_t dyn0 = tc::smem_u32(dyn);
    const uint64_t a0 = kMnA ? desc_mn128(dyn0) : tc::desc_sw128(dyn0);
    const uint64_t b0 = kMnB ? desc_mn128(dyn0 + C::kA) : tc::desc_sw128(dyn0 + C::kA);
    const uint32_t fmt = p.bf16 ? 1u : 0u;
    const uint32_t idesc0 = tc::idesc_f16(kTileM * C::CG, 0) | (fmt << 7) | (fmt << 10) | (kMnA ? 1u << 15 : 0u) |
                            (kMnB ? 1u << 16 : 0u);
    auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
        if (C::CG == 2) tc::mma_f16_pair(d, a, b, idesc, acc);
        else tc::mma_f16(d, a, b, idesc, acc);
    };
    auto commit = [](uint64_t *bar) {
        if (C::CG == 2) tc::mma_commit_pair(bar);
        else tc::mma_commit(bar);
    };
    Ring at(p.stages);
    Buffers bufs;
    bool ok = true;
    for (int tau = blockIdx.x / C::CG; tau < total && ok && !s.abort; tau += gridDim.x / C::CG) {
        const Tile t = walk.tile(p, tau);
        const int KS = stages_of<C>(p, t);
        if (KS == 0) continue;  // wgrad of an expert without rows
        const Segments segs = segments_of<C>(p, KS);
        const uint32_t idesc = idesc0 | (uint32_t(t.npad >> 3) << 17);
        const int accs = p.out_fp32 ? C::kAccs : 1;
        int left = C::PASS == kWgrad ? t.rows : p.I;
        for (int seg = 0; seg < segs.count && ok; ++seg) {
            uint32_t phase;
            const int buf = bufs.take(seg, phase), here = min(segs.per, KS - seg * segs.per);
            if (!tc::mbar_wait_warp(&s.tempty[buf], phase ^ 1, kWaitNs)) {
                ok = false;
                break;
            }
            tc::fence_after();
            const uint32_t d0 = tmem + uint32_t(buf * C::kBuf);
            for (int ks = 0; ks < here; ++ks, left -= kTileI, at.next()) {
                if (!tc::mbar_wait_warp(&s.full[at.stage], at.phase, kWaitNs)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint64_t a = a0 + uint32_t(at.stage * (C::kStage >> 4)),
                               b = b0 + uint32_t(at.stage * (C::kStage >> 4));
                const uint32_t d = d0 + uint32_t((ks & (accs - 1)) * C::TN);
                if (tc::elect_one()) {
                    mma(d, a, b, idesc, ks >= accs ? 1u : 0u);
                    if (left > 48) {
                        mma(d, a + kStepA, b + kStepB, idesc, 1u);
                        mma(d, a + 2 * kStepA, b + 2 * kStepB, idesc, 1u);
                        mma(d, a + 3 * kStepA, b + 3 * kStepB, idesc, 1u);
                    } else {  // steps of 16; the last one reads zeros past the end
                        if (left > 16) mma(d, a + kStepA, b + kStepB, idesc, 1u);
                        if (left > 32) mma(d, a + 2 * kStepA, b + 2 * kStepB, idesc, 1u);
                    }
                    commit(&s.empty[at.stage]);
                    if (ks == here - 1) commit(&s.tfull[buf]);
                }
                __syncwarp();
            }
        }
        bufs.turn(segs);
    }
    if (!ok) stop(s, p.status);
}

// Epilogue warps: lane quadrant warp % 4 of tensor memory, every second 32
// columns. Results pass through this warp's 2 KB of shared memory and leave as
// TMA boxes of 32 M and 32 columns (fp32: 16), those of a tile's ragged end as
// plain stores: a box would reach the next expert's rows. An fp32 sum so far
// that is in place is added to by the reduction of the boxes, where they land;
// another one, and one of 16 bits (which is rounded only after the addition),
// comes as the same boxes into 2 KB more, one box ahead of its use.
struct Out {
    const CUtensorMap *out, *base;
    uint64_t *based;      // this warp's barrier for boxes of the sum so far
    uint32_t turn, sum;   // the two 2 KB
    // Lane 0: ask for the box of the sum at column c of tile t.
    __device__ __forceinline__ void want(const Tile &t, int m1, int c) const {
        if ((threadIdx.x & 31) == 0) {
            tc::mbar_arrive_expect_tx(based, kTurn);
            tc::tma_load_3d_at(sum, base, m1, t.c0 + c, t.e, tc::smem_u32(based));
        }
    }
    __device__ __forceinline__ bool got(uint32_t &phase) const {
        const bool ok = tc::mbar_wait_warp(based, phase, kWaitNs);
        phase ^= 1;
        return ok;
    }
    // The buffer's last box has been read by its store.
    __device__ __forceinline__ void free_turn() const {
        if ((threadIdx.x & 31) == 0) tc::bulk_wait_read<0>();
        __syncwarp();
    }
    // The buffer, written by the whole warp, as a box.
    __device__ __forceinline__ void store(int m1, int row, int slab, bool add) const {
        tc::fence_proxy_async();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            if (add) tc::tma_add_3d(out, m1, row, slab, turn);
            else tc::tma_store_3d(out, m1, row, slab, turn);
            tc::bulk_commit();
        }
    }
};

// 16-bit results. 32 x 32 accumulators (lanes M, columns), as fragments of two
// 16-lane halves, are packed along the columns and turned by the transposing
// matrix store into [column][32], 16-byte chunks in the 64-byte swizzle. The
// next 32 columns are on their way while these are stored.
template <typename C, typename O, bool ADD>
__device__ __forceinline__ bool store_tile16(const GemmParams &p, const Out &to, uint32_t &based, const Tile &t,
                                             bool sums, uint32_t td, int half, int m1) {
    const int lane = threadIdx.x & 31;
    const uint32_t at = (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);  // + 512 i: column 8 i + lane % 8
    bool ok = true;
    uint32_t v[2][2][16];
    auto fetch = [&](int c, uint32_t(&f)[2][16]) {
        if (sums && c < t.n) {
            tc::tmem_ld16x256_x4_nowait(td + c, f[0]);
            tc::tmem_ld16x256_x4_nowait(td + c + (16u << 16), f[1]);
        }
    };
    auto put = [&](int c, const uint32_t(&f)[2][16]) {
        uint32_t old[4][4];
        if (ADD) {
            ok = to.got(based) && ok;
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::ldmatrix_x4_trans(to.sum + at + 512 * i, old[i]);
            __syncwarp();
            if (c + 64 < t.n) to.want(t, m1, c + 64);
        }
        to.free_turn();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float lo = __uint_as_float(f[j >> 1][4 * i + 2 * (j & 1)]);
                float hi = __uint_as_float(f[j >> 1][4 * i + 2 * (j & 1) + 1]);
                if (ADD) {
                    const O *o = reinterpret_cast<const O *>(&old[i][j]);
                    lo += to_f32(o[0]);
                    hi += to_f32(o[1]);
                }
                const O pair[2] = {from_f32<O>(lo), from_f32<O>(hi)};
                w[j] = *reinterpret_cast<const uint32_t *>(pair);
            }
            tc::stmatrix_x4_trans(to.turn + at + 512 * i, w[0], w[1], w[2], w[3]);
        }
        if (C::PASS == kWgrad || c + 32 <= t.n) {
            to.store(m1, t.c0 + c, C::PASS == kWgrad ? t.e : 0, false);
        } else {
            __syncwarp();
            const int ch = lane & 3, n0 = lane >> 2;  // 16 bytes a lane; columns 8 apart have the same swizzle
            O *o = static_cast<O *>(p.out) + int64_t(t.c0 + c + n0) * p.M + m1 + 8 * ch;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 r;
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                             : "r"(to.turn + n0 * 64 + ((ch ^ ((n0 >> 1) & 3)) << 4) + i * 512));
                if (m1 + 8 * ch < p.M && c + n0 + 8 * i < t.n)
                    *reinterpret_cast<uint4 *>(o + int64_t(8 * i) * p.M) = r;
            }
        }
    };
    if (!sums)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[0][0][i] = v[0][1][i] = v[1][0][i] = v[1][1][i] = 0u;
    if constexpr (C::PICK == 2) {  // 640 threads have no registers for it
        for (int c = 32 * half; c < t.n; c += 64) {
            fetch(c, v[0]);
            tc::tmem_ld_wait();
            put(c, v[0]);
        }
        return ok;
    }
    fetch(32 * half, v[0]);
    for (int c = 32 * half; c < t.n; c += 128) {
        tc::tmem_ld_wait();
        fetch(c + 64, v[1]);
        put(c, v[0]);
        if (c + 64 < t.n) {
            tc::tmem_ld_wait();
            fetch(c + 128, v[0]);
            put(c + 64, v[1]);
        }
    }
    return ok;
}

// 32 columns of fp32, the sum of `accs` accumulators at td (none: zeros) and of
// `more` at td2.
template <typename C>
__device__ __forceinline__ void fetch32(uint32_t td, int accs, uint32_t td2, int more, uint32_t (&v)[32]) {
    if (accs == 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0u;
        return;
    }
    tc::tmem_ld32_nowait(td, v);
    tc::tmem_ld_wait();
    for (int a = 1; a < accs + more; ++a) {
        const uint32_t from = a < accs ? td + uint32_t(a * C::TN) : td2 + uint32_t((a - accs) * C::TN);
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            uint32_t u[16];
            tc::tmem_ld16_nowait(from + h, u);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[h + i] = __float_as_uint(__uint_as_float(v[h + i]) + __uint_as_float(u[i]));
        }
    }
}

// Adds this warp's values of the `accs` accumulators at from to those at td, in
// tensor memory, rounding to nearest.
template <typename C>
__device__ __forceinline__ void add_segment(uint32_t td, uint32_t from, int accs, int n, int half) {
    for (int a = 0; a < accs; ++a)
        for (int c = a * C::TN + 32 * half; c < a * C::TN + n; c += 64)
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                uint32_t v[16], u[16];
                tc::tmem_ld16_nowait(td + c + h, v);
                tc::tmem_ld16_nowait(from + c + h, u);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
                tc::tmem_st16(td + c + h, v);
            }
    tc::tmem_st_wait();
}

// fp32 results, [column][32], 16 columns at a time.
template <typename C, bool ADD>
__device__ __forceinline__ bool store_tile32(const GemmParams &p, const Out &to, uint32_t &based, const Tile &t,
                                             int accs, uint32_t td, int more, uint32_t td2, int half, int m1) {
    const int lane = threadIdx.x & 31, m = m1 + lane;
    bool ok = true;
    float *o = static_cast<float *>(p.out) + int64_t(t.c0) * p.M + m;
    for (int c = 32 * half; c < t.n; c += 64) {
        uint32_t v[32];
        fetch32<C>(td + c, accs, td2 + c, more, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c1 = c + 16 * h;
            if (c1 >= t.n) break;
            if (ADD) {
                ok = to.got(based) && ok;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float old;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(old) : "r"(to.sum + i * 128 + lane * 4));
                    v[16 * h + i] = __float_as_uint(__uint_as_float(v[16 * h + i]) + old);
                }
                __syncwarp();
                const int next = h ? c + 64 : c1 + 16 < t.n ? c1 + 16 : c + 64;
                if (next < t.n) to.want(t, m1, next);
            }
            if (C::PASS == kWgrad || c1 + 16 <= t.n) {
                to.free_turn();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to.turn + i * 128 + lane * 4), "r"(v[16 * h + i])
                                 : "memory");
                to.store(m1, t.c0 + c1, C::PASS == kWgrad ? t.e : 0, C::PASS == kWgrad && p.base && !ADD);
            } else if (m < p.M) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c1 + i < t.n) o[int64_t(c1 + i) * p.M] = __uint_as_float(v[16 * h + i]);
            }
        }
    }
    return ok;
}

template <typename C, typename O, bool ADD>
__device__ void store_tiles(const GemmParams &p, GemmSmem &s, const GemmMaps &maps, unsigned char *dyn, Walk<C> walk,
                            int total, uint32_t tmem) {
    const int warp = (threadIdx.x >> 5) - kEpiWarp0, lane = threadIdx.x & 31;
    const int q = (warp + kEpiWarp0) & 3, half = warp >> 2;
    const uint32_t turn = tc::smem_u32(dyn) + p.stages * C::kStage + warp * kTurn;
    const Out to = {&maps.out, &maps.base, &s.based[warp], turn, turn + kEpiWarps * kTurn};
    uint32_t based = 0;
    Buffers bufs;
    for (int tau = blockIdx.x / C::CG; tau < total && !s.abort; tau += gridDim.x / C::CG) {
        const Tile t = walk.tile(p, tau);
        const int KS = stages_of<C>(p, t);
        // (forward's and dgrad's 16-bit results: N and K stop at 16384)
        constexpr bool kMany = sizeof(O) == 4 || C::PASS == kWgrad;
        const Segments segs = kMany ? segments_of<C>(p, KS) : Segments{1, KS};
        const int m1 = t.m0 + 32 * q;
        const bool any = m1 < p.M && 32 * half < t.n;  // of this warp's values lie in the result
        if (ADD && any) to.want(t, m1, 32 * half);
        const uint32_t quad = tmem + (uint32_t(32 * q) << 16);
        auto filled = [&](int b, uint32_t phase) {
            // a segment of many stages may rightly take longer than one wait
            const bool ok = tc::mbar_wait_warp(&s.tfull[b], phase, kWaitNs + 2000ull * segs.per);
            tc::fence_after();
            return ok;
        };
        auto release = [&](int b) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = tc::smem_u32(&s.tempty[b]);
                tc::mbar_arrive_cluster(C::CG == 2 ? tc::at_rank(bar, 0) : bar);
            }
        };
        bool ok = true;
        int buf = 0, last = 0, accs = 0, more = 0;  // more: accumulators of the last segment, still in their buffer
        if (KS > 0) {
            uint32_t phase;
            buf = bufs.take(0, phase);
            accs = accs_of<C>(p, segs.per);
            ok = filled(buf, phase);
            for (int seg = 1; kMany && seg < segs.count && ok; ++seg) {
                last = bufs.take(seg, phase);
                ok = filled(last, phase);
                const int here = accs_of<C>(p, min(segs.per, KS - seg * segs.per));
                if (sizeof(O) == 4 && seg == segs.count - 1) {
                    more = here;
                } else {
                    if (ok && any) add_segment<C>(quad + buf * C::kBuf, quad + last * C::kBuf, here, t.n, half);
                    release(last);
                }
            }
            bufs.turn(segs);
        }
        const uint32_t td = quad + uint32_t(buf * C::kBuf), td2 = quad + uint32_t(last * C::kBuf);
        if (ok && any) {
            if constexpr (sizeof(O) == 2) ok = store_tile16<C, O, ADD>(p, to, based, t, accs > 0, td, half, m1);
            else ok = store_tile32<C, ADD>(p, to, based, t, accs, td, more, td2, half, m1);
        }
        if (!ok) {  // no box may land after this CTA's shared memory has another owner
            stop(s, p.status);
            if (ADD && any) to.got(based);
            break;
        }
        if (accs) release(buf);
        if (more) release(last);
    }
    if (lane == 0) tc::bulk_wait_read<0>();
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ GemmMaps maps) {
    extern __shared__ __align__(1024) unsigned char dyn_raw[];
    unsigned char *dyn =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    __shared__ GemmSmem s;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rank = C::CG == 2 ? int(tc::cluster_rank()) : 0;
    const int MT = (p.M + kTileM * C::CG - 1) / (kTileM * C::CG);
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            tc::mbar_init(&s.full[i], 1 + (C::PICK ? C::CG : 0));
            tc::mbar_init(&s.empty[i], 1);
            tc::mbar_init(&s.landed[i], kPickThreads);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.tfull[i], 1);
            tc::mbar_init(&s.tempty[i], C::CG * kEpiWarps);
        }
        for (int i = 0; i < kEpiWarps; ++i) tc::mbar_init(&s.based[i], 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if (C::CG == 2) tc::tmem_alloc_pair(&s.tmem_base, C::kCols);
        else tc::tmem_alloc(&s.tmem_base, C::kCols);
    }
    after_previous();
    Entry *table = reinterpret_cast<Entry *>(dyn + p.stages * C::kStage + kEpiWarps * kTurn * (1 + p.read_base));
    const int total = build_table<C>(p, s, table, MT);
    tc::fence_before();
    if (C::CG == 2) tc::cluster_sync();  // both CTAs' barriers are set up
    else __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s.tmem_base;
    const Walk<C> walk(s, table, MT, rank);
    if (warp == kLoadWarp) {
        load_tiles<C>(p, s, maps, dyn, walk, total);
    } else if (warp == kMmaWarp) {
        if (rank == 0) issue_mma<C>(p, s, dyn, walk, total, tmem);
    } else if (warp >= kPickWarp0) {
        if constexpr (C::PICK) {
            if (warp == C::kRelayWarp) relay_stages<C>(p, s, walk, total);
            else gather_tiles<C>(p, s, dyn, walk, total);
        }
    } else {
        auto store = [&](auto add) {
            constexpr bool kAdd = decltype(add)::value;
            if (p.out_fp32) store_tiles<C, float, kAdd>(p, s, maps, dyn, walk, total, tmem);
            else if (p.bf16) store_tiles<C, __nv_bfloat16, kAdd>(p, s, maps, dyn, walk, total, tmem);
            else store_tiles<C, __half, kAdd>(p, s, maps, dyn, walk, total, tmem);
        };
        if (C::PASS == kWgrad && p.read_base) store(std::integral_constant<bool, C::PASS == kWgrad>());
        else store(std::false_type());
    }
    __syncwarp();
    tc::fence_before();
    if (C::CG == 2) tc::cluster_sync();  // neither leaves while the other's products or arrivals may reach it
    else __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        if (C::CG == 2) tc::tmem_dealloc_pair(tmem, C::kCols);
        else tc::tmem_dealloc(tmem, C::kCols);
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

// 16-bit tensor of up to 4 dimensions (innermost first, strides in elements) in
// boxes 64 wide, 128-byte swizzle, zeros outside.
bool map16(CUtensorMap *m, bool bf16, const void *base, int rank, const int64_t (&extent)[4], const int64_t (&stride)[4],
           const uint32_t (&box)[4]) {
    cuuint64_t dims[4], strides[3];
    cuuint32_t b[4], es[4];
    for (int i = 0; i < rank; ++i) {
        dims[i] = cuuint64_t(extent[i]);
        if (i) strides[i - 1] = cuuint64_t(stride[i]) * 2;
        b[i] = box[i];
        es[i] = 1;
    }
    return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                    const_cast<void *>(base), dims, strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The result [slabs][rows][inner], boxes of 32 x 32 16-bit values (64-byte
// swizzle) or 16 x 32 fp32 ones.
bool map_out(CUtensorMap *m, bool bf16, bool fp32, const void *base, int64_t inner, int64_t rows, int64_t slabs) {
    const cuuint64_t size = fp32 ? 4 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(slabs)};
    const cuuint64_t strides[2] = {cuuint64_t(inner) * size, cuuint64_t(inner) * cuuint64_t(rows) * size};
    const cuuint32_t box[3] = {32, fp32 ? 16u : 32u, 1}, es[3] = {1, 1, 1};
    return g_encode(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                            : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    3, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    fp32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// rows x inner, boxes of box_rows x 64.
bool map_rows(CUtensorMap *m, bool bf16, const void *base, int64_t inner, int64_t rows, int box_rows) {
    return map16(m, bf16, base, 2, {inner, rows, 1, 1}, {1, inner, 0, 0}, {64, uint32_t(box_rows), 1, 1});
}
// rows x inner as 64-wide blocks (inner a multiple of 64), boxes of two blocks x 64 rows.
bool map_blocks(CUtensorMap *m, bool bf16, const void *base, int64_t inner, int64_t rows) {
    return map16(m, bf16, base, 3, {64, rows, inner / 64, 1}, {1, inner, 64, 0}, {64, 64, 2, 1});
}

// encode fills in the tensor maps. It is a driver call, which takes the context
// that the attribute's call before it has made current to this host thread.
template <typename C, typename Encode>
moe_status launch(GemmParams &p, const Encode &encode, int64_t most_tiles, int sms, cudaStream_t stream) {
    p.stages = C::stages(p.E, p.read_base);
    const size_t smem = p.stages * C::kStage + C::fixed(p.E, p.read_base);
    if (!allow_smem(expert_gemm_kernel<C>, kMaxDynamic)) return MOE_ERR_CUDA;
    GemmMaps maps;
    if (!encode(maps)) return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(sms / C::CG, most_tiles)) * C::CG);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    void *args[] = {&p, &maps};
    if (launch_early(cfg, attrs, C::CG, reinterpret_cast<const void *>(expert_gemm_kernel<C>), args) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

// rows: a (forward, wgrad) or dy (dgrad).
moe_status run_gemm(int pass, GemmParams &p, const void *w, int N, int K, cudaStream_t stream) {
    int sms = 0;
    if (!host_setup(sms)) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const bool bf = p.bf16, pick = p.sorted_tok != nullptr;
    const int64_t experts = std::min<int64_t>(p.E, p.P);
    // Few rows an expert: the weights' bytes bound the call, so tiles are narrow
    // and single, with more stages of weights in flight and more of them.
    const bool narrow = pass != kWgrad && p.P <= 16 * experts;
    // One box of two blocks instead of two loads (90 cycles of the issuing
    // thread each), where the extent along MN has no ragged last block.
    p.blocks2 = pass == kWgrad ? N % 64 == 0 && K % 64 == 0 : pass == kDgrad && K % 64 == 0;
    p.read_base = p.base && (!p.out_fp32 || p.base != p.out);
    auto encode = [&](GemmMaps &maps) {
        bool ok = pass == kWgrad ? map_out(&maps.out, bf, p.out_fp32, p.out, K, N, p.E)
                                 : map_out(&maps.out, bf, p.out_fp32, p.out, p.M, p.P, 1);
        if (p.read_base) ok = ok && map_out(&maps.base, bf, p.out_fp32, p.base, K, N, p.E);
        if (p.P > 0) {  // an empty batch (wgrad) has no rows to describe, and loads none
            if (pass == kForward)
                ok = ok && map16(&maps.w, bf, w, 3, {K, N, p.E, 1}, {1, K, int64_t(N) * K, 0}, {64, 128, 1, 1});
            else if (pass == kDgrad)
                ok = ok && (p.blocks2
                                ? map16(&maps.w, bf, w, 4, {64, N, K / 64, p.E}, {1, K, 64, int64_t(N) * K}, {64, 64, 2, 1})
                                : map16(&maps.w, bf, w, 3, {K, N, p.E, 1}, {1, K, int64_t(N) * K, 0}, {64, 64, 1, 1}));
            else
                ok = ok && (p.blocks2 ? map_blocks(&maps.dy, bf, p.dy, N, p.P) : map_rows(&maps.dy, bf, p.dy, N, p.P, 64));
            if (!pick && pass == kWgrad)
                ok = ok && (p.blocks2 ? map_blocks(&maps.rows[0], bf, p.rows, K, p.rows_a)
                                      : map_rows(&maps.rows[0], bf, p.rows, K, p.rows_a, 64));
            if (!pick && pass != kWgrad)
                for (int i = 0; i < (narrow ? 2 : kBoxes); ++i)
                    ok = ok && map_rows(&maps.rows[i], bf, p.rows, p.I, p.rows_a, box_rows(i));
        }
        return ok;
    };
    const int64_t MT1 = (p.M + kTileM - 1) / kTileM, MT2 = (MT1 + 1) / 2;
    if (pass == kWgrad)
        return launch<Cfg<kWgrad, 2, 256, 1>>(p, encode, MT2 * ((N + 255) / 256) * p.E, sms, stream);
    if (narrow) {
        const int64_t most = MT1 * (experts + p.P / 32);
        if (pass == kDgrad) return launch<Cfg<kDgrad, 1, 32, 0>>(p, encode, most, sms, stream);
        return pick ? launch<Cfg<kForward, 1, 32, 2>>(p, encode, most, sms, stream)
                    : launch<Cfg<kForward, 1, 32, 0>>(p, encode, most, sms, stream);
    }
    const int64_t most = MT2 * (experts + p.P / 256);
    if (pass == kDgrad) return launch<Cfg<kDgrad, 2, 256, 0>>(p, encode, most, sms, stream);
    return pick ? launch<Cfg<kForward, 2, 256, 2>>(p, encode, most, sms, stream)
                : launch<Cfg<kForward, 2, 256, 0>>(p, encode, most, sms, stream);
}

moe_status check_gemm(int dtype, int T, int E, int k, int N, int K, int out_dtype) {
    if (T < 0 || E <= 0 || k <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (!half_type(dtype) || !out_type_ok(dtype, out_dtype)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED;
    if (N % 8 || K % 8 || N > 2 * kMaxDim || K > 2 * kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (int64_t(T) * k > kMaxPairs) return MOE_ERR_OVERFLOW;
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
    GemmParams p = {offsets, sorted_tok, static_cast<const uint16_t *>(a), nullptr, nullptr, out, sorted_tok ? T : T * k,
                    T * k, E, N, K, 0, dtype == MOE_BF16, out_dtype == MOE_FP32, 0, 0, 0, dev_status};
    return run_gemm(kForward, p, W, N, K, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_dgrad(const void *dy, const void *W, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, void *da, int out_dtype, int32_t *dev_status,
                                         moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK || T == 0) return st;
    if (!dy || !W || !offsets || !da || !aligned16(dy) || !aligned16(W) || !aligned16(da)) return MOE_ERR_INVALID_ARG;
    GemmParams p = {offsets, nullptr, static_cast<const uint16_t *>(dy), nullptr, nullptr, da,
                    T * k, T * k, E, K, N, 0, dtype == MOE_BF16, out_dtype == MOE_FP32, 0, 0, 0, dev_status};
    return run_gemm(kDgrad, p, W, N, K, as_cuda(stream));
}

MOE_API moe_status moe_expert_gemm_wgrad(const void *dy, const void *a, int dtype, int T, int E, int k, int N, int K,
                                         const int32_t *offsets, const int32_t *sorted_tok, const void *base,
                                         void *dW, int out_dtype, int32_t *dev_status, moe_stream_t stream) {
    const moe_status st = check_gemm(dtype, T, E, k, N, K, out_dtype);
    if (st != MOE_OK) return st;
    if (!offsets || !dW || !aligned16(dW) || !aligned16(base)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !a || !aligned16(dy) || !aligned16(a))) return MOE_ERR_INVALID_ARG;
    GemmParams p = {offsets, sorted_tok, static_cast<const uint16_t *>(a), static_cast<const uint16_t *>(dy), base, dW,
                    sorted_tok ? T : T * k, T * k, E, K, 0, N, dtype == MOE_BF16, out_dtype == MOE_FP32, 0, 0, 0,
                    dev_status};
    return run_gemm(kWgrad, p, nullptr, N, K, as_cuda(stream));
}
