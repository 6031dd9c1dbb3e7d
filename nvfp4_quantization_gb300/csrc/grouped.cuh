// Matrix products grouped by expert, on the tensor cores: the kernel behind
// ep_grouped_gemm, ep_grouped_wgrad and their NVFP4 forms.
//
// Rows lie in expert order, expert e's in [off_e, off_e + n_e).  Two shapes:
//   rows as N (kWgrad false):  y[r][m] = sum_k w_e[m][k] x[r][k].  The weights
//     are the M side of the matrix instruction and the rows its N side, whose
//     size may change from tile to tile: a slot of 128 rows costs 128, not 256.
//   rows as K (kWgrad true):   d_w[e][m][n] = sum_r dy[r][m] x[r][n].
//
// A persistent kernel: one CTA a SM, tiles of 128 x kCtas by up to 256 dealt
// out in turn.  Warps 0-7 take finished sums from tensor memory to global memory
// while the next tile is computed in the other half of tensor memory; warp 8
// feeds a ring of shared-memory stages by TMA (128 bytes along K a row and
// stage: 64 BF16 or 256 E2M1), one thread of warp 9 issues the matrix products
// into tensor memory, warp 10 cuts ragged blocks.
//
// The columnwise NVFP4 operands are a matrix of its own for every expert, whose
// pitch only the device knows, so no tensor map of the host's fits them.  There
// warps 12-15 copy the rows in 16-byte pieces, and warp 8 (in a pair's second
// CTA warps 8-10 in turn) passes the arrival of a stage on to the matrix products.
//
// What bounds it (times of calls back to back for seconds, "alone" of one call
// after a pause).  Large BF16 products: the tensor cores (busy 97 % of the time on
// 8192 x 8192 x 4096), and with them the card's power: 8192^3 runs at 1.86 PFLOP/s
// alone and 1.68 for seconds on end, where torch.matmul has 1.86 and 1.73.  NVFP4
// products of packed rows: the copies into shared memory, two lines to every 128
// bytes: 4.6 PFLOP/s (98304 rows, 64 experts of 4096 x 4096: 716 us, 705 alone).
// Of rows that start on a line: 5.3 (621 us, 582 alone), then at the power limit.
// Copies of the block scales to tensor memory cost the products a quarter of their
// rate where the tile has 128 columns, little where it has 256.  Small batches:
// reading the weights (128 tokens, 8 of 64 experts of 4096 x 4096: NVFP4 118 us, 5.2
// TB/s; BF16 344 us, 6.2 TB/s).  Weight gradients with few rows an expert: writing
// them (1536 rows, NVFP4, FP32 out, 64 experts of 2048 x 4096: 335 us, 6.4 TB/s).
// With many, in NVFP4: not that (98304 rows: 545 us, where a fill of the results
// takes 278), but copying rows by threads, which keeps the matrix unit waiting (busy
// a third of the time).  Adding to FP32 results: reading and writing them (the same,
// 915 us, 5.1 TB/s).
//
// Why it is as it is, each step against the state before (98304 rows, 64 experts
// of 4096 x 4096, BF16 / NVFP4):
//  - CTA pairs, tiles of 256 x 256: a CTA reads half of the N side and the matrix
//    unit the other half from its neighbour.  One CTA a tile is within 6 % of the
//    pair's time for BF16, but takes 1.36 times it for NVFP4.
//  - instructions that take uniform registers (copies, products) under an elected
//    thread (umma.cuh): 2.19 / 1.18 ms -> 1.88 / 0.69.
//  - the next tiles worked out 32 at a time, a lane each: a change of tiles made
//    the products pause for about 0.5 us before.
//  - accumulators of 256 columns twice, so that a tile is written while the next
//    is computed.  Block scales take 48 columns; there the two overlap in 64,
//    which are emptied first and waited for only where both tiles use them
//    (1021 tokens, 5 of 61 experts of 2056 x 1056: 31.9 -> 28.7 us with the next
//    step).
//  - eight warps for the epilogue, one piece of output each: with two pieces a
//    warp, and so a stage less, the weight gradients took 5 to 9 % longer.
//  - measured and dropped: tiles of 128 columns for pairs with short slots, with
//    more stages (128 tokens, 8 of 64 experts of 4096 x 4096: BF16 354 -> 344 us,
//    NVFP4 no change; 56.5 -> 59.4 us where a few slots are longer); hints to L2
//    for what is written or read, and other sizes of its fetches (no change);
//    block scales copied as 64-bit words in one piece (no change); a register
//    split between the warps (the epilogue spilled more, not less).
#pragma once

#include "epq_internal.h"
#include "umma.cuh"

namespace epq {

constexpr int kGroupTiles = 8;       // tiles of the N side that share the M side's tiles in L2
constexpr int kOutWarps = 8;         // two to a quarter of the accumulator's lanes
constexpr int kWarpCopy = 8, kWarpMma = 9, kWarpCut = 10, kWarpRows = 12, kRowWarps = 4;
// Warps of a pair's second CTA that pass on what its threads copied (from
// kWarpCopy on; the products and cut blocks of that CTA are not theirs).  Their
// arrivals release at cluster scope, which takes longer than a stage: one warp
// held the NVFP4 weight gradient of 98304 rows (64 experts of 2048 x 4096) at 642
// us and that of 65536 (8 of 4096 x 4096) at 697, two 541 and 504, three 539 and
// 498, four 539 and 496.
constexpr int kPassers = 3;
constexpr uint64_t kWaitNs = 2000000000ull;

enum { kMapA = 0, kMapB = 1, kMapSa = 2, kMapSb = 3 };

struct GroupedParams {
    CUtensorMap map[4];              // A, B, block scales of A and B
    CUtensorMap out;
    const uint8_t *col[4];           // NVFP4 weight gradient: the same, as the columnwise operands
    const int32_t *offsets;          // [E + 1], or NULL: one expert with all R_cap rows
    const int32_t *counts;           // BF16 weight gradient: [E] or NULL
    const float *m_scale;            // NVFP4: rows as N: [E * M] of the weights' rows; rows as K: [E] of dy
    const float *n_scale;            //        [R_cap] of the rows;                     [E] of x
    uint32_t *status;
    int R_cap, E;
    int M, N, K;                     // rows as N: M features, K; rows as K: M x N
    int add;                         // rows as K, FP32: add to d_w
};

template <bool kFp4_, bool kWgrad_, bool kAmn_, int kCtas_, bool kF32_> struct GroupedCfg {
    static constexpr bool kFp4 = kFp4_, kWgrad = kWgrad_, kF32 = kF32_;
    static constexpr int kCtas = kCtas_;                      // that compute a tile: one or a pair
    // columns of a tile: where single CTAs take a product, slots are short and
    // stages in flight count
    static constexpr int kTileN = kCtas == 1 && !kWgrad ? 128 : 256;
    static constexpr int kSpan = 128 * kCtas;                 // of the M side
    static constexpr bool kAmn = kAmn_;                       // A with its M side contiguous (BF16)
    static constexpr bool kRows = kFp4 && kWgrad;             // copied in pieces, not by TMA
    static constexpr int kThreads = kRows ? 32 * (kWarpRows + kRowWarps) : 352;
    static constexpr bool kBmn = kWgrad && !kFp4;
    static constexpr int kBlockK = kFp4 ? 256 : 64;           // elements of K a stage
    static constexpr int kStepK = kFp4 ? 64 : 16;             // elements of K a matrix instruction
    static constexpr uint32_t kABytes = 128 * 128;
    static constexpr uint32_t kBBytes = kTileN / kCtas * 128;
    static constexpr uint32_t kSaBytes = kFp4 ? 2048 : 0;
    static constexpr uint32_t kSbBytes = kFp4 ? kTileN / 128 * 2048 : 0;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
    static constexpr uint32_t kOutBytes = kWgrad ? 4096 : 2048;   // a warp's piece of a tile
    static constexpr uint32_t kOutAll = kOutWarps * kOutBytes;
    static constexpr uint32_t kPlan = 2560;                       // barriers and tile counts of 1024 experts
    static constexpr uint32_t kRest = kOutAll + kPlan;
    static constexpr int kStages = (int)((232448 - kRest) / kStageBytes);
    // tensor memory: two accumulators of 256 columns; with block scales the two
    // overlap in 64 columns, which are emptied first
    static constexpr uint32_t kAcc1 = kFp4 ? 192 : 256;
    static constexpr uint32_t kSaCol = 448, kSbCol = 464;
    static constexpr int kChunk = kWgrad && !kF32 ? 64 : 32;      // columns that the epilogue takes at a time
    // FP32 outputs: a sum is taken out of tensor memory after this many blocks of K
    // and its parts added up in FP32.  The matrix unit truncates as it adds, so its
    // error grows with its additions: over 2048 rows of BF16 (128 additions) 2.1e-6
    // of the result, over 65536 7.6e-5; in parts of 768 rows 6.8e-7 and 7.5e-7.
    // NVFP4 loses less (16384 rows 2.0e-6, in parts of 8192 8.2e-7).  BF16 keeps
    // its parts in registers (4 % of a step with 2048 rows an expert; the 128 of them
    // leave about 240 bytes a thread that are spilled), NVFP4, where there is seldom
    // more than one, adds them in global memory.
    static constexpr bool kParts = kWgrad && kF32, kKeep = kParts && !kFp4;
    static constexpr int kPartBlocks = kFp4 ? 32 : 12;
};

struct __align__(8) GroupedBars {      // up to 8 stages
    uint64_t full[8], empty[8], tail[8];        // tail: what landed here, before it is passed on
    uint64_t acc_full[2], acc_empty[2], acc_shared;
    uint32_t tmem, pad;
};

template <class C> constexpr uint32_t grouped_smem_bytes()
{
    return C::kRest + C::kStages * C::kStageBytes;
}

// A tile: its expert, the expert's rows, where it lies and its steps.
struct GroupedTile {
    int e, row0, rows;    // the expert's first row and number of rows (rows as N: of this tile)
    int m0, n0;           // first row of the M side (of the pair), first of the N side
    int n;                // columns of the N side
    int kb;               // blocks of K
};

template <class C>
__device__ __forceinline__ int expert_rows(const GroupedParams &p, int e, int &off, uint32_t &err)
{
    if (!p.offsets) {
        off = 0;
        return p.R_cap;
    }
    off = ld_word(p.offsets + e);
    const int end = ld_word(p.offsets + e + 1);
    if (off < 0 || end < off || ((off | end) & 127)) {
        err |= kDevErrBadExpert;
        return 0;
    }
    if (end > p.R_cap) {
        err |= kDevErrCapacity;      // the columnwise layout of a cut slot is not known: none of it
        return C::kRows ? 0 : max(0, p.R_cap - off);
    }
    return end - off;
}

template <class C> __device__ __forceinline__ int m_tiles(const GroupedParams &p)
{
    return (p.M + C::kSpan - 1) / C::kSpan;
}

template <class C>
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedParams &p, const int *start, int t)
{
    GroupedTile o = {};
    if (t >= start[(p.E + 1) >> 1])
        return o;
    int lo = 0, hi = (p.E - 1) >> 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    uint32_t err = 0;
    const int mt = m_tiles<C>(p);
    int j = t - start[lo];
    o.e = 2 * lo;
    int rows = expert_rows<C>(p, o.e, o.row0, err);
    int nt = ((C::kWgrad ? p.N : rows) + C::kTileN - 1) / C::kTileN;
    if (j >= mt * nt) {
        j -= mt * nt;
        rows = expert_rows<C>(p, ++o.e, o.row0, err);
        nt = ((C::kWgrad ? p.N : rows) + C::kTileN - 1) / C::kTileN;
    }
    // groups of kGroupTiles tiles of the N side; in a group they change fastest
    const int g = j / (kGroupTiles * mt), in = j - g * kGroupTiles * mt;
    const int gn = min(kGroupTiles, nt - g * kGroupTiles);
    const int mi = in / gn, ni = g * kGroupTiles + in - mi * gn;
    o.m0 = mi * C::kSpan;
    o.n0 = ni * C::kTileN;
    if (C::kWgrad) {
        o.rows = rows;
        if (p.counts)
            o.rows = max(0, min(rows, ld_word(p.counts + o.e)));
        o.n = min(C::kTileN, p.N - o.n0);
        o.kb = (o.rows + C::kBlockK - 1) / C::kBlockK;
    } else {
        o.rows = o.n = min(C::kTileN, rows - o.n0);
        o.kb = (p.K + C::kBlockK - 1) / C::kBlockK;
    }
    return o;
}

// The tiles of one CTA (pair) in order, for a whole warp: each lane works out
// one of the next 32, so that a change of tiles costs a few shuffles (worked
// out one by one the products paused for about 0.5 us a tile).
template <class C> struct GroupedWalk {
    const GroupedParams &p;
    const int *start;
    int next, step, i;
    GroupedTile mine;

    __device__ __forceinline__ GroupedWalk(const GroupedParams &p_, const int *start_, int first, int step_)
        : p(p_), start(start_), next(first), step(step_), i(32)
    {
    }

    __device__ __forceinline__ GroupedTile tile()
    {
        if (i == 32) {
            mine = grouped_tile<C>(p, start, next + step * (int)(threadIdx.x & 31));
            next += 32 * step;
            i = 0;
        }
        GroupedTile o;
        o.e = __shfl_sync(0xffffffffu, mine.e, i);
        o.row0 = __shfl_sync(0xffffffffu, mine.row0, i);
        o.rows = __shfl_sync(0xffffffffu, mine.rows, i);
        o.m0 = __shfl_sync(0xffffffffu, mine.m0, i);
        o.n0 = __shfl_sync(0xffffffffu, mine.n0, i);
        o.n = __shfl_sync(0xffffffffu, mine.n, i);
        o.kb = __shfl_sync(0xffffffffu, mine.kb, i);
        ++i;
        return o;
    }
};

// Tiles before every second expert, and all of them, in shared memory; what is
// wrong with the offsets goes to the status word.
template <class C>
__device__ __forceinline__ void grouped_plan(const GroupedParams &p, int *start, int *partial)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = 4;                       // experts of a thread: 1024 and more in all
    const int e0 = tid * kPer, mt = m_tiles<C>(p);
    uint32_t err = 0;
    int n[kPer], mine = 0, off;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int rows = e0 + i < p.E ? expert_rows<C>(p, e0 + i, off, err) : 0;
        n[i] = e0 + i < p.E ? mt * (((C::kWgrad ? p.N : rows) + C::kTileN - 1) / C::kTileN) : 0;
        mine += n[i];
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d)
            sum += v;
    }
    if (lane == 31)
        partial[warp] = sum;
    __syncthreads();
    int at = sum - mine;
    for (int w = 0; w < warp; ++w)
        at += partial[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if ((i & 1) == 0 && e0 + i < p.E)
            start[(e0 + i) >> 1] = at;
        at += n[i];
    }
    if (tid == C::kThreads - 1)
        start[(p.E + 1) >> 1] = at;               // the last thread has no expert
    if (err && blockIdx.x == 0)
        raise_status(p.status, err);
}

// A place in the ring of stages.
template <int kStages> struct GroupedRing {
    uint32_t s = 0, phase = 0;
    __device__ __forceinline__ void step()
    {
        if (++s == kStages) {
            s = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ GroupedRing before(uint32_t n) const      // n <= kStages
    {
        GroupedRing r = *this;
        if (r.s < n) {
            r.s += kStages;
            r.phase ^= 1;
        }
        r.s -= n;
        return r;
    }
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) grouped_kernel(const __grid_constant__ GroupedParams p)
{
    constexpr int kCtas = C::kCtas, kStages = C::kStages;
    extern __shared__ __align__(1024) uint8_t g_smem[];          // stages, pieces of output, barriers, plan
    uint8_t *const base = g_smem;
    const uint32_t ring = smem_u32(base);
    uint8_t *const out_s = base + kStages * C::kStageBytes;
    GroupedBars &bar = *reinterpret_cast<GroupedBars *>(out_s + C::kOutAll);
    int *const partial = reinterpret_cast<int *>(&bar + 1);      // [C::kThreads / 32]
    int *const start = partial + C::kThreads / 32;               // [(E + 1) / 2 + 1]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
    const int unit = (int)blockIdx.x / kCtas, units = (int)gridDim.x / kCtas;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar.full[s], kCtas);
            mbar_init(&bar.empty[s], 1);
            mbar_init(&bar.tail[s], C::kRows ? 32 * kRowWarps : 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar.acc_full[b], 1);
            mbar_init(&bar.acc_empty[b], kOutWarps * kCtas);
        }
        mbar_init(&bar.acc_shared, kOutWarps * kCtas);
        fence_mbar_init();
    }
    if (warp == kWarpCut)
        tmem_alloc<kCtas>(smem_u32(&bar.tmem), 512);
    pdl_launch_dependents();
    pdl_wait();
    grouped_plan<C>(p, start, partial);
    tmem_fence_before();
    if constexpr (kCtas == 2)
        cluster_sync();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bar.tmem;
    const int tiles = start[(p.E + 1) >> 1];
    // barriers that the products wait on: the leader's
    auto at_leader = [&](uint64_t *b) { return kCtas == 2 ? at_rank(smem_u32(b), 0) : smem_u32(b); };
    const uint32_t full0 = at_leader(&bar.full[0]);
    // after writes to this CTA's stage s by threads
    auto arrive_at_leader = [&](uint32_t s) {
        if (rank == 0)
            mbar_arrive(&bar.full[s]);
        else
            mbar_arrive_release_at(full0 + 8 * s);
    };
    bool ok = true;
    GroupedWalk<C> walk(p, start, unit, units);

    if (C::kRows && warp >= kWarpCopy && warp < kWarpCopy + (rank == 0 ? 1 : kPassers)) {
        // ------------------------------------------------------------ arrivals
        // what the other threads copied, ordered before the matrix unit's reads;
        // each passing warp has every `passers`-th stage
        const int passers = rank == 0 ? 1 : kPassers, first = warp - kWarpCopy;
        GroupedRing<kStages> at;
        int turn = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            const GroupedTile o = walk.tile();
            for (int kb = 0; kb < o.kb; ++kb) {
                if (turn == first) {
                    ok = __all_sync(0xffffffffu, mbar_wait_for(&bar.tail[at.s], at.phase, kWaitNs));
                    if (!ok)
                        break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        arrive_at_leader(at.s);
                }
                turn = turn + 1 == passers ? 0 : turn + 1;
                at.step();
            }
        }
    } else if (C::kRows && warp >= kWarpRows) {
        // ------------------------------------------------------------ rows
        const int id = tid - 32 * kWarpRows, c = id & 7, r0 = id >> 3;   // piece of a row; first of every 16 rows
        GroupedRing<kStages> at;
        uint32_t used = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            const GroupedTile o = walk.tile();
            // M and N are multiples of 128 here, so a tile's rows on either side are
            // there or not as a whole.  What is not there is not copied and not used:
            // lanes past M are not stored, steps past a row's end are not made.
            const int half = o.n / kCtas, m = o.m0 + 128 * (int)rank, n = o.n0 + half * (int)rank;
            const bool have_a = m < p.M;
            const int64_t pitch = o.rows / 2, blocks = (int64_t)o.rows * 8;    // bytes of a row, of 128 rows' scales
            const int64_t pitch16 = 16 * pitch;
            const uint8_t *ca = p.col[kMapA] + (int64_t)o.row0 * p.M / 2 + (m + r0) * pitch + 16 * c;
            const uint8_t *cb = p.col[kMapB] + (int64_t)o.row0 * p.N / 2 + (n + r0) * pitch + 16 * c;
            const uint8_t *sa = p.col[kMapSa] + (int64_t)o.row0 * p.M / 16 + m / 128 * blocks + 16 * id;
            const uint8_t *sb = p.col[kMapSb] + (int64_t)o.row0 * p.N / 16 + o.n0 / 128 * blocks + 16 * id;
            const uint32_t to = 128 * r0 + ((c ^ (r0 & 7)) << 4);       // 128-byte swizzle
            for (int kb = 0; kb < o.kb; ++kb, ca += 128, cb += 128, sa += 2048, sb += 2048) {
                if (used >= kStages &&
                    !__all_sync(0xffffffffu, mbar_wait_for(&bar.empty[at.s], at.phase ^ 1, kWaitNs))) {
                    ok = false;
                    break;
                }
                const uint32_t a = ring + at.s * C::kStageBytes, b = a + C::kABytes, s0 = b + C::kBBytes + 16 * id;
                if (128 * kb + 16 * c < pitch) {
                    if (have_a) {
                        const uint8_t *q = ca;
#pragma unroll
                        for (int i = 0; i < 8; ++i, q += pitch16)
                            copy16(a + to + 2048 * i, q);
                    }
                    const uint8_t *q = cb;
#pragma unroll
                    for (int i = 0; i < C::kTileN / kCtas / 16; ++i, q += pitch16)
                        if (16 * i < half)
                            copy16(b + to + 2048 * i, q);
                }
                if (2048 * kb + 16 * id < blocks) {
                    if (have_a)
                        copy16(s0, sa);
                    copy16(s0 + C::kSaBytes, sb);
                    if (o.n > 128)
                        copy16(s0 + C::kSaBytes + 2048, sb + blocks);
                }
                copy16_arrive(smem_u32(&bar.tail[at.s]));
                at.step();
                ++used;
            }
        }
        copy16_wait_all();
        // leave only when every stage has been read
        for (uint32_t i = min(used, (uint32_t)kStages); i > 0 && ok; --i) {
            const GroupedRing<kStages> back = at.before(i);
            ok = mbar_wait_for(&bar.empty[back.s], back.phase, kWaitNs);
        }
        ok = __all_sync(0xffffffffu, ok);
    } else if (!C::kRows && warp == kWarpCopy) {
        // ------------------------------------------------------------ copies
        GroupedRing<kStages> at;
        uint32_t used = 0, cut_it = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            const GroupedTile o = walk.tile();
            const int half = ((o.n + 63) / 64 * 64) / kCtas;              // of the N side: this CTA's
            const uint32_t bytes = C::kABytes + C::kSaBytes + C::kSbBytes + (half + 63) / 64 * 8192;
            const bool has_cut = C::kBmn && p.counts && o.rows % C::kBlockK;
            const int m = o.m0 + 128 * (int)rank, n = o.n0 + half * (int)rank;
            for (int kb = 0; kb < o.kb; ++kb) {
                if (used >= kStages &&
                    !__all_sync(0xffffffffu, mbar_wait_for(&bar.empty[at.s], at.phase ^ 1, kWaitNs))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    // a last block of rows that has to be cut is counted on a barrier
                    // of this CTA's own first
                    const uint32_t f = has_cut && kb == o.kb - 1 ? smem_u32(&bar.tail[cut_it % kStages])
                                                                 : full0 + 8 * at.s;
                    const uint32_t a = ring + at.s * C::kStageBytes, b = a + C::kABytes;
                    const int k0 = kb * C::kBlockK;
                    mbar_arrive_expect_tx_at(f, bytes);
                    // the N side: a box of 64 at a time
                    auto load_b = [&](int i, int x, int y) {
                        tma_load_3d<kCtas>(b + i * 128, p.map + kMapB, x, y, 0, f);
                    };
                    if constexpr (C::kFp4) {
                        const int x = k0 / 2, ys = k0 / 16;               // bytes; pieces of 128 bytes of scales
                        const uint32_t sa = b + C::kBBytes, sb = sa + C::kSaBytes;
                        tma_load_3d<kCtas>(a, p.map + kMapA, x, m, o.e, f);
                        for (int i = 0; i < half; i += 64)
                            load_b(i, x, o.row0 + n + i);
                        tma_load_3d<kCtas>(sa, p.map + kMapSa, 0, ys, o.e * ((p.M + 127) / 128) + m / 128, f);
                        tma_load_3d<kCtas>(sb, p.map + kMapSb, 0, ys, (o.row0 + o.n0) / 128, f);
                    } else if constexpr (C::kWgrad) {
                        for (int i = 0; i < 128; i += 64)
                            tma_load_3d<kCtas>(a + i * 128, p.map + kMapA, m + i, o.row0 + k0, 0, f);
                        for (int i = 0; i < half; i += 64)
                            load_b(i, n + i, o.row0 + k0);
                    } else {
                        if constexpr (C::kAmn) {
                            for (int i = 0; i < 128; i += 64)
                                tma_load_3d<kCtas>(a + i * 128, p.map + kMapA, m + i, k0, o.e, f);
                        } else {
                            tma_load_3d<kCtas>(a, p.map + kMapA, k0, m, o.e, f);
                        }
                        for (int i = 0; i < half; i += 64)
                            load_b(i, k0, o.row0 + n + i);
                    }
                }
                __syncwarp();
                at.step();
                ++used;
            }
            cut_it += has_cut;
        }
        // never leave with copies in flight: in each stage the last one's
        // consumption, or at least its arrival
        if (elect_one()) {
            for (uint32_t i = min(used, (uint32_t)kStages); i > 0; --i) {
                const GroupedRing<kStages> back = at.before(i);
                if (!mbar_wait_for(&bar.empty[back.s], back.phase, kWaitNs)) {
                    ok = false;
                    if (rank == 0)
                        (void)mbar_wait_for(&bar.full[back.s], back.phase, kWaitNs);
                }
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    } else if (warp == kWarpMma && rank == 0) {
        // ------------------------------------------------------------ products
        GroupedRing<kStages> at;
        uint32_t acc_it = 0, last_un = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            const GroupedTile o = walk.tile();
            if (o.kb == 0)
                continue;
            const uint32_t un = (uint32_t)(o.n + 63) / 64 * 64;
            uint32_t idesc = (1u << 7) | (1u << 10) | ((un >> 3) << 17) | ((uint32_t)(8 * kCtas) << 24);
            if (!C::kFp4)
                idesc |= (1u << 4) | ((uint32_t)C::kAmn << 15) | ((uint32_t)C::kBmn << 16);
            const int k_all = C::kWgrad ? o.rows : p.K;
            if (elect_one()) {
                uint32_t b = 0, d = 0;
                bool add = true;
                for (int kb = 0; kb < o.kb; ++kb) {
                    if (kb == 0 || (C::kParts && kb % C::kPartBlocks == 0)) {
                        b = acc_it & 1;
                        d = tmem + b * C::kAcc1;
                        add = false;
                        ok = acc_it < 2 || mbar_wait_for(&bar.acc_empty[b], ((acc_it >> 1) - 1) & 1, kWaitNs);
                        // the columns that the accumulators share, where both sums use them
                        if (C::kFp4 && acc_it > 0 && (b ? last_un : un) > C::kAcc1)
                            ok = ok && mbar_wait_for(&bar.acc_shared, (acc_it - 1) & 1, kWaitNs);
                        if (!ok)
                            break;
                        last_un = un;
                        ++acc_it;
                        tmem_fence_after();
                    }
                    // a stage that threads wrote, in a pair those of both CTAs
                    const bool threads = kCtas == 2 && (C::kRows || (C::kBmn && p.counts && kb == o.kb - 1));
                    ok = threads ? mbar_wait_for<true>(&bar.full[at.s], at.phase, kWaitNs)
                                 : mbar_wait_for(&bar.full[at.s], at.phase, kWaitNs);
                    if (!ok)
                        break;
                    tmem_fence_after();
                    const uint32_t a = ring + at.s * C::kStageBytes, bb = a + C::kABytes;
                    const uint64_t da = C::kAmn ? desc_mn_major(a) : desc_k_major(a);
                    const uint64_t db = C::kBmn ? desc_mn_major(bb) : desc_k_major(bb);
                    constexpr uint64_t ja = (C::kAmn ? 2048 : 32) >> 4, jb = (C::kBmn ? 2048 : 32) >> 4;   // a step
                    const int steps = (k_all - kb * C::kBlockK + C::kStepK - 1) / C::kStepK;
                    if constexpr (C::kFp4) {
                        const uint64_t dsa = desc_scales(bb + C::kBBytes), dsb = dsa + (C::kSaBytes >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j < steps) {
                                tmem_cp_scales<kCtas>(tmem + C::kSaCol + 4 * j, dsa + 32 * j);
                                tmem_cp_scales<kCtas>(tmem + C::kSbCol + 8 * j, dsb + 32 * j);
                                if (un > 128)
                                    tmem_cp_scales<kCtas>(tmem + C::kSbCol + 8 * j + 4, dsb + 128 + 32 * j);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < steps)
                                mma_nvfp4<kCtas>(d, da + ja * j, db + jb * j, idesc, tmem + C::kSaCol + 4 * j,
                                                 tmem + C::kSbCol + 8 * j, add || j > 0);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < steps)
                                mma_bf16<kCtas>(d, da + ja * j, db + jb * j, idesc, add || j > 0);
                    }
                    add = true;
                    mma_commit<kCtas>(smem_u32(&bar.empty[at.s]));
                    at.step();
                    if (kb == o.kb - 1 || (C::kParts && (kb + 1) % C::kPartBlocks == 0))
                        mma_commit<kCtas>(smem_u32(&bar.acc_full[b]));
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
    } else if (C::kWgrad && !C::kFp4 && (warp == kWarpCut || warp == kWarpMma) && p.counts) {
        // ------------------------------------------------------------ cut blocks
        // rows of a slot behind the expert's tokens count as zero, whatever they hold;
        // in a pair's second CTA, whose arrivals take longer, two warps take them in
        // turn (5000 rows, 61 experts of 1000 x 2056: 72 us, with one 76)
        const uint32_t cutters = rank == 0 ? 1 : 2, first = rank == 0 ? 0 : warp - kWarpMma;
        uint32_t it = 0, cut_it = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            const GroupedTile o = walk.tile();
            const int rem = o.rows % C::kBlockK;
            it += o.kb;
            if (!rem)
                continue;
            if (cut_it % cutters != first) {
                ++cut_it;
                continue;
            }
            const int s = (int)((it - 1) % kStages);
            ok = __all_sync(0xffffffffu,
                            mbar_wait_for(&bar.tail[cut_it % kStages], (cut_it / kStages) & 1, kWaitNs));
            if (!ok)
                break;
            ++cut_it;
            const int boxes = 2 + (((o.n + 63) / 64 * 64) / kCtas + 63) / 64;
            uint8_t *const a = base + s * C::kStageBytes;       // A's boxes, then B's
            for (int x = 0; x < boxes; ++x)
                for (int i = rem * 8 + lane; i < 512; i += 32)
                    reinterpret_cast<uint4 *>(a + 8192 * x)[i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                arrive_at_leader(s);
        }
    } else if (warp < kOutWarps) {
        // ------------------------------------------------------------ sums
        const int w = warp & 3, side = warp >> 2;               // its lanes; which of every two pieces
        uint8_t *const dst = out_s + warp * C::kOutBytes;
        const uint32_t d = smem_u32(dst);
        const uint32_t acc_empty0 = at_leader(&bar.acc_empty[0]), acc_shared = at_leader(&bar.acc_shared);
        uint32_t acc_it = 0;
        for (int t = unit; t < tiles; t += units) {
            const GroupedTile o = walk.tile();
            if (o.kb == 0 && p.add)
                continue;
            const int m = o.m0 + 128 * (int)rank + 32 * w;      // first of this warp's 32 rows of the M side
            const int nch = (o.n + C::kChunk - 1) / C::kChunk;
            const int parts = C::kParts ? (o.kb + C::kPartBlocks - 1) / C::kPartBlocks : 1;
            // with overlapping accumulators the shared columns come first: the end
            // of the one, the beginning of the other (not of a sum in
            // parts: a warp's columns stay the same)
            const bool back = C::kFp4 && (acc_it & 1) == 0 && parts == 1;
            float ms[4], scale0 = 1.f, scale1 = 1.f;
            if constexpr (C::kFp4 && !C::kWgrad) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int f = m + 8 * h + lane / 4;
                    ms[h] = f < p.M ? ld_word(p.m_scale + (int64_t)o.e * p.M + f) : 0.f;
                }
            } else if constexpr (C::kFp4) {
                scale0 = __fdiv_rn(1.f, ld_word(p.m_scale + o.e));
                scale1 = __fdiv_rn(1.f, ld_word(p.n_scale + o.e));
            }
            // the row scale of token `lane` of a piece
            auto row_scale = [&](int cc) {
                const int i = 32 * (back ? nch - 1 - cc : cc) + lane;
                return C::kFp4 && !C::kWgrad && cc < nch && i < o.n ? ld_word(p.n_scale + o.row0 + o.n0 + i) : 0.f;
            };
            float ts_next = row_scale(side), ts_lane = 0.f;
            auto emit = [&](int cc, uint32_t *r, bool add) {
                if (m >= p.M)
                    return;
                const int c = back ? nch - 1 - cc : cc;
                if (elect_one())
                    tma_store_wait_read0();
                __syncwarp();
                if constexpr (!C::kWgrad) {
                    // 32 tokens x 32 features, a token's 64 bytes in a row (64-byte swizzle)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 ts = make_float2(1.f, 1.f);
                        if constexpr (C::kFp4) {
                            ts.x = __shfl_sync(0xffffffffu, ts_lane, 8 * i + 2 * (lane & 3));
                            ts.y = __shfl_sync(0xffffffffu, ts_lane, 8 * i + 2 * (lane & 3) + 1);
                        }
                        uint32_t q[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            float v0 = u2f(r[16 * (h / 2) + 4 * i + 2 * (h & 1)]);
                            float v1 = u2f(r[16 * (h / 2) + 4 * i + 2 * (h & 1) + 1]);
                            if constexpr (C::kFp4) {
                                v0 = v0 * ms[h] * ts.x;
                                v1 = v1 * ms[h] * ts.y;
                            }
                            q[h] = cvt_bf16x2(v0, v1);
                        }
                        const int row = 8 * i + (lane & 7), chunk = lane >> 3;
                        st_matrix_trans(d + 64 * row + ((chunk ^ ((row >> 1) & 3)) << 4), q[0], q[1], q[2], q[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) {
                        tma_store_3d<false>(&p.out, m, o.row0 + o.n0 + 32 * c, 0, d);
                        tma_store_commit();
                    }
                } else {
                    // 32 rows of 128 bytes (128-byte swizzle)
                    if constexpr (C::kFp4) {
#pragma unroll
                        for (int i = 0; i < C::kChunk; ++i)
                            r[i] = f2u(u2f(r[i]) * scale0 * scale1);
                    }
                    if constexpr (!C::kF32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = cvt_bf16x2(u2f(r[2 * i]), u2f(r[2 * i + 1]));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(dst + 128 * lane + ((i ^ (lane & 7)) << 4)) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) {
                        if (C::kF32 && add)
                            tma_store_3d<true>(&p.out, o.n0 + C::kChunk * c, m, o.e, d);
                        else
                            tma_store_3d<false>(&p.out, o.n0 + C::kChunk * c, m, o.e, d);
                        tma_store_commit();
                    }
                }
            };
            uint32_t r[C::kChunk];
            if (C::kWgrad && o.kb == 0) {          // no rows: zeros
                for (int cc = side; cc < nch; cc += 2) {
#pragma unroll
                    for (int i = 0; i < C::kChunk; ++i)
                        r[i] = 0u;
                    emit(cc, r, false);
                }
                continue;
            }
            float keep[C::kKeep ? C::kTileN / 64 : 1][32];
            for (int part = 0; part < parts; ++part) {
                if (C::kParts && !C::kKeep && part > 0 && elect_one())
                    tma_store_wait0();             // what is added to has been written
                const uint32_t b = acc_it & 1;
                const uint32_t acc = tmem + ((uint32_t)(32 * w) << 16) + b * C::kAcc1;
                if (!__all_sync(0xffffffffu, mbar_wait_for(&bar.acc_full[b], (acc_it >> 1) & 1,
                                                           kWaitNs + 4096ull * (uint64_t)o.kb))) {
                    ok = false;
                    break;
                }
                ++acc_it;
                tmem_fence_after();
                const bool shared_first = C::kFp4 && (back || b == 1);
#pragma unroll
                for (int q = 0; q < C::kTileN / 2 / C::kChunk; ++q) {
                    const int cc = side + 2 * q;
                    if (q > 0 && cc >= nch)
                        break;
                    if (cc < nch) {
                        const uint32_t at0 = acc + C::kChunk * (back ? nch - 1 - cc : cc);
                        if constexpr (!C::kWgrad) {
                            tmem_ld_16x32(at0, r);
                            tmem_ld_16x32(at0 + (16u << 16), r + 16);
                        } else {
                            tmem_ld_32x32(at0, r);
                            if constexpr (C::kChunk == 64)
                                tmem_ld_32x32(at0 + 32, r + 32);
                        }
                        ts_lane = ts_next;
                        ts_next = row_scale(cc + 2);
                        tmem_wait_ld(r);
                        if constexpr (C::kChunk == 64)
                            tmem_wait_ld(r + 32);
                    }
                    // what the next products wait for
                    const bool last = cc + 2 >= nch, shared = C::kFp4 && (shared_first ? q == 0 : last);
                    if (shared || last) {
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (shared)
                                mbar_arrive_at(acc_shared);
                            if (last)
                                mbar_arrive_at(acc_empty0 + 8 * b);
                        }
                    }
                    if (cc >= nch)
                        break;
                    if constexpr (C::kKeep) {
                        if (part > 0) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = f2u(u2f(r[i]) + keep[q][i]);
                        }
                        if (part < parts - 1) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                keep[q][i] = u2f(r[i]);
                            continue;
                        }
                    }
                    emit(cc, r, p.add || (!C::kKeep && part > 0));
                }
            }
            if (!ok)
                break;
        }
        if (elect_one())
            tma_store_wait0();
    }

    if (!ok && lane == 0)
        raise_status(p.status, kDevErrTimeout);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if constexpr (kCtas == 2)
        cluster_sync();
    if (warp == kWarpCut)
        tmem_dealloc<kCtas>(tmem, 512);
}

// ---------------------------------------------------------------- launch
// CTAs or pairs of this kernel that are resident at once.
template <class C> cudaError_t grouped_units(const LaunchCtx &c, int &units)
{
    static std::atomic<int> known[64];
    static std::atomic<uint32_t> limit_set[2];
    const uint32_t smem = grouped_smem_bytes<C>();
    cudaError_t e = ensure_smem_limit(grouped_kernel<C>, c.device, (int)smem, limit_set);
    if (e != cudaSuccess)
        return e;
    if (C::kCtas == 1) {
        units = c.num_sms;
        return cudaSuccess;
    }
    if (c.device < 64 && (units = known[c.device].load(std::memory_order_relaxed)) > 0)
        return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C::kCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(c.num_sms / C::kCtas * C::kCtas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&units, grouped_kernel<C>, &cfg);
    if (e != cudaSuccess)
        return e;
    if (units < 1)
        units = 1;
    if (c.device < 64)
        known[c.device].store(units, std::memory_order_relaxed);
    return cudaSuccess;
}

// Whether single CTAs rather than pairs take a call whose M side has M rows and
// whose N sides make n_tiles of the single CTA's tiles.  Products (128 x 128 a
// tile): where all tiles run at once.  Measured on GB300, single against pair:
// 8.5 us against 9.2 (one token, 2 of 8 experts of 1024 x 1024), 8.8 against 10.6
// and in NVFP4 7.2 against 8.7 (300 tokens, 2 of 8 of 1024 x 1024); with two rounds
// 8.8 against 8.5 (1000 tokens, 4 experts of 2048 x 512).  Weight gradients (128 x
// 256): there, and where rounds of tiles decide: 13.1 against 18 (16 experts of
// 1152 x 1024, NVFP4: 4 rounds against 5); with many rounds a single CTA's tile
// takes 1.14 to 1.23 times the pair's time.
template <class C> bool single_ctas(const LaunchCtx &c, int64_t M, int64_t n_tiles)
{
    const int64_t one = (M + 127) / 128 * n_tiles, pair = (M + 255) / 256 * n_tiles;
    const int64_t rounds1 = (one + c.num_sms - 1) / c.num_sms, rounds2 = (pair + c.num_sms / 2 - 1) / (c.num_sms / 2);
    return one <= c.num_sms || (C::kWgrad && rounds1 * 12 < rounds2 * 10);
}

// `most_tiles`: a bound on the call's tiles that the host knows.
template <class C> cudaError_t launch_grouped(const LaunchCtx &c, const GroupedParams &p, int64_t most_tiles)
{
    int units = 0;
    cudaError_t e = grouped_units<C>(c, units);
    if (e != cudaSuccess)
        return e;
    if (most_tiles < units)
        units = (int)(most_tiles < 1 ? 1 : most_tiles);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::kCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(units * C::kCtas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = grouped_smem_bytes<C>();
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = C::kCtas == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, grouped_kernel<C>, p);
}

} // namespace epq
