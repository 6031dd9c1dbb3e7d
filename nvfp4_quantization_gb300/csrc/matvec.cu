// Products of a few tokens with NVFP4 expert weights (decode batches).
//
//   y[s] = W_e(s) x(s),  W[n][i] = code(n, i) * s_b(n, i / 16) * S(n)
//
// The weights are packed NVFP4 rows as the pack writes them (E2M1 codes, an
// E4M3 scale per 16 elements, an FP32 row scale in the trailer): one row per
// output feature.
//
// Bound: the rows of the experts in use are read once from HBM; everything
// else is small.  To keep up, the arithmetic goes to the warp-level matrix
// instruction (m16n8k16, f16 inputs, FP32 accumulators) with 16 weight rows as
// M and up to 8 slots of the same expert as N:
//  - code * s_b has at most six significant bits and lies in [2^-10, 2688], so
//    it is exact in f16, and one accumulator runs over the whole row; S(n) is
//    applied to the finished sum.
//  - x is BF16; a slot's elements are scaled by one power of two that brings
//    its largest to [2^14, 2^15) and taken to f16: exact for every element
//    within 2^-31 of the largest, and off by at most 2^-39 of the largest
//    below that (FP32 accumulation loses more).  Infinities and NaN stay.
//  - two codes are converted by one instruction; taking them apart by shifts
//    and masks costs four times the instructions and twice the time.
//  - the summation index is free to be permuted: lane (g, t) of a warp takes
//    64 consecutive elements of rows g and g + 8, so no fragment shuffle is
//    needed, and x is brought into the order in which the lanes want it.
//  - the rows come by TMA, 16 rows x 512 elements at a time, into a ring of
//    each warp's own: a warp waits for nobody but its own copies.
// What bounds it: HBM, with the conversion, the scaling and the matrix
// instructions close behind (57 % of the issue slots; without the copies the
// arithmetic alone takes 0.8 of the time), so a step's bookkeeping has to be
// small beside its 32 matrix instructions.
//  - two warps share a tile, each taking every second step of its rows, and one
//    of them adds the partial sums up.  The warps wait for each other where the
//    group of slots (and so x) changes, for a tile's time at worst; but every
//    tile costs two barriers (32 tokens x 8 of 64 experts of 4096 x 4096: 122 us
//    with one warp a tile, 115 with two, 120 with four, 140 with eight).  Where
//    there are not enough tiles for all teams, up to 16 share one (21 tokens x
//    121 outputs of 3936: 11 -> 7 us).
//  - x is staged with each thread on one slot, and in an order without bank
//    conflicts: with every thread on all slots it held the group changes back
//    (the batch above: 115 -> 110 us; 19 tokens x 6 of 13 experts of 404 x 128:
//    15 -> 9 us).
//  - measured and dropped: fragments loaded straight to registers (8 cache
//    lines a request held the L1 at 80 %: 202 us for the batch above); whole row
//    blocks by one bulk copy with x in registers and a row split over 16 warps
//    (their hand-over of partial sums: 159 us); the copies issued by a warp of
//    their own (17 warps leave 96 registers: 127 us).
// Measured on GB300, 4096 x 4096 per expert, 64 experts top-8: one token 17.4 us
// (76 MB, 4.4 TB/s, of which 4 us are the launch, the ids and x), 8 tokens 66 us
// (5.5 TB/s of the rows in use), 32 tokens 109 us (5.4 TB/s).  7168 x 4096: one
// token 26.7 us (5.0 TB/s), 32 tokens 198 us (5.2 TB/s).
// Every further 8 slots of an expert are another pass over its rows, which L2
// may hold by then but which are converted and scaled again: one expert of 4096
// x 16384 (floor 5.6 us) takes 13.7 us for 8 tokens, 18.9 for 16, 30.4 for 32 and
// 97 for 128; 32 tokens top-2 of 8 experts of 4096 x 4096 30.8 us (floor 11.2).
// The order of a row's sum depends on the call's shape (T, k, K, N, E) and the
// number of SMs, by which the launcher chooses how many warps share a tile,
// never on the routing: a slot's result does not depend on where the other
// slots went.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;        // weight rows of a warp's tile
constexpr int kHalf = 256;       // elements of a row that a warp multiplies at a time
constexpr int kMaxDepth = 3;     // steps in flight per warp, at most ...
constexpr int kMinDepth = 2;     // ... and at least
constexpr int kMaxE = 1024;
constexpr int kIds = 512;        // slots whose expert is kept in shared memory
constexpr int kMaxParts = 2;     // warps that share a tile, where tiles are many

// One word of eight E2M1 codes -> four f16 pairs (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Block scales 2i and 2i + 1 of a word of four, each in both halves (moves
// that the multiplication's operands absorb).
__device__ __forceinline__ void scale_pair(uint32_t two, uint32_t &s0, uint32_t &s1)
{
    const uint32_t v = cvt_f16x2_from_e4m3x2(two);
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b32 %0, {lo, lo};\n\tmov.b32 %1, {hi, hi};\n\t}"
        : "=r"(s0), "=r"(s1) : "r"(v));
}

// 256 elements of 16 rows: this lane's 64 elements of rows g and g + 8 against
// its column of x.  `x(j)`: elements 8j .. 8j + 7 of the 64 as f16; `lo`, `hi`:
// the rows' codes in the lane's order; `slo`, `shi`: their four block scales.
// Two accumulators, whose sum is the result: one instruction need not wait for
// the one before.
template <typename X>
__device__ __forceinline__ void multiply(float (&acc)[2][4], const uint4 (&lo)[2], const uint4 (&hi)[2], uint32_t slo,
                                         uint32_t shi, X x)
{
    uint32_t s_lo[4], s_hi[4];
    scale_pair(slo & 0xffffu, s_lo[0], s_lo[1]);
    scale_pair(slo >> 16, s_lo[2], s_lo[3]);
    scale_pair(shi & 0xffffu, s_hi[0], s_hi[1]);
    scale_pair(shi >> 16, s_hi[2], s_hi[3]);
    const uint32_t w_lo[8] = {lo[0].x, lo[0].y, lo[0].z, lo[0].w, lo[1].x, lo[1].y, lo[1].z, lo[1].w};
    const uint32_t w_hi[8] = {hi[0].x, hi[0].y, hi[0].z, hi[0].w, hi[1].x, hi[1].y, hi[1].z, hi[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 b = x(j);
        uint32_t l[4], h[4];
        codes_to_f16(w_lo[j], l);
        codes_to_f16(w_hi[j], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[i] = hmul2_rn(l[i], s_lo[j >> 1]);
            h[i] = hmul2_rn(h[i], s_hi[j >> 1]);
        }
        mma16816(acc[0], l[0], h[0], l[1], h[1], b.x, b.y);
        mma16816(acc[1], l[2], h[2], l[3], h[3], b.z, b.w);
    }
}

// The same for a single column of x, whose seven neighbours the instruction
// computes anyway: lane t's elements of x stand in column t for its even blocks
// and in column 4 + t for its odd ones, with zeros elsewhere, so eight
// instructions leave the sums of eight blocks a row apart, and the block scales
// are applied to those sums instead of to the weights (12 operations a row
// pair in place of 32).  `x(j, odd)`: as above where the lane's column is t (or
// 4 + t), else zeros; `slo`, `shi`: the block scales of lanes L and L + 1, L =
// 2 (t mod 2), of rows g and g + 8; `pick`: selects byte t / 2 of both words.
template <typename X>
__device__ __forceinline__ void multiply_one(float2 &acc, const uint4 (&lo)[2], const uint4 (&hi)[2], uint2 slo,
                                             uint2 shi, uint32_t pick, X x)
{
    const uint32_t w_lo[8] = {lo[0].x, lo[0].y, lo[0].z, lo[0].w, lo[1].x, lo[1].y, lo[1].z, lo[1].w};
    const uint32_t w_hi[8] = {hi[0].x, hi[0].y, hi[0].z, hi[0].w, hi[1].x, hi[1].y, hi[1].z, hi[1].w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {       // blocks 2i and 2i + 1 of every lane
        float sums[4] = {};
#pragma unroll
        for (int j = 4 * i; j < 4 * i + 4; ++j) {
            const uint4 b = x(j, (j >> 1) & 1);
            uint32_t l[4], h[4];
            codes_to_f16(w_lo[j], l);
            codes_to_f16(w_hi[j], h);
            mma16816(sums, l[0], h[0], l[1], h[1], b.x, b.y);
            mma16816(sums, l[2], h[2], l[3], h[3], b.z, b.w);
        }
        const uint32_t sel = pick + 0x22u * i;
        const float2 s_lo = f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(__byte_perm(slo.x, slo.y, sel)));
        const float2 s_hi = f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(__byte_perm(shi.x, shi.y, sel)));
        acc.x = fmaf(sums[0], s_lo.x, acc.x);
        acc.y = fmaf(sums[2], s_hi.x, acc.y);
        acc.x = fmaf(sums[1], s_lo.y, acc.x);
        acc.y = fmaf(sums[3], s_hi.y, acc.y);
    }
}

// A warp's place of the ring: kTile rows of HALVES halves of codes, whose pitch
// of 16 bytes more than they need (the next step's first ones) keeps the lanes
// of a warp off each other's banks; then their scales.
template <int HALVES> struct Place {
    static constexpr int code_pitch = HALVES * kHalf / 2 + 16;
    static constexpr int scale_pitch = HALVES * kHalf / 16;
    static constexpr int codes = kTile * code_pitch;
    static constexpr int bytes = codes + kTile * scale_pitch;
};

__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// The copy and barrier helpers on shared-memory addresses: a warp's place and
// barrier move from step to step, and as generic pointers they would be converted
// at every use.
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap *m, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"((uint64_t)m), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx_at(uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __noinline__ bool mbar_wait_bounded_at(uint32_t bar, uint32_t parity)
{
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait_at(bar, parity))
            return true;
        if (i > 64)
            __nanosleep(256);
    }
    return false;
}

// Bounded wait of a whole warp on its barrier (the first attempt in line).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_try_wait_at(bar, parity)))
        return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded_at(bar, parity));
}

struct Shared {
    int16_t ids[kIds];      // expert of a slot (-1: none), batches up to kIds slots
    int warp_sum[kWarps];
    int slot[8];            // the group's slots
    uint32_t top[8];        // largest finite |x| of each, as BF16 bits
    uint64_t full[kWarps * kMaxDepth];   // a place of a ring has its rows
    float4 partial[kWarps][32];          // partial sums of a tile, lane by lane
};

// Dynamic shared memory: the warps' rings, x of a group, kZeros bytes of zeros
// (where it is one slot), and int[E + 1] `first`, the groups of slots before
// each expert.
constexpr int kZeros = 2 * kHalf * 2;
constexpr int kMaxSmem = 227 * 1024 - (int)sizeof(Shared);

// Expert of a slot as the caller gave it, with ids outside [-1, E) as -2.
__device__ __forceinline__ int read_id(const MatvecArgs &a, int s)
{
    const int e = a.topk ? __ldg(a.topk + s) : 0;
    return e >= a.E || e < -1 ? -2 : e;
}

__device__ __forceinline__ int slot_expert(const MatvecArgs &a, const Shared &sh, int s)
{
    return a.T * a.k <= kIds ? sh.ids[s] : read_id(a, s);
}

// Exclusive prefix of one value per thread over the CTA; *total gets the sum.
__device__ __forceinline__ int cta_prefix(int v, int *warp_sum, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        before += i < warp ? warp_sum[i] : 0;
        all += warp_sum[i];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// Number of groups of each expert, as a prefix over the experts (`first` holds
// the slots of each while they are counted).
__device__ int count_groups(const MatvecArgs &a, Shared &sh, int *first, int per_group)
{
    const int slots = a.T * a.k;
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        first[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const int e = read_id(a, s);
        if (slots <= kIds)
            sh.ids[s] = (int16_t)e;
        if (e >= 0)
            atomicAdd(&first[e], 1);
        else if (e == -2 && blockIdx.x == 0)
            raise_status(a.status, kDevErrBadExpert);
    }
    __syncthreads();
    constexpr int kPer = kMaxE / kThreads;
    int g[kPer], mine = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        g[i] = e < a.E ? (first[e] + per_group - 1) / per_group : 0;
        mine += g[i];
    }
    int at = cta_prefix(mine, sh.warp_sum, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e < a.E)
            first[e] = at;
        at += g[i];
    }
    if (threadIdx.x == 0)
        first[a.E] = total;
    __syncthreads();
    return total;
}

// Batches of up to 32 slots: every warp works the groups out for itself, one
// slot a lane, without a barrier (a kernel's first copies start a microsecond
// sooner).
struct SmallBatch {
    int id;            // the lane's expert; negative: none
    int rank;          // of the slot among its expert's
    uint32_t leaders;  // lanes that begin a group

    __device__ __forceinline__ void read(const MatvecArgs &a, int per_group)
    {
        const int lane = threadIdx.x & 31, slots = a.T * a.k;
        id = lane < slots ? read_id(a, lane) : -1;
        if (id == -2 && blockIdx.x == 0 && threadIdx.x < 32)
            raise_status(a.status, kDevErrBadExpert);
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        rank = __popc(same & ((1u << lane) - 1));
        leaders = __ballot_sync(0xffffffffu, id >= 0 && rank % per_group == 0);
    }
    __device__ __forceinline__ int groups() const { return __popc(leaders); }
    __device__ __forceinline__ int leader(int group) const
    {
        const int lane = threadIdx.x & 31;
        const bool it = (leaders >> lane & 1u) && __popc(leaders & ((1u << lane) - 1)) == group;
        return __ffs(__ballot_sync(0xffffffffu, it)) - 1;
    }
    __device__ __forceinline__ int expert(int group) const { return __shfl_sync(0xffffffffu, id, leader(group)); }
    // the group's slots to shared memory (the caller's barrier publishes them)
    __device__ __forceinline__ int find(Shared &sh, int group, int per_group) const
    {
        const int lane = threadIdx.x & 31, l = leader(group);
        const int e = __shfl_sync(0xffffffffu, id, l), c = rank - __shfl_sync(0xffffffffu, rank, l);
        const bool hit = id == e && c >= 0 && c < per_group;
        if (threadIdx.x < 32) {
            if (hit)
                sh.slot[c] = lane;
            if (lane < 8)
                sh.top[lane] = 0;
        }
        return __popc(__ballot_sync(0xffffffffu, hit));
    }
};

__device__ __forceinline__ int64_t quotient(int64_t a, int b)
{
    return a < (int64_t)UINT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Zero rows for the slots without an expert.
__device__ void zero_rows(const MatvecArgs &a, const Shared &sh)
{
    const int slots = a.T * a.k;
    for (int s = blockIdx.x; s < slots; s += gridDim.x)
        if ((slots <= 32 ? read_id(a, s) : slot_expert(a, sh, s)) < 0)
            for (int n = threadIdx.x; n < a.N; n += kThreads)
                a.y[(int64_t)s * a.N + n] = 0;
}

// The slots of expert e with rank [from, from + per_group), in slot order;
// returns how many there are.
__device__ int find_slots(const MatvecArgs &a, Shared &sh, int e, int from, int per_group)
{
    const int slots = a.T * a.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = (slots + kThreads - 1) / kThreads * 32;   // slots of a warp, whole 32s
    const int s0 = warp * share, s1 = min(s0 + share, slots);
    int mine = 0;
    for (int s = s0 + lane; s < s1; s += 32)
        mine += slot_expert(a, sh, s) == e;
    int total;
    int rank = cta_prefix(mine, sh.warp_sum, &total);
    rank = __shfl_sync(0xffffffffu, rank, 0);                   // of the warp's first match
    for (int s = s0; s < s1; s += 32) {
        const bool hit = s + lane < s1 && slot_expert(a, sh, s + lane) == e;
        const uint32_t all = __ballot_sync(0xffffffffu, hit);
        const int r = rank + __popc(all & ((1u << lane) - 1)) - from;
        if (hit && r >= 0 && r < per_group)
            sh.slot[r] = s + lane;
        rank += __popc(all);
    }
    if (threadIdx.x < 8)
        sh.top[threadIdx.x] = 0;
    __syncthreads();
    return min(per_group, total - from);
}

// The power of two that a slot's x is multiplied by: its largest element comes
// to [2^14, 2^15).  A subnormal largest counts as 2^-126.
__device__ __forceinline__ int x_shift(uint32_t top) { return top ? 14 - (max((int)(top >> 7), 1) - 127) : 0; }

// Largest finite |x| of 8 BF16 values and `top`, as bits.  (Halves compared in
// pairs; an infinity, or two NaN meeting, sends it the long way.)
__device__ __forceinline__ uint32_t finite_absmax(uint32_t top, uint4 v)
{
    uint32_t m;
    asm("{\n\t.reg .b32 p, q;\n\t"
        "max.xorsign.abs.bf16x2 p, %1, %2;\n\t"
        "max.xorsign.abs.bf16x2 q, %3, %4;\n\t"
        "max.xorsign.abs.bf16x2 %0, p, q;\n\t}" : "=r"(m) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
    m = max(m & 0x7fffu, (m >> 16) & 0x7fffu);
    if (m >= 0x7f80u) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t l = w[i] & 0x7fffu, h = (w[i] >> 16) & 0x7fffu;
            m = max(m, max(l < 0x7f80u ? l : 0u, h < 0x7f80u ? h : 0u));
        }
    }
    return max(top, m);
}

// 8 BF16 values times 2^shift, as f16.  The power comes in two factors: it
// reaches 2^140.
__device__ __forceinline__ uint4 to_f16(uint4 v, int shift)
{
    const float2 f0 = make_float2(exp2i(shift / 2), exp2i(shift / 2));
    const float2 f1 = make_float2(exp2i(shift - shift / 2), exp2i(shift - shift / 2));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = mul2(mul2(make_float2(u2f(w[i] << 16), u2f(w[i] & 0xffff0000u)), f0), f1);
        h[i] = cvt_f16x2(p.x, p.y);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

__device__ __forceinline__ const uint16_t *x_row(const MatvecArgs &a, int s)
{
    return a.x + (int64_t)(a.per_slot ? s : s / a.k) * a.ld_x;
}

// v * scale * 2^-shift, rounded once to FP32 in its normal range: the two
// scales together may pass that range where the result does not, so the
// exponents are added as integers and applied in two factors.  (64-bit
// arithmetic would say it shorter and is slow here.)
__device__ __forceinline__ float rescale(float v, float scale, int shift)
{
    const uint32_t b = f2u(scale);
    int e = (int)((b >> 23) & 0xffu);
    float m = scale;
    if (e == 0 || e == 255)
        e = 0;                          // zero, subnormal, infinity, NaN: as it is
    else {
        m = u2f((b & 0x807fffffu) | 0x3f800000u);
        e -= 127;
    }
    e = max(-250, min(250, e - shift));     // beyond these the result is 0 or infinite anyway
    return v * m * exp2i(e / 2) * exp2i(e - e / 2);
}

// The finished sums of a lane (rows `row` and row + 8, slots 2t and 2t + 1).
__device__ __forceinline__ void write_sums(const MatvecArgs &a, const Shared &sh, const float (&acc)[4], int m, int row,
                                           int t, float scale_lo, float scale_hi)
{
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int c = 2 * t + (v & 1), n = row + (v & 2 ? 8 : 0);
        if (c < m && n < a.N)
            a.y[(int64_t)sh.slot[c] * a.N + n] =
                (uint16_t)cvt_bf16x2(rescale(acc[v], v & 2 ? scale_hi : scale_lo, x_shift(sh.top[c])), 0.0f);
    }
}

// Expert of a group of slots: the last one with first[e] <= group.
__device__ __forceinline__ int expert_of_group(const int *first, int E, int group)
{
    int e = 0, hi = E - 1;
    while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (first[mid] <= group)
            e = mid;
        else
            hi = mid - 1;
    }
    return e;
}

// x of the group's m slots -> f16 in shared memory: elements 8q .. 8q + 7 of
// slot c at 16-byte place (((q / 32) * 8 + q % 8) * G + c) * 4 + (q / 8) % 4,
// which is where lane (c, t) looks for word q % 8 of its 64 elements of half
// step q / 32 (eight neighbouring lanes: 128 neighbouring bytes).  kThreads / G
// threads have a slot; a warp's lanes take the 32 places of a half step in an
// order in which four neighbours write 64 neighbouring bytes.
template <int G>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, Shared &sh, int m, uint4 *xs, int halves)
{
    constexpr int kSpan = kThreads / G, kKeep = G;
    const int nq = a.K / 8, c = threadIdx.x / kSpan, l = threadIdx.x & 31;
    const int q0 = (threadIdx.x % kSpan & ~31) + (l & 3) * 8 + (l >> 2);
    const uint4 *x = reinterpret_cast<const uint4 *>(x_row(a, sh.slot[c < m ? c : 0]));
    const bool here = c < m, once = nq <= kKeep * kSpan;    // once: what was read is kept
    uint4 kept[kKeep];
    uint32_t top = 0;
    if (here) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            kept[i] = make_uint4(0, 0, 0, 0);
            if (i * kSpan < nq && q0 + i * kSpan < nq)
                kept[i] = __ldg(x + q0 + i * kSpan);
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (i * kSpan >= nq)
                break;
            top = finite_absmax(top, kept[i]);
        }
        for (int q = q0 + kKeep * kSpan; q < nq; q += kSpan)
            top = finite_absmax(top, __ldg(x + q));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (l == 0 && top)
        atomicMax(&sh.top[c], top);
    __syncthreads();
    if (here) {
        const int shift = x_shift(sh.top[c]);
        auto put = [&](int q, uint4 v) {
            xs[(((q >> 5) * 8 + (q & 7)) * G + c) * 4 + ((q >> 3) & 3)] = to_f16(v, shift);
        };
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (i * kSpan >= halves * 32)
                break;
            if (q0 + i * kSpan < halves * 32)
                put(q0 + i * kSpan, kept[i]);               // (zeros past K)
        }
        if (!once)
            for (int q = q0 + kKeep * kSpan; q < halves * 32; q += kSpan)
                put(q, q < nq ? __ldg(x + q) : make_uint4(0, 0, 0, 0));
    }
}

// Persistent: the (group of slots, tile of rows) pairs are dealt to the CTAs
// in contiguous ranges, so a CTA meets few groups; a CTA's teams of `parts`
// warps take the pairs of its range in turn.  The steps of a warp's pairs run
// through its ring without a gap, also where the group changes.  G: columns of
// x in shared memory (slots per group); HALVES: of a step.
template <int G, int HALVES>
__global__ void __launch_bounds__(kThreads, 1)
matvec_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap scales_map,
              MatvecArgs a, int depth, int parts)
{
    using P = Place<HALVES>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int halves = (a.K + kHalf - 1) / kHalf;
    const int steps = (halves + HALVES - 1) / HALVES;
    const int part = warp & (parts - 1), team = warp / parts, teams = kWarps / parts;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * depth * P::bytes);
    uint4 *xs = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * depth * P::bytes);
    uint4 *zeros = xs + (size_t)halves * 32 * G;
    int *first = reinterpret_cast<int *>(G == 1 ? zeros + kZeros / 16 : zeros);
    if (G == 1 && threadIdx.x < kZeros / 16)
        zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);    // (published by the barriers before the first product)
    uint64_t *full = sh.full + warp * kMaxDepth;
    if (lane == 0) {
        for (int i = 0; i < depth; ++i)
            mbar_init(full + i, 1);
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const bool small = a.T * a.k <= 32;
    SmallBatch batch;
    int groups;
    if (small) {
        batch.read(a, G);
        groups = batch.groups();
        __syncwarp();                   // the warp's mbarriers are its own
    } else {
        groups = count_groups(a, sh, first, G);
    }
    auto expert = [&](int group) { return small ? batch.expert(group) : expert_of_group(first, a.E, group); };
    const int tiles = (a.N + kTile - 1) / kTile;
    const int64_t total = (int64_t)groups * tiles;
    int64_t at = quotient(total * blockIdx.x, gridDim.x);
    const int64_t end = quotient(total * (blockIdx.x + 1), gridDim.x);

    // the step to load next: step p_step of the tile at row p_row, into place p_at
    const uint32_t ring_bytes = (uint32_t)(depth * P::bytes), bars = smem_u32(full);
    int64_t p_item = at + team;
    int p_tile = 0, p_row = 0, p_step = part, in_flight = 0;
    uint32_t p_at = 0, p_bar = bars;
    bool p_more = p_item < end;
    auto locate = [&]() {
        const int group = (int)quotient(p_item, tiles);
        p_tile = (int)(p_item - (int64_t)group * tiles);
        p_row = expert(group) * a.N + p_tile * kTile;
    };
    auto load = [&]() {
        if (!p_more)
            return;
        if (lane == 0) {
            const uint32_t to = ring + p_at;
            mbar_arrive_expect_tx_at(p_bar, P::bytes);
            tma_load_2d_at(to, &codes_map, p_step * (HALVES * kHalf / 4), p_row, p_bar);
            tma_load_2d_at(to + P::codes, &scales_map, p_step * (HALVES * kHalf / 16), p_row, p_bar);
        }
        ++in_flight;
        p_at += P::bytes;
        p_bar += sizeof(uint64_t);
        if (p_at == ring_bytes) {
            p_at = 0;
            p_bar = bars;
        }
        p_step += parts;
        if (p_step >= steps) {
            p_step = part;
            p_item += teams;
            p_tile += teams;
            p_row += teams * kTile;
            p_more = p_item < end;
            if (p_tile >= tiles && p_more)
                locate();
        }
    };
    if (p_more)
        locate();
    for (int i = 0; i < depth; ++i)
        load();

    int64_t item = at + team;
    int turn = 0;                       // whose it is to add a tile's parts up
    uint32_t c_at = 0, c_bar = bars, parity = 0;
    bool lost = false;                  // a wait gave up: no more loads, no more waits
    const uint32_t c_lane = ring + (uint32_t)(g * P::code_pitch + t * 32);
    const uint32_t s_lane = ring + (uint32_t)(P::codes + g * P::scale_pitch + t * 4);
    const uint32_t x_lane = smem_u32(xs) + (uint32_t)(((g % G) * 4 + t) * 16);
    // one slot: which blocks' x this lane's column holds, and the scales of its sums
    const bool even = g == t, odd = g == t + 4;
    const uint32_t s_one = ring + (uint32_t)(P::codes + g * P::scale_pitch + (t & 1) * 8);
    const uint32_t pick = (uint32_t)(t >> 1) * 0x11u + 0x40u;
    while (at < end) {
        const int group = (int)quotient(at, tiles);
        const int64_t stop = min(end, (int64_t)(group + 1) * tiles);
        const int e = expert(group);
        const uint8_t *w = a.w + (int64_t)e * a.N * a.S + a.S - 16;     // the row scales
        int m;
        if (small) {
            m = batch.find(sh, group, G);
            __syncthreads();
        } else {
            m = find_slots(a, sh, e, (group - first[e]) * G, G);
        }
        stage_x<G>(a, sh, m, xs, halves);
        __syncthreads();

        for (; item < stop; item += teams) {
            const int row = (int)(item - (int64_t)group * tiles) * kTile + g;
            const bool adds = part == turn;
            turn = (turn + 1) & (parts - 1);
            float row_lo = 0.0f, row_hi = 0.0f;
            if (adds) {
                row_lo = __ldg(reinterpret_cast<const float *>(w + (int64_t)min(row, a.N - 1) * a.S));
                row_hi = __ldg(reinterpret_cast<const float *>(w + (int64_t)min(row + 8, a.N - 1) * a.S));
            }
            uint32_t x = x_lane + (uint32_t)(part * HALVES * 32 * G * 16);
            float acc[2][4] = {};
            float2 one = make_float2(0.0f, 0.0f);
            for (int left = halves - part * HALVES; left > 0 && !lost; left -= parts * HALVES) {
                if (!warp_wait(c_bar, parity)) {
                    lost = true;
                    break;
                }
                --in_flight;
                const uint32_t place = c_at, c = c_lane + place;
                const uint32_t x_even = even ? x : smem_u32(zeros), x_odd = odd ? x : smem_u32(zeros);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    if (h < left) {
                        const uint32_t ch = c + h * (kHalf / 2);
                        const uint4 wl[2] = {lds128(ch), lds128(ch + 16)};
                        const uint4 wh[2] = {lds128(ch + 8 * P::code_pitch), lds128(ch + 8 * P::code_pitch + 16)};
                        if (G == 1) {
                            const uint32_t s = s_one + place + h * (kHalf / 16);
                            multiply_one(one, wl, wh, lds64(s), lds64(s + 8 * P::scale_pitch), pick, [&](int j, int o) {
                                return lds128((o ? x_odd : x_even) + (h * 32 + j * 4) * 16);
                            });
                        } else {
                            const uint32_t s = s_lane + place + h * (kHalf / 16);
                            multiply(acc, wl, wh, lds32(s), lds32(s + 8 * P::scale_pitch),
                                     [&](int j) { return lds128(x + (h * 32 * G + j * 4 * G) * 16); });
                        }
                    }
                }
                x += (uint32_t)(parts * HALVES * 32 * G * 16);
                c_at += P::bytes;
                c_bar += sizeof(uint64_t);
                if (c_at == ring_bytes) {
                    c_at = 0;
                    c_bar = bars;
                    parity ^= 1u;
                }
                __syncwarp();           // every lane has read the place that is loaded next
                load();
            }
            float sum[4] = {acc[0][0] + acc[1][0], acc[0][1] + acc[1][1], acc[0][2] + acc[1][2], acc[0][3] + acc[1][3]};
            if (G == 1) {               // the lanes of a row hold a quarter of its blocks each
                for (int o = 1; o < 4; o <<= 1) {
                    one.x += __shfl_xor_sync(0xffffffffu, one.x, o);
                    one.y += __shfl_xor_sync(0xffffffffu, one.y, o);
                }
                sum[0] = one.x;         // (slot 0 is lane t = 0's)
                sum[2] = one.y;
            }
            if (parts > 1) {
                named_bar_sync(1 + team, 32 * parts);       // the tile before has been added up
                sh.partial[warp][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
                named_bar_sync(1 + team, 32 * parts);
                if (adds) {
                    sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
                    for (int p = 0; p < parts; ++p) {
                        const float4 v = sh.partial[team * parts + p][lane];
                        sum[0] += v.x;
                        sum[1] += v.y;
                        sum[2] += v.z;
                        sum[3] += v.w;
                    }
                }
            }
            if (adds && !lost)
                write_sums(a, sh, sum, m, row, t, row_lo, row_hi);
        }
        at = stop;
        __syncthreads();                // before the next group's x and slots
    }
    if (lost && lane == 0) {
        raise_status(a.status, kDevErrTimeout);
        // never leave with a load in flight
        for (; in_flight > 0; --in_flight) {
            (void)mbar_wait_bounded_at(c_bar, parity);
            c_bar += sizeof(uint64_t);
            if (c_bar == bars + depth * sizeof(uint64_t)) {
                c_bar = bars;
                parity ^= 1u;
            }
        }
    }
    zero_rows(a, sh);
}

// Depth of the rings that x of G slots leaves room for.
template <int HALVES> int ring_depth(size_t x_bytes, int E)
{
    const size_t ring = (size_t)kWarps * Place<HALVES>::bytes;
    const size_t rest = x_bytes + sizeof(int) * (size_t)(E + 1);
    const int d = rest < (size_t)kMaxSmem ? (int)((kMaxSmem - rest) / ring) : 0;
    return d > kMaxDepth ? kMaxDepth : d;
}

template <int G, int HALVES> cudaError_t launch_ring(const LaunchCtx &c, const MatvecArgs &a, size_t x_bytes)
{
    using P = Place<HALVES>;
    static std::atomic<uint32_t> done[2] = {};
    cudaError_t e = ensure_smem_limit(matvec_kernel<G, HALVES>, c.device, kMaxSmem, done);
    if (e != cudaSuccess)
        return e;
    const uint64_t rows = (uint64_t)a.E * a.N;
    const int depth = ring_depth<HALVES>(x_bytes, a.E);
    CUtensorMap codes, scales;
    // codes in 16-bit units: a box has at most 256 of them along a side
    if (!make_map(&codes, a.w, (uint64_t)a.K / 4, rows, (uint64_t)a.S, P::code_pitch / 2, kTile, 2) ||
        !make_map(&scales, a.w + a.K / 2, (uint64_t)a.K / 16, rows, (uint64_t)a.S, P::scale_pitch, kTile))
        return cudaErrorInvalidValue;
    const int steps = (a.K + HALVES * kHalf - 1) / (HALVES * kHalf);
    // two warps a tile if each has two steps of it (one step a warp, rows of
    // 1024: 43 us where a warp a tile takes 38); more where there is less than a
    // tile for every team at most
    const int64_t slots = (int64_t)a.T * a.k;
    const int64_t groups = slots < a.E + slots / G ? slots : a.E + slots / G;
    const int64_t tiles = groups * ((a.N + kTile - 1) / kTile);
    int parts = 1;
    while (2 * parts <= steps && ((2 * parts <= kMaxParts && 4 * parts <= steps) ||
                                  (2 * parts <= kWarps && tiles * 2 * parts <= (int64_t)c.num_sms * kWarps)))
        parts *= 2;
    return launch_pdl(matvec_kernel<G, HALVES>, dim3((unsigned)c.num_sms), dim3(kThreads),
                      (size_t)kWarps * depth * P::bytes + x_bytes + sizeof(int) * (size_t)(a.E + 1), c.stream, codes,
                      scales, a, depth, parts);
}

template <int G> cudaError_t launch_group(const LaunchCtx &c, const MatvecArgs &a, size_t x_bytes)
{
    // whole steps where two of them fit beside x; half steps, which copy 18 bytes
    // for 16, take longer (the 32-token batch above: 130 us against 120)
    return ring_depth<2>(G * x_bytes, a.E) >= kMinDepth ? launch_ring<G, 2>(c, a, G * x_bytes)
                                                        : launch_ring<G, 1>(c, a, G * x_bytes);
}

} // namespace

cudaError_t launch_matvec(const LaunchCtx &c, const MatvecArgs &a)
{
    if (a.T == 0)
        return cudaSuccess;
    // Slots of one expert that share a pass over its rows: as many as there are
    // tokens (a router names an expert once per token; if it is named more
    // often, it gets more passes), at most 8, and as leave the rings two of the
    // smaller steps.
    const size_t x_bytes = (size_t)((a.K + kHalf - 1) / kHalf) * kHalf * 2;
    if (a.T == 1)
        return launch_group<1>(c, a, x_bytes + kZeros);
    if (a.T == 2 || ring_depth<1>(4 * x_bytes, a.E) < kMinDepth)
        return launch_group<2>(c, a, x_bytes);
    if (a.T <= 4 || ring_depth<1>(8 * x_bytes, a.E) < kMinDepth)
        return launch_group<4>(c, a, x_bytes);
    return launch_group<8>(c, a, x_bytes);
}

} // namespace epq
