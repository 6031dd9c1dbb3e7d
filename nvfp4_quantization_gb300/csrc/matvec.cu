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
//    within 2^-28 of the largest, and off by at most 2^-40 of the largest
//    below that (FP32 accumulation loses more).  Infinities and NaN stay.
//    (Hardware converts two codes in one instruction; taking them apart by
//    shifts and masks instead costs 4.3 instructions a pair and twice the time.)
//  - the summation index is free to be permuted: lane (g, t) of a warp takes
//    64 consecutive elements of rows g and g + 8, so no fragment shuffle is
//    needed; x lies in shared memory in the order in which the lanes want it.
//  - the rows come by TMA, 16 rows x 512 elements (256 bytes of codes, 32 of
//    scales a row) at a time, into a ring of each warp's own.  Loaded straight
//    to registers the same fragments cost the L1 eight lines a request and
//    held the kernel at 40 % of HBM.
// A row's sum is computed by one warp in one order, whatever else is in the
// batch: a slot's result does not depend on the other slots.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;        // weight rows of a warp's tile
constexpr int kHalf = 256;       // elements of a row that a warp multiplies at a time
constexpr int kStep = 512;       // ... and loads at a time
constexpr int kHalfBytes = kTile * kHalf / 2;     // codes of a half step
constexpr int kCodeBytes = kTile * kStep / 2;     // of a step
constexpr int kScaleBytes = kTile * kStep / 16;
constexpr int kMinDepth = 2;     // steps in flight per warp
constexpr int kMaxDepth = 3;
constexpr int kMaxE = 1024;
constexpr int kIds = 2048;       // slots whose expert is kept in shared memory
constexpr int kMaxSmem = 212 * 1024;   // dynamic: the warps' rings and x

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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Block scales 2i and 2i + 1 of a word of four, each in both halves.
__device__ __forceinline__ void scale_pair(uint32_t two, uint32_t &s0, uint32_t &s1)
{
    const uint32_t v = cvt_f16x2_from_e4m3x2(two);
    s0 = __byte_perm(v, v, 0x1010);
    s1 = __byte_perm(v, v, 0x3232);
}

// Half a step of 16 rows: this lane's 64 elements of rows g and g + 8 against
// its column of x, whose words lie 4 * G places apart.  `c0`, `c1`: the places of
// the lane's two 16-byte chunks of row g (row g + 8 is 1024 bytes on).
template <int G>
__device__ __forceinline__ void multiply(float (&acc)[4], const uint8_t *c0, const uint8_t *c1, const uint8_t *scales,
                                         const uint4 *xs)
{
    const uint32_t two_lo = *reinterpret_cast<const uint32_t *>(scales);
    const uint32_t two_hi = *reinterpret_cast<const uint32_t *>(scales + 8 * (kStep / 16));
    const uint4 lo0 = *reinterpret_cast<const uint4 *>(c0), lo1 = *reinterpret_cast<const uint4 *>(c1);
    const uint4 hi0 = *reinterpret_cast<const uint4 *>(c0 + 1024), hi1 = *reinterpret_cast<const uint4 *>(c1 + 1024);
    uint32_t slo[4], shi[4];
    scale_pair(two_lo & 0xffffu, slo[0], slo[1]);
    scale_pair(two_lo >> 16, slo[2], slo[3]);
    scale_pair(two_hi & 0xffffu, shi[0], shi[1]);
    scale_pair(two_hi >> 16, shi[2], shi[3]);
    const uint32_t lo[8] = {lo0.x, lo0.y, lo0.z, lo0.w, lo1.x, lo1.y, lo1.z, lo1.w};
    const uint32_t hi[8] = {hi0.x, hi0.y, hi0.z, hi0.w, hi1.x, hi1.y, hi1.z, hi1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 b = xs[j * 4 * G];
        uint32_t l[4], h[4];
        codes_to_f16(lo[j], l);
        codes_to_f16(hi[j], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[i] = hmul2_rn(l[i], slo[j >> 1]);
            h[i] = hmul2_rn(h[i], shi[j >> 1]);
        }
        mma16816(acc, l[0], h[0], l[1], h[1], b.x, b.y);
        mma16816(acc, l[2], h[2], l[3], h[3], b.z, b.w);
    }
}

struct Shared {
    int first[kMaxE + 1];   // groups of slots before expert e
    int count[kMaxE];       // slots of expert e
    int16_t ids[kIds];      // expert of a slot (-1: none), batches up to kIds slots
    int warp_sum[kWarps];
    int slot[8];            // the group's slots
    uint32_t top[8];        // largest finite |x| of each, as BF16 bits
    uint64_t full[kWarps * kMaxDepth];   // a ring place has its step
};

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

// Number of groups of each expert, as a prefix over the experts.
__device__ int count_groups(const MatvecArgs &a, Shared &sh, int per_group)
{
    const int slots = a.T * a.k;
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        sh.count[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const int e = read_id(a, s);
        if (slots <= kIds)
            sh.ids[s] = (int16_t)e;
        if (e >= 0)
            atomicAdd(&sh.count[e], 1);
        else if (e == -2 && blockIdx.x == 0)
            raise_status(a.status, kDevErrBadExpert);
    }
    __syncthreads();
    constexpr int kPer = kMaxE / kThreads;
    int g[kPer], mine = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        g[i] = e < a.E ? (sh.count[e] + per_group - 1) / per_group : 0;
        mine += g[i];
    }
    int at = cta_prefix(mine, sh.warp_sum, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e < a.E)
            sh.first[e] = at;
        at += g[i];
    }
    if (threadIdx.x == 0)
        sh.first[a.E] = total;
    __syncthreads();
    return total;
}

// Zero rows for the slots without an expert.
__device__ void zero_rows(const MatvecArgs &a, const Shared &sh)
{
    const int slots = a.T * a.k;
    for (int s = blockIdx.x; s < slots; s += gridDim.x)
        if (slot_expert(a, sh, s) < 0)
            for (int n = threadIdx.x; n < a.N; n += kThreads)
                a.y[(int64_t)s * a.N + n] = 0;
}

// The slots of expert e with rank [from, from + per_group), in slot order.
__device__ void find_slots(const MatvecArgs &a, Shared &sh, int e, int from, int per_group)
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
}

// The power of two that a slot's x is multiplied by: its largest element comes
// to [2^14, 2^15).  A subnormal largest counts as 2^-126.
__device__ __forceinline__ int x_shift(uint32_t top) { return top ? 14 - (max((int)(top >> 7), 1) - 127) : 0; }

// x of the group's m slots -> f16 in shared memory: elements 8q .. 8q + 7 of
// slot c at 16-byte place (((q / 32) * 8 + q % 8) * G + c) * 4 + (q / 8) % 4,
// which is where lane (c, t) looks for word q % 8 of its 64 elements of half
// step q / 32 (eight neighbouring lanes: 128 neighbouring bytes).
template <int G>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, Shared &sh, int m, uint4 *xs, int halves)
{
    const int nq = a.K / 8;
    const uint4 *x[G];
    uint32_t top[G];
#pragma unroll
    for (int c = 0; c < G; ++c) {
        const int s = sh.slot[c < m ? c : 0];
        x[c] = reinterpret_cast<const uint4 *>(a.x + (int64_t)(a.per_slot ? s : s / a.k) * a.ld_x);
        top[c] = 0;
    }
    for (int q = threadIdx.x; q < nq; q += kThreads) {
#pragma unroll
        for (int c = 0; c < G; ++c) {
            if (c >= m)
                break;
            const uint4 v = __ldg(x[c] + q);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t l = w[i] & 0x7fffu, h = (w[i] >> 16) & 0x7fffu;
                top[c] = max(top[c], max(l < 0x7f80u ? l : 0u, h < 0x7f80u ? h : 0u));
            }
        }
    }
#pragma unroll
    for (int c = 0; c < G; ++c) {
        const uint32_t w = __reduce_max_sync(0xffffffffu, top[c]);
        if (c < m && (threadIdx.x & 31) == 0 && w)
            atomicMax(&sh.top[c], w);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < G; ++c) {
        if (c >= m)
            break;
        // in two factors: the shift reaches 140
        const int shift = x_shift(sh.top[c]);
        const float2 f0 = make_float2(exp2i(shift / 2), exp2i(shift / 2));
        const float2 f1 = make_float2(exp2i(shift - shift / 2), exp2i(shift - shift / 2));
        for (int q = threadIdx.x; q < halves * 32; q += kThreads) {
            uint4 o = make_uint4(0, 0, 0, 0);
            if (q < nq) {
                const uint4 v = __ldg(x[c] + q);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = mul2(mul2(make_float2(u2f(w[i] << 16), u2f(w[i] & 0xffff0000u)), f0), f1);
                    h[i] = cvt_f16x2(p.x, p.y);
                }
                o = make_uint4(h[0], h[1], h[2], h[3]);
            }
            xs[(((q >> 5) * 8 + (q & 7)) * G + c) * 4 + ((q >> 3) & 3)] = o;
        }
    }
}

// Expert of a group of slots: the last one with first[e] <= group.
__device__ __forceinline__ int expert_of_group(const Shared &sh, int E, int group)
{
    int e = 0, hi = E - 1;
    while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (sh.first[mid] <= group)
            e = mid;
        else
            hi = mid - 1;
    }
    return e;
}

// Persistent: the (group of slots, tile of rows) pairs are dealt to the CTAs
// in contiguous ranges, so a CTA meets few groups; a CTA's warps take the
// pairs of its range in turn.  The steps of a warp's pairs run through its ring
// without a gap, also where the group changes.  G: columns of x in shared
// memory (slots per group).
template <int G>
__global__ void __launch_bounds__(kThreads, 1)
matvec_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap scales_map,
              MatvecArgs a, int depth)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint64_t *full = sh.full + warp * depth;
    if (lane == 0) {
        for (int i = 0; i < depth; ++i)
            mbar_init(full + i, 1);
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int groups = count_groups(a, sh, G);          // (its barriers publish the mbarriers too)
    const int tiles = (a.N + kTile - 1) / kTile;
    const int steps = (a.K + kStep - 1) / kStep, halves = (a.K + kHalf - 1) / kHalf;
    const int64_t total = (int64_t)groups * tiles;
    int64_t at = total * blockIdx.x / gridDim.x;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;

    uint8_t *codes = smem + (size_t)warp * depth * kCodeBytes;
    uint8_t *scales = smem + (size_t)kWarps * depth * kCodeBytes + (size_t)warp * depth * kScaleBytes;
    uint4 *xs = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * depth * (kCodeBytes + kScaleBytes));

    // the step to load next: tile p_tile of group p_group, step p_step, into place p_at
    int64_t p_item = at + warp;
    int p_group = 0, p_tile = 0, p_row = 0, p_step = 0, p_at = 0;
    auto locate = [&]() {
        if (p_item >= end)
            return;
        p_group = (int)(p_item / tiles);
        p_tile = (int)(p_item - (int64_t)p_group * tiles);
        p_row = expert_of_group(sh, a.E, p_group) * a.N + p_tile * kTile;
    };
    int in_flight = 0;
    auto load = [&]() {
        if (p_item >= end)
            return;
        if (lane == 0) {
            const bool two = 2 * p_step + 1 < halves;
            uint8_t *to = codes + p_at * kCodeBytes;
            mbar_arrive_expect_tx(full + p_at, (two ? kCodeBytes : kHalfBytes) + kScaleBytes);
            tma_load_2d(to, &codes_map, p_step * (kStep / 2), p_row, full + p_at);
            if (two)
                tma_load_2d(to + kHalfBytes, &codes_map, p_step * (kStep / 2) + kHalf / 2, p_row, full + p_at);
            tma_load_2d(scales + p_at * kScaleBytes, &scales_map, p_step * (kStep / 16), p_row, full + p_at);
        }
        ++in_flight;
        if (++p_at == depth)
            p_at = 0;
        if (++p_step == steps) {
            p_step = 0;
            p_item += kWarps;
            p_tile += kWarps;
            p_row += kWarps * kTile;
            if (p_tile >= tiles)
                locate();
        }
    };
    locate();
    for (int i = 0; i < depth; ++i)
        load();

    int64_t item = at + warp;
    int c_at = 0;
    uint32_t parity = 0;
    bool lost = false;                  // a wait gave up: no more loads, no more waits
    while (at < end) {
        const int group = (int)(at / tiles);
        const int64_t stop = min(end, (int64_t)(group + 1) * tiles);
        const int e = expert_of_group(sh, a.E, group);
        const int from = (group - sh.first[e]) * G;
        const int m = min(G, sh.count[e] - from);
        const uint8_t *w = a.w + (int64_t)e * a.N * a.S + a.S - 16;     // the row scales
        find_slots(a, sh, e, from, G);
        stage_x<G>(a, sh, m, xs, halves);
        __syncthreads();

        const uint4 *x_lane = xs + (g % G) * 4 + t;
        for (; item < stop && !lost; item += kWarps) {
            const int row = (int)(item - (int64_t)group * tiles) * kTile + g;
            const float row_lo = __ldg(reinterpret_cast<const float *>(w + (int64_t)min(row, a.N - 1) * a.S));
            const float row_hi = __ldg(reinterpret_cast<const float *>(w + (int64_t)min(row + 8, a.N - 1) * a.S));
            const uint4 *x = x_lane;
            float acc[4] = {};
            for (int s = 0; s < steps; ++s) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(full + c_at, parity))) {
                    lost = true;
                    break;
                }
                --in_flight;
                const uint8_t *c = codes + c_at * kCodeBytes + g * 128;
                const uint8_t *c0 = c + (((2 * t) ^ g) << 4), *c1 = c + (((2 * t + 1) ^ g) << 4);
                const uint8_t *sc = scales + c_at * kScaleBytes + g * (kStep / 16) + t * 4;
                multiply<G>(acc, c0, c1, sc, x);
                if (2 * s + 1 < halves)
                    multiply<G>(acc, c0 + kHalfBytes, c1 + kHalfBytes, sc + kHalf / 16, x + 32 * G);
                x += 64 * G;
                if (++c_at == depth) {
                    c_at = 0;
                    parity ^= 1u;
                }
                __syncwarp();           // every lane has read the place that is loaded next
                load();
            }
            if (lost)
                break;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = 2 * t + (v & 1), n = row + (v & 2 ? 8 : 0);
                if (c < m && n < a.N) {
                    // in 64 bits: the two scales together may pass FP32's range
                    const double back = __hiloint2double((1023 - x_shift(sh.top[c])) << 20, 0);
                    const double r = (double)acc[v] * (v & 2 ? row_hi : row_lo) * back;
                    a.y[(int64_t)sh.slot[c] * a.N + n] = (uint16_t)cvt_bf16x2((float)r, 0.0f);
                }
            }
        }
        at = stop;
        __syncthreads();                    // before the next group's x and slots
    }
    if (lost && lane == 0) {
        raise_status(a.status, kDevErrTimeout);
        // never leave with a load in flight
        for (; in_flight > 0; --in_flight) {
            (void)mbar_wait_bounded(full + c_at, parity);
            if (++c_at == depth) {
                c_at = 0;
                parity ^= 1u;
            }
        }
    }
    zero_rows(a, sh);
}

template <int G> cudaError_t launch_group(const LaunchCtx &c, const MatvecArgs &a, size_t x_bytes)
{
    static std::atomic<uint32_t> done[2] = {};
    cudaError_t e = ensure_smem_limit(matvec_kernel<G>, c.device, kMaxSmem, done);
    if (e != cudaSuccess)
        return e;
    const uint64_t rows = (uint64_t)a.E * a.N;
    CUtensorMap codes, scales;
    if (!make_map(&codes, a.w, (uint64_t)a.K / 2, rows, (uint64_t)a.S, kHalf / 2, kTile, true) ||
        !make_map(&scales, a.w + a.K / 2, (uint64_t)a.K / 16, rows, (uint64_t)a.S, kStep / 16, kTile))
        return cudaErrorInvalidValue;
    const size_t ring = (size_t)kWarps * (kCodeBytes + kScaleBytes);
    int depth = (int)((kMaxSmem - G * x_bytes) / ring);
    depth = depth > kMaxDepth ? kMaxDepth : depth;
    return launch_pdl(matvec_kernel<G>, dim3((unsigned)c.num_sms), dim3(kThreads), depth * ring + G * x_bytes,
                      c.stream, codes, scales, a, depth);
}

} // namespace

cudaError_t launch_matvec(const LaunchCtx &c, const MatvecArgs &a)
{
    if (a.T == 0)
        return cudaSuccess;
    // Slots of one expert that share a pass over its rows: as many as there are
    // tokens (a router names an expert once per token; if it is named more
    // often, it gets more passes), at most 8, and as leave the rings two steps.
    const size_t x_bytes = (size_t)((a.K + kHalf - 1) / kHalf) * kHalf * 2;
    const size_t room = kMaxSmem - (size_t)kMinDepth * kWarps * (kCodeBytes + kScaleBytes);
    if (a.T == 1)
        return launch_group<1>(c, a, x_bytes);
    if (a.T == 2 || 4 * x_bytes > room)
        return launch_group<2>(c, a, x_bytes);
    if (a.T <= 4 || 8 * x_bytes > room)
        return launch_group<4>(c, a, x_bytes);
    return launch_group<8>(c, a, x_bytes);
}

} // namespace epq
