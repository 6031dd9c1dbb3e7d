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
//    64 consecutive elements of rows g and g + 8 (two 16-byte loads each), so
//    a warp reads 128 contiguous bytes of every row, and no fragment shuffle
//    is needed; x lies in shared memory in the order in which the lanes want
//    it.
// A row's sum is computed by one warp in one order, whatever else is in the
// batch: a slot's result does not depend on the other slots.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;        // weight rows of a warp's tile
constexpr int kStep = 256;       // elements of a row that a warp takes at a time
constexpr int kDepth = 4;        // steps in flight per warp
constexpr int kMaxE = 1024;
constexpr int kIds = 2048;       // slots whose expert is kept in shared memory
constexpr int kMaxSmem = 200 * 1024;   // of x: three slots at the longest row, K = 32768

// A lane's share of a step: 64 elements of rows g and g + 8.
struct Step {
    uint4 lo0, lo1, hi0, hi1;
    uint32_t slo, shi;    // four block scales each
};

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

// 16 rows x 64 elements of this lane's share against its column of x, whose
// words lie 4 * G places apart.
template <int G>
__device__ __forceinline__ void multiply(float (&acc)[4], const Step &st, const uint4 *xs)
{
    uint32_t slo[4], shi[4];
    scale_pair(st.slo & 0xffffu, slo[0], slo[1]);
    scale_pair(st.slo >> 16, slo[2], slo[3]);
    scale_pair(st.shi & 0xffffu, shi[0], shi[1]);
    scale_pair(st.shi >> 16, shi[2], shi[3]);
    const uint32_t lo[8] = {st.lo0.x, st.lo0.y, st.lo0.z, st.lo0.w, st.lo1.x, st.lo1.y, st.lo1.z, st.lo1.w};
    const uint32_t hi[8] = {st.hi0.x, st.hi0.y, st.hi0.z, st.hi0.w, st.hi1.x, st.hi1.y, st.hi1.z, st.hi1.w};
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
// slot c at 16-byte place (((q / 32) * 8 + q % 8) * 4 + (q / 8) % 4) * G + c,
// which is where lane (c, t) looks for word q % 8 of its 64 elements of step
// q / 32.
template <int G>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, Shared &sh, int m, uint4 *xs, int steps)
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
        for (int q = threadIdx.x; q < steps * 32; q += kThreads) {
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
            xs[(((q >> 5) * 8 + (q & 7)) * 4 + ((q >> 3) & 3)) * G + c] = o;
        }
    }
}

// Persistent: the (group of slots, tile of rows) pairs are dealt to the CTAs
// in contiguous ranges, so a CTA meets few groups; its warps take the tiles of
// a group in turn, each with kDepth steps of loads in flight, the next tile's
// first ones among them.  G: columns of x in shared memory (slots per group).
// FULL: K is a whole number of steps.
template <int G, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(MatvecArgs a)
{
    extern __shared__ uint4 xs[];
    __shared__ Shared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int groups = count_groups(a, sh, G);
    const int tiles = (a.N + kTile - 1) / kTile;
    const int steps = (a.K + kStep - 1) / kStep;
    const int64_t total = (int64_t)groups * tiles;
    int64_t at = total * blockIdx.x / gridDim.x;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;

    while (at < end) {
        const int group = (int)(at / tiles);
        const int tile0 = (int)(at - (int64_t)group * tiles);
        const int tile1 = (int)min((int64_t)tiles, end - (int64_t)group * tiles);
        at += tile1 - tile0;
        int e = 0, hi = a.E - 1;            // last expert with first[e] <= group
        while (e < hi) {
            const int mid = (e + hi + 1) >> 1;
            if (sh.first[mid] <= group)
                e = mid;
            else
                hi = mid - 1;
        }
        const int from = (group - sh.first[e]) * G;
        const int m = min(G, sh.count[e] - from);

        const uint8_t *w = a.w + (int64_t)e * a.N * a.S;
        const uint8_t *lo, *hi8;            // this lane's rows of the tile being loaded
        Step st[kDepth];
        auto rows_of = [&](int tile) {      // rows past N read the last one
            lo = w + (int64_t)min(tile * kTile + g, a.N - 1) * a.S;
            hi8 = w + (int64_t)min(tile * kTile + g + 8, a.N - 1) * a.S;
        };
        auto load = [&](Step &p, int step) {
            const int k0 = step * kStep + t * 64;
            if (FULL || k0 + 32 < a.K) {
                p.lo0 = __ldg(reinterpret_cast<const uint4 *>(lo + k0 / 2));
                p.lo1 = __ldg(reinterpret_cast<const uint4 *>(lo + k0 / 2 + 16));
                p.hi0 = __ldg(reinterpret_cast<const uint4 *>(hi8 + k0 / 2));
                p.hi1 = __ldg(reinterpret_cast<const uint4 *>(hi8 + k0 / 2 + 16));
                p.slo = __ldg(reinterpret_cast<const uint32_t *>(lo + a.K / 2 + k0 / 16));
                p.shi = __ldg(reinterpret_cast<const uint32_t *>(hi8 + a.K / 2 + k0 / 16));
            } else {
                p.lo0 = p.lo1 = p.hi0 = p.hi1 = make_uint4(0, 0, 0, 0);
                p.slo = p.shi = 0;
                if (k0 < a.K) {             // the row ends after 32 elements and two scales
                    p.lo0 = __ldg(reinterpret_cast<const uint4 *>(lo + k0 / 2));
                    p.hi0 = __ldg(reinterpret_cast<const uint4 *>(hi8 + k0 / 2));
                    p.slo = __ldg(reinterpret_cast<const uint16_t *>(lo + a.K / 2 + k0 / 16));
                    p.shi = __ldg(reinterpret_cast<const uint16_t *>(hi8 + a.K / 2 + k0 / 16));
                }
            }
        };
        int tile = tile0 + warp;
        float scale_lo = 0.0f, scale_hi = 0.0f;
        if (tile < tile1) {
            rows_of(tile);
#pragma unroll
            for (int d = 0; d < kDepth; ++d)
                if (d < steps)
                    load(st[d], d);
            scale_lo = __ldg(reinterpret_cast<const float *>(lo + a.S - 16));
            scale_hi = __ldg(reinterpret_cast<const float *>(hi8 + a.S - 16));
        }

        find_slots(a, sh, e, from, G);
        stage_x<G>(a, sh, m, xs, steps);
        __syncthreads();

        const uint4 *x_lane = xs + t * G + g % G;
        while (tile < tile1) {
            const int next = tile + kWarps;
            const uint4 *x = x_lane;
            float acc[4] = {};
            for (int s0 = 0; s0 < steps; s0 += kDepth) {
                const bool last = s0 + kDepth >= steps;
                if (last && next < tile1)
                    rows_of(next);
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    if (s0 + d < steps)
                        multiply<G>(acc, st[d], x + d * 32 * G);
                    const int ahead = last ? d : s0 + kDepth + d;
                    if ((!last || next < tile1) && ahead < steps)
                        load(st[d], ahead);
                }
                x += kDepth * 32 * G;
            }
            const float row_lo = scale_lo, row_hi = scale_hi;
            if (next < tile1) {
                scale_lo = __ldg(reinterpret_cast<const float *>(lo + a.S - 16));
                scale_hi = __ldg(reinterpret_cast<const float *>(hi8 + a.S - 16));
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = 2 * t + (v & 1), n = tile * kTile + g + (v & 2 ? 8 : 0);
                if (c < m && n < a.N) {
                    // in 64 bits: the two scales together may pass FP32's range
                    const double back = __hiloint2double((1023 - x_shift(sh.top[c])) << 20, 0);
                    const double r = (double)acc[v] * (v & 2 ? row_hi : row_lo) * back;
                    a.y[(int64_t)sh.slot[c] * a.N + n] = (uint16_t)cvt_bf16x2((float)r, 0.0f);
                }
            }
            tile = next;
        }
        __syncthreads();                    // before the next group's x and slots
    }
    zero_rows(a, sh);
}

template <int G, bool FULL> cudaError_t launch_group(const LaunchCtx &c, const MatvecArgs &a, size_t smem)
{
    static std::atomic<uint32_t> done[2] = {};
    cudaError_t e = ensure_smem_limit(matvec_kernel<G, FULL>, c.device, kMaxSmem, done);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(matvec_kernel<G, FULL>, dim3((unsigned)c.num_sms), dim3(kThreads), smem, c.stream, a);
}

template <int G> cudaError_t launch_steps(const LaunchCtx &c, const MatvecArgs &a, size_t x_bytes)
{
    return a.K % kStep == 0 ? launch_group<G, true>(c, a, G * x_bytes) : launch_group<G, false>(c, a, G * x_bytes);
}

} // namespace

cudaError_t launch_matvec(const LaunchCtx &c, const MatvecArgs &a)
{
    if (a.T == 0)
        return cudaSuccess;
    // Slots of one expert that share a pass over its rows: as many as there are
    // tokens (a router names an expert once per token; if it is named more
    // often, it gets more passes), at most 8, and as fit in shared memory.
    const size_t x_bytes = (size_t)((a.K + kStep - 1) / kStep) * kStep * 2;
    if (a.T == 1 || 2 * x_bytes > kMaxSmem)
        return launch_steps<1>(c, a, x_bytes);
    if (a.T == 2 || 4 * x_bytes > kMaxSmem)
        return launch_steps<2>(c, a, x_bytes);
    if (a.T <= 4 || 8 * x_bytes > kMaxSmem)
        return launch_steps<4>(c, a, x_bytes);
    return launch_steps<8>(c, a, x_bytes);
}

} // namespace epq
