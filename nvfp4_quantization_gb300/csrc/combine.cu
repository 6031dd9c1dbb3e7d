// Tokens to expert rows and back, unquantised (BF16 or FP32), with the
// router's weights and the gradients.
//
//   ep_pack              rows[d(t,j)] = tokens[t],          padding rows = 0
//   ep_combine           out[t] = sum_j w(t,j) rows[d(t,j)]
//   ep_combine_backward  d_rows[d(t,j)] = w(t,j) d_out[t],  padding rows = 0
//                        d_w(t,j) = <d_out[t], rows[d(t,j)]>
//
// d(t,j) is the row the routing plan gave slot j of token t (negative: the
// slot was dropped).  Every product and sum is FP32 and is rounded once, on
// the way out; the sum over slots is in slot order and the dot products are
// reduced in a fixed tree, so results do not depend on scheduling.
//
// Bound: HBM; each row, token and gradient passes once, in 16-byte blocks, with
// the loads of a token's slots in flight together.
// Measured on GB300 at 16384 tokens x 7168, BF16: pack, 64 experts top-6 254 us
// (6.5 TB/s, padding rows not counted), combine, 256 experts top-8 336 us (6.3
// TB/s), its gradient with the weights' 629 us (6.3 TB/s, 6.7 with the padding
// rows).
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 256;

// Everything moves in blocks of 16 bytes of a row, E elements of type T.
template <typename T> constexpr int E = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(uint4 r, float (&f)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = u2f(w[i] << 16);
        f[2 * i + 1] = u2f(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(uint4 r, float (&f)[4])
{
    f[0] = u2f(r.x);
    f[1] = u2f(r.y);
    f[2] = u2f(r.z);
    f[3] = u2f(r.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8])
{
    return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4])
{
    return make_uint4(f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3]));
}

__device__ __forceinline__ uint4 load16(const void *p) { return __ldg(static_cast<const uint4 *>(p)); }

// ---------------------------------------------------------------- rows that start anywhere
// E elements from any element's address, as the two aligned 16-byte words that
// hold them (the second is the neighbouring thread's first: it comes from L1)
// and a shift by a number of bytes that is the same all along a row.  For the
// blocks at a row's ends the words reach up to 28 bytes before it and 32 after
// it, into its neighbours; rows that have less of the buffer there (its first
// and last) are read element by element.
template <typename T> __device__ __forceinline__ bool inner_row(int64_t row, int64_t rows, int64_t ld)
{
    return row * ld * (int)sizeof(T) >= 32 && (rows - 1 - row) * ld * (int)sizeof(T) >= 32;
}

struct Window {
    uint4 lo, hi;
    uint32_t shift;
};

template <typename T>
__device__ __forceinline__ Window load_window(const T *p, bool inner, int first, int n)
{
    Window w;
    if (inner) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        w.shift = (uint32_t)at & 15u;
        const uint4 *q = reinterpret_cast<const uint4 *>(at - w.shift);
        w.lo = __ldg(q);
        w.hi = __ldg(q + (w.shift ? 1 : 0));
    } else {
        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < E<T>; ++i)
            if (i >= first && i < n) {
                if constexpr (sizeof(T) == 2)
                    v[i / 2] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
                else
                    v[i] = f2u(__ldg(p + i));
            }
        w.lo = w.hi = make_uint4(v[0], v[1], v[2], v[3]);
        w.shift = 0;
    }
    return w;
}

__device__ __forceinline__ uint4 value(const Window &w)
{
    const uint32_t r = 8 * (w.shift & 3u);
    auto at = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e) {
        return make_uint4(__funnelshift_r(a, b, r), __funnelshift_r(b, c, r), __funnelshift_r(c, d, r),
                          __funnelshift_r(d, e, r));
    };
    switch (w.shift >> 2) {
    case 0: return at(w.lo.x, w.lo.y, w.lo.z, w.lo.w, w.hi.x);
    case 1: return at(w.lo.y, w.lo.z, w.lo.w, w.hi.x, w.hi.y);
    case 2: return at(w.lo.z, w.lo.w, w.hi.x, w.hi.y, w.hi.z);
    default: return at(w.lo.w, w.hi.x, w.hi.y, w.hi.z, w.hi.w);
    }
}

// Elements [first, n) of a block to p, which is 16-byte aligned where all of
// them are there.
template <typename T>
__device__ __forceinline__ void store_part(T *p, uint4 v, int first, int n)
{
    if (first == 0 && n == E<T>) {
        *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < E<T>; ++i)
        if (i >= first && i < n) {
            if constexpr (sizeof(T) == 2)
                p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            else
                p[i] = u2f(w[i]);
        }
}

// Elements between p and the 16-byte boundary before it.
template <typename T> __device__ __forceinline__ int before(const T *p)
{
    return (int)(reinterpret_cast<uintptr_t>(p) & 15u) / (int)sizeof(T);
}

// A CTA's token.  SHORT: blockDim.y tokens a CTA, for rows that leave most of
// one's threads idle (16121 tokens x 192, top-1: 19 us with a CTA of a warp each,
// 6 with eight tokens a CTA).  Kept apart because a token that is the same for
// the whole CTA costs a fifth of the registers less.
template <bool SHORT> __device__ __forceinline__ int64_t token_of()
{
    return SHORT ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : (int64_t)blockIdx.x;
}

// Row of a slot, or -1 for a dropped one; a row outside the buffer is
// reported and dropped.
__device__ __forceinline__ int live_row(int d, int R_cap, uint32_t *status)
{
    if (d >= R_cap) {
        raise_status(status, kDevErrCapacity);
        return -1;
    }
    return d < 0 ? -1 : d;
}

// ---------------------------------------------------------------- combine
// Rows (as they are given) and weights of KCH slots of a token from slot j0 on.
template <int KCH>
__device__ __forceinline__ void read_slots(const CombineArgs &a, int64_t slot0, int j0, int (&d)[KCH], float (&w)[KCH])
{
#pragma unroll
    for (int j = 0; j < KCH; ++j) {
        d[j] = -1;
        w[j] = 1.0f;
        if (j0 + j < a.k) {
            const int64_t s = slot0 + j0 + j;
            d[j] = a.index ? __ldg(a.index + s) : 0;
            if (a.slot_order && d[j] >= 0)
                d[j] = (int)s;
            if (a.weights)
                w[j] = __ldg(a.weights + s);
        }
    }
}

// Rows of whole 16-byte blocks.  One thread per UNR blocks of a token, a CTA's
// share of the row side by side; the rows of KCH slots are in flight at once.
// With two slots, two blocks: one leaves too few bytes in flight (8192 x 4096
// FP32 top-2: 71 us, with two 59 us; with eight slots two cost 3 %).
template <typename T, int KCH, bool SHORT>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a)
{
    constexpr int UNR = KCH > 2 ? 1 : 2;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = token_of<SHORT>();
    const int c0 = (blockIdx.y * UNR * blockDim.x + threadIdx.x) * E<T>, step = blockDim.x * E<T>;
    if ((SHORT && t >= a.T) || c0 >= a.H)
        return;
    const T *rows = static_cast<const T *>(a.rows);
    float acc[UNR][E<T>] = {};
    for (int j0 = 0; j0 < a.k; j0 += KCH) {
        int d[KCH];
        float w[KCH];
        read_slots<KCH>(a, t * a.k, j0, d, w);
        uint4 raw[KCH][UNR];
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            d[j] = live_row(d[j], a.R_cap, a.status);
            if (d[j] >= 0) {
#pragma unroll
                for (int u = 0; u < UNR; ++u)
                    if (c0 + u * step < a.H)
                        raw[j][u] = load16(rows + (int64_t)d[j] * a.ld_rows + c0 + u * step);
            }
        }
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            if (d[j] < 0)
                continue;
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                float f[E<T>];
                unpack(raw[j][u], f);
#pragma unroll
                for (int i = 0; i < E<T>; ++i)
                    acc[u][i] = fmaf(w[j], f[i], acc[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u)
        if (c0 + u * step < a.H)
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + t * a.H + c0 + u * step) = pack(acc[u]);
}

// Rows that start anywhere: a thread has one aligned block of the output (part
// of one at the row's ends) and a window of each row (8192 x 7001 BF16 top-8: 203
// us; with loads of single elements, four a thread, 356).
template <typename T, int KCH, bool SHORT>
__global__ void __launch_bounds__(kThreads) combine_any_kernel(CombineArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = token_of<SHORT>();
    if (SHORT && t >= a.T)
        return;
    T *out = static_cast<T *>(a.out) + t * a.H;
    const int c = (int)(blockIdx.y * blockDim.x + threadIdx.x) * E<T> - before(out);
    if (c >= a.H)
        return;
    const int first = c < 0 ? -c : 0, n = min(E<T>, a.H - c);
    const T *rows = static_cast<const T *>(a.rows);
    float acc[E<T>] = {};
    for (int j0 = 0; j0 < a.k; j0 += KCH) {
        int d[KCH];
        float w[KCH];
        read_slots<KCH>(a, t * a.k, j0, d, w);
        Window raw[KCH];
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            d[j] = live_row(d[j], a.R_cap, a.status);
            if (d[j] >= 0)
                raw[j] = load_window<T>(rows + (int64_t)d[j] * a.ld_rows + c, inner_row<T>(d[j], a.R_cap, a.ld_rows),
                                        first, n);
        }
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            if (d[j] < 0)
                continue;
            float f[E<T>];
            unpack(value(raw[j]), f);
#pragma unroll
            for (int i = 0; i < E<T>; ++i)
                acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    }
    store_part<T>(out + c, pack(acc), first, n);
}

// ---------------------------------------------------------------- scatter
// Zero the padding rows [offsets[e] + counts[e], offsets[e + 1]) of expert
// e = cta / a.pad_split, every a.pad_split-th row of them (and of those, if
// SHORT, this threadIdx.y's).
template <typename T, bool SHORT>
__device__ void zero_padding(const ScatterArgs &a, int cta)
{
    const int e = cta / a.pad_split;
    const int end = __ldg(a.offsets + e + 1);
    T *rows = static_cast<T *>(a.rows_out);
    const int first = __ldg(a.offsets + e) + __ldg(a.counts + e) + (SHORT ? (int)threadIdx.y * a.pad_split : 0);
    for (int r = first + cta % a.pad_split; r < end; r += SHORT ? a.pad_split * (int)blockDim.y : a.pad_split) {
        if (r < 0 || r >= a.R_cap) {
            if (threadIdx.x == 0)
                raise_status(a.status, kDevErrCapacity);
            return;
        }
        for (int c = threadIdx.x * E<T>; c < a.H; c += blockDim.x * E<T>)
            *reinterpret_cast<uint4 *>(rows + (int64_t)r * a.H + c) = make_uint4(0, 0, 0, 0);
    }
}

// Rows of whole 16-byte blocks: a token (SHORT: blockDim.y of them) a CTA, read
// once by its blockDim.x threads; CTAs past the tokens write the padding rows.
template <typename T, int KCH, bool DOT, bool SHORT>
__global__ void __launch_bounds__(kThreads) scatter_kernel(ScatterArgs a)
{
    __shared__ float part[kThreads / 32][KCH];
    pdl_launch_dependents();
    pdl_wait();
    const int token_ctas = SHORT ? (a.T + (int)blockDim.y - 1) / (int)blockDim.y : a.T;
    if ((int)blockIdx.x >= token_ctas) {
        zero_padding<T, SHORT>(a, blockIdx.x - token_ctas);
        return;
    }
    const int64_t t = token_of<SHORT>();
    const bool here = !SHORT || t < a.T;    // (the last CTA's may not be)
    const int64_t slot0 = t * a.k;
    const T *src = static_cast<const T *>(a.src) + t * a.ld_src;
    const T *rows_in = static_cast<const T *>(a.rows_in);
    T *rows_out = static_cast<T *>(a.rows_out);
    for (int j0 = 0; j0 < a.k; j0 += KCH) {
        int d[KCH];
        float w[KCH], dot[KCH];
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            d[j] = -1;
            w[j] = 1.0f;
            dot[j] = 0.0f;
            if (here && j0 + j < a.k) {
                d[j] = live_row(__ldg(a.dest + slot0 + j0 + j), a.R_cap, a.status);
                if (a.weights)
                    w[j] = __ldg(a.weights + slot0 + j0 + j);
            }
        }
        for (int c = here ? threadIdx.x * E<T> : a.H; c < a.H; c += blockDim.x * E<T>) {
            const uint4 raw = load16(src + c);
            uint4 in[KCH];
            if (DOT) {
#pragma unroll
                for (int j = 0; j < KCH; ++j)
                    if (d[j] >= 0)
                        in[j] = load16(rows_in + (int64_t)d[j] * a.ld_in + c);
            }
            float f[E<T>];
            unpack(raw, f);
#pragma unroll
            for (int j = 0; j < KCH; ++j) {
                if (d[j] < 0)
                    continue;
                uint4 *to = reinterpret_cast<uint4 *>(rows_out + (int64_t)d[j] * a.H + c);
                if (a.weights) {
                    float o[E<T>];
#pragma unroll
                    for (int i = 0; i < E<T>; ++i)
                        o[i] = w[j] * f[i];
                    *to = pack(o);
                } else {
                    *to = raw;
                }
                if (DOT) {
                    float g[E<T>];
                    unpack(in[j], g);
#pragma unroll
                    for (int i = 0; i < E<T>; ++i)
                        dot[j] = fmaf(f[i], g[i], dot[j]);
                }
            }
        }
        if (DOT) {
            const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            const int warp0 = SHORT ? threadIdx.y * warps : 0, warp = warp0 + (threadIdx.x >> 5);
#pragma unroll
            for (int j = 0; j < KCH; ++j) {
                float v = dot[j];
                for (int o = 16; o; o >>= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0)
                    part[warp][j] = v;
            }
            __syncthreads();
            if (here && (int)threadIdx.x < KCH && j0 + (int)threadIdx.x < a.k) {
                float v = 0.0f;
                for (int i = 0; i < warps; ++i)
                    v += part[warp0 + i][threadIdx.x];
                a.d_weights[slot0 + j0 + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
}

// The same for rows that start anywhere: an expert's padding rows lie together,
// and a CTA zeroes a share of their elements.
template <typename T>
__device__ void zero_padding_any(const ScatterArgs &a, int cta)
{
    const int e = cta / a.pad_split, part = cta % a.pad_split;
    const int64_t row0 = (int64_t)__ldg(a.offsets + e) + __ldg(a.counts + e);
    int64_t row1 = __ldg(a.offsets + e + 1);
    if (row1 > a.R_cap || row0 < 0) {
        if (threadIdx.x == 0)
            raise_status(a.status, kDevErrCapacity);
        row1 = min(row1, (int64_t)a.R_cap);
    }
    if (row0 < 0 || row0 >= row1)
        return;
    const int64_t all = (row1 - row0) * a.H;
    T *p = static_cast<T *>(a.rows_out) + row0 * a.H + all * part / a.pad_split;
    T *end = static_cast<T *>(a.rows_out) + row0 * a.H + all * (part + 1) / a.pad_split;
    const int head = (int)min((int64_t)((E<T> - before(p)) % E<T>), (int64_t)(end - p));
    if ((int)threadIdx.x < head)
        p[threadIdx.x] = T(0);
    p += head;
    const int64_t blocks = (end - p) / E<T>;
    for (int64_t b = threadIdx.x; b < blocks; b += blockDim.x)
        reinterpret_cast<uint4 *>(p)[b] = make_uint4(0, 0, 0, 0);
    p += blocks * E<T>;
    if (p + threadIdx.x < end)
        p[threadIdx.x] = T(0);
}

// Rows that start anywhere: L threads per slot, a warp (a CTA where slots are
// few: 96 slots of 3993 FP32 took 20 us on one warp each; a quarter of a warp
// for short rows without a sum along them: 25032 slots of 117 took 18), because
// each of a token's rows wants the token at another shift; the token is read k
// times, from L1 and L2 after the first.  A lane has U aligned blocks of the row (parts of one at its
// ends) and the windows that belong to them in flight (with two windows a block,
// two blocks of BF16: 8192 x 7001 top-6 296 us, with one 314; one of FP32: 1021
// x 1001 top-5 14.9 us, with two 18.1).
template <typename T, bool DOT, int L>
__global__ void __launch_bounds__(kThreads) scatter_any_kernel(ScatterArgs a)
{
    constexpr int U = !DOT ? 4 : sizeof(T) == 2 ? 2 : 1, kSlots = kThreads / L;
    __shared__ float part[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t slots = (int64_t)a.T * a.k;
    const int slot_ctas = (int)((slots + kSlots - 1) / kSlots);
    if ((int)blockIdx.x >= slot_ctas) {
        zero_padding_any<T>(a, blockIdx.x - slot_ctas);
        return;
    }
    const int lane = threadIdx.x % L;
    const int64_t s = (int64_t)blockIdx.x * kSlots + threadIdx.x / L;
    const int d = s < slots ? live_row(__ldg(a.dest + s), a.R_cap, a.status) : -1;
    float dot = 0.0f;
    if (d >= 0) {
        const int64_t t = s / a.k;
        const float w = a.weights ? __ldg(a.weights + s) : 1.0f;
        const T *src = static_cast<const T *>(a.src) + t * a.ld_src;
        const T *in = DOT ? static_cast<const T *>(a.rows_in) + (int64_t)d * a.ld_in : nullptr;
        T *to = static_cast<T *>(a.rows_out) + (int64_t)d * a.H;
        const bool src_inner = inner_row<T>(t, a.T, a.ld_src), in_inner = DOT && inner_row<T>(d, a.R_cap, a.ld_in);
        for (int c0 = lane * E<T> - before(to); c0 < a.H; c0 += L * U * E<T>) {
            Window x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * L * E<T>;
                if (c >= a.H)
                    break;
                const int first = c < 0 ? -c : 0, n = min(E<T>, a.H - c);
                x[u] = load_window<T>(src + c, src_inner, first, n);
                if (DOT)
                    y[u] = load_window<T>(in + c, in_inner, first, n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * L * E<T>;
                if (c >= a.H)
                    break;
                const int first = c < 0 ? -c : 0, n = min(E<T>, a.H - c);
                const uint4 raw = value(x[u]);
                float f[E<T>];
                unpack(raw, f);
                if (a.weights) {
                    float o[E<T>];
#pragma unroll
                    for (int i = 0; i < E<T>; ++i)
                        o[i] = w * f[i];
                    store_part<T>(to + c, pack(o), first, n);
                } else {
                    store_part<T>(to + c, raw, first, n);
                }
                if (DOT) {
                    float g[E<T>];
                    unpack(value(y[u]), g);
#pragma unroll
                    for (int i = 0; i < E<T>; ++i)
                        if (i >= first && i < n)
                            dot = fmaf(f[i], g[i], dot);
                }
            }
        }
    }
    if (DOT) {
        for (int o = L < 32 ? L / 2 : 16; o; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (L > 32) {
            if ((lane & 31) == 0)
                part[lane / 32] = dot;
            __syncthreads();
            dot = 0.0f;
            for (int i = 0; i < L / 32; ++i)
                dot += part[i];
        }
        if (lane == 0 && s < slots)
            a.d_weights[s] = dot;
    }
}

// Every row starts on 16 bytes and is a whole number of them.
bool in_blocks(const void *p, int64_t ld, int64_t H, int elem)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elem) % 16 == 0 && (H * elem) % 16 == 0;
}

// Threads for `units` of work side by side: the fewest whole warps that take
// them in the same number of CTAs as kThreads would; short rows several to a
// CTA.
dim3 block_of(int64_t units)
{
    const int64_t passes = (units + kThreads - 1) / kThreads;
    const int x = (int)(((units + passes - 1) / passes + 31) / 32 * 32);
    return dim3(x, kThreads / x);
}

template <typename T, int KCH> cudaError_t combine_slots(const LaunchCtx &c, const CombineArgs &a, bool blocks)
{
    constexpr int UNR = KCH > 2 ? 1 : 2;
    // (a row that starts inside a block has up to one block more)
    const int64_t n = blocks ? (a.H / E<T> + UNR - 1) / UNR : (a.H + 2 * E<T> - 2) / E<T>;
    const dim3 block = block_of(n);
    const dim3 grid((unsigned)((a.T + block.y - 1) / block.y), (unsigned)((n + block.x - 1) / block.x));
    constexpr int K2 = KCH == 8 ? E<T> / 2 : KCH;
    if (block.y > 1)
        return blocks ? launch_pdl(combine_kernel<T, KCH, true>, grid, block, 0, c.stream, a)
                      : launch_pdl(combine_any_kernel<T, K2, true>, grid, block, 0, c.stream, a);
    return blocks ? launch_pdl(combine_kernel<T, KCH, false>, grid, block, 0, c.stream, a)
                  : launch_pdl(combine_any_kernel<T, K2, false>, grid, block, 0, c.stream, a);
}

template <typename T> cudaError_t combine_type(const LaunchCtx &c, const CombineArgs &a)
{
    const bool blocks = in_blocks(a.rows, a.ld_rows, a.H, sizeof(T)) && in_blocks(a.out, a.H, a.H, sizeof(T));
    return a.k <= 2 ? combine_slots<T, 2>(c, a, blocks) : combine_slots<T, 8>(c, a, blocks);
}

template <typename T, bool DOT> cudaError_t scatter_type(const LaunchCtx &c, ScatterArgs a)
{
    // CTAs an expert's padding rows are shared by.  Few leave a long tail where
    // rows are long, many are mostly idle where they are short (pack, 8 against
    // 32: 64 experts, 4096 x 4096 top-6 43.7, 41.5 us, 2048 x 1001 12.4, 14.0; 256
    // experts top-8, 65.6, 63.1 and 18.9, 30.6).
    a.pad_split = a.E >= 256 ? 8 : 32;
    const unsigned pad = (unsigned)(a.E * a.pad_split);
    if (!(in_blocks(a.src, a.ld_src, a.H, sizeof(T)) && in_blocks(a.rows_out, a.H, a.H, sizeof(T)) &&
          in_blocks(a.rows_in, a.rows_in ? a.ld_in : 0, a.H, sizeof(T)))) {
        const int64_t slots = (int64_t)a.T * a.k;
        auto grid = [&](int per_cta) { return dim3((unsigned)((slots + per_cta - 1) / per_cta) + pad); };
        if (!DOT && a.H <= 16 * E<T>)
            return launch_pdl(scatter_any_kernel<T, false, 8>, grid(kThreads / 8), dim3(kThreads), 0, c.stream, a);
        // A CTA a slot where a warp a slot would leave the SMs with less than two
        // CTAs each.  That is where rows of a warp's many turns gain (gradient, 600
        // slots of 3993: FP32 10.7 us on CTAs, 38.0 on warps, BF16 5.6, 16.2; 2432
        // slots 21.0, 41.1 and 15.3, 20.5); rows of one or two turns lose a little
        // (1200 slots of BF16: 1001 5.2, 4.7 us; 331 5.0, 3.2).
        if (slots < (int64_t)c.num_sms * 2 * (kThreads / 32))
            return launch_pdl(scatter_any_kernel<T, DOT, kThreads>, grid(1), dim3(kThreads), 0, c.stream, a);
        return launch_pdl(scatter_any_kernel<T, DOT, 32>, grid(kThreads / 32), dim3(kThreads), 0, c.stream, a);
    }
    const int64_t units = a.H / E<T>;
    const int x = (int)(units >= kThreads ? kThreads : (units + 31) / 32 * 32);
    const dim3 block(x, kThreads / x);
    const dim3 grid((a.T + block.y - 1) / block.y + pad);
    if (block.y > 1)
        return a.k <= 2 ? launch_pdl(scatter_kernel<T, 2, DOT, true>, grid, block, 0, c.stream, a)
                        : launch_pdl(scatter_kernel<T, 8, DOT, true>, grid, block, 0, c.stream, a);
    return a.k <= 2 ? launch_pdl(scatter_kernel<T, 2, DOT, false>, grid, block, 0, c.stream, a)
                    : launch_pdl(scatter_kernel<T, 8, DOT, false>, grid, block, 0, c.stream, a);
}

template <typename T> cudaError_t scatter_dot(const LaunchCtx &c, const ScatterArgs &a)
{
    return a.d_weights ? scatter_type<T, true>(c, a) : scatter_type<T, false>(c, a);
}

} // namespace

cudaError_t launch_combine(const LaunchCtx &c, const CombineArgs &a, int dtype)
{
    if (a.T == 0)
        return cudaSuccess;
    return dtype == kF32 ? combine_type<float>(c, a) : combine_type<uint16_t>(c, a);
}

cudaError_t launch_scatter(const LaunchCtx &c, const ScatterArgs &a, int dtype)
{
    return dtype == kF32 ? scatter_dot<float>(c, a) : scatter_dot<uint16_t>(c, a);
}

} // namespace epq
