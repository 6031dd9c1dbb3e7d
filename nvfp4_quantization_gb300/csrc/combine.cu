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
// Bound: HBM; each row, token and gradient passes once, in 16-byte units where
// the rows allow it, with the loads of all of a token's slots in flight together.
// Measured on GB300 at 16384 tokens x 7168, BF16: pack, 64 experts top-6 255 us
// (6.4 TB/s, padding rows not counted), combine, 256 experts top-8 335 us (6.3
// TB/s), its gradient with the weights' 631 us (6.3 TB/s, 6.7 with the padding
// rows).
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 256;

// What a thread loads and stores at a time, a unit: VEC consecutive elements of
// type T, 16 bytes where every row starts on 16 bytes and is a whole number of
// them, else 4, else (BF16 rows of odd length) one element.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int VEC> using RawOf = typename Raw<(int)sizeof(T) * VEC>::type;

template <typename T, int VEC>
__device__ __forceinline__ RawOf<T, VEC> load_raw(const T *p)
{
    return __ldg(reinterpret_cast<const RawOf<T, VEC> *>(p));
}

template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T *p, RawOf<T, VEC> v)
{
    *reinterpret_cast<RawOf<T, VEC> *>(p) = v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return u2f(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return u2f(w & 0xffff0000u); }

__device__ __forceinline__ void unpack_raw(uint4 r, float (&f)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void unpack_raw(uint32_t r, float (&f)[2])
{
    f[0] = bf16_lo(r);
    f[1] = bf16_hi(r);
}
__device__ __forceinline__ void unpack_raw(uint16_t r, float (&f)[1]) { f[0] = u2f((uint32_t)r << 16); }
__device__ __forceinline__ void unpack_raw(uint4 r, float (&f)[4])
{
    f[0] = u2f(r.x);
    f[1] = u2f(r.y);
    f[2] = u2f(r.z);
    f[3] = u2f(r.w);
}
__device__ __forceinline__ void unpack_raw(uint32_t r, float (&f)[1]) { f[0] = u2f(r); }

template <typename T, int VEC> __device__ __forceinline__ RawOf<T, VEC> pack_raw(const float (&f)[VEC]);
template <> __device__ __forceinline__ uint4 pack_raw<uint16_t, 8>(const float (&f)[8])
{
    return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}
template <> __device__ __forceinline__ uint32_t pack_raw<uint16_t, 2>(const float (&f)[2])
{
    return cvt_bf16x2(f[0], f[1]);
}
template <> __device__ __forceinline__ uint16_t pack_raw<uint16_t, 1>(const float (&f)[1])
{
    return (uint16_t)cvt_bf16x2(f[0], 0.0f);
}
template <> __device__ __forceinline__ uint4 pack_raw<float, 4>(const float (&f)[4])
{
    return make_uint4(f2u(f[0]), f2u(f[1]), f2u(f[2]), f2u(f[3]));
}
template <> __device__ __forceinline__ uint32_t pack_raw<float, 1>(const float (&f)[1]) { return f2u(f[0]); }

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
// One thread per UNR units of a token, a CTA's share of the row side by side;
// the rows of KCH slots are in flight at once.  Narrow units come several to a
// thread: with one, too few bytes are in flight (4096 tokens x 4097, top-4,
// FP32: 115 us; with two 83 us).
template <typename T, int VEC, int KCH> constexpr int units_in_flight()
{
    return sizeof(T) * VEC >= 16 ? (KCH > 2 ? 1 : 2) : sizeof(T) * VEC >= 4 && KCH > 2 ? 2 : 4;
}

template <typename T, int VEC, int KCH>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a)
{
    constexpr int UNR = units_in_flight<T, VEC, KCH>();
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int c0 = (blockIdx.y * UNR * blockDim.x + threadIdx.x) * VEC, step = blockDim.x * VEC;
    if (c0 >= a.H)
        return;
    const T *rows = static_cast<const T *>(a.rows);
    const int64_t slot0 = t * a.k;
    float acc[UNR][VEC] = {};
    for (int j0 = 0; j0 < a.k; j0 += KCH) {
        int d[KCH];
        float w[KCH];
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
        RawOf<T, VEC> raw[KCH][UNR];
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            d[j] = live_row(d[j], a.R_cap, a.status);
            if (d[j] >= 0) {
#pragma unroll
                for (int u = 0; u < UNR; ++u)
                    if (c0 + u * step < a.H)
                        raw[j][u] = load_raw<T, VEC>(rows + (int64_t)d[j] * a.ld_rows + c0 + u * step);
            }
        }
#pragma unroll
        for (int j = 0; j < KCH; ++j) {
            if (d[j] < 0)
                continue;
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                float f[VEC];
                unpack_raw(raw[j][u], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    acc[u][i] = fmaf(w[j], f[i], acc[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u)
        if (c0 + u * step < a.H)
            store_raw<T, VEC>(static_cast<T *>(a.out) + t * a.H + c0 + u * step, pack_raw<T, VEC>(acc[u]));
}

// ---------------------------------------------------------------- scatter
// Zero the padding rows [offsets[e] + counts[e], offsets[e + 1]) of expert
// e = cta / a.pad_split, every a.pad_split-th row of them.
template <typename T, int VEC>
__device__ void zero_padding(const ScatterArgs &a, int cta)
{
    const int e = cta / a.pad_split;
    const int end = __ldg(a.offsets + e + 1);
    T *rows = static_cast<T *>(a.rows_out);
    const RawOf<T, VEC> zero = {};
    for (int r = __ldg(a.offsets + e) + __ldg(a.counts + e) + cta % a.pad_split; r < end; r += a.pad_split) {
        if (r < 0 || r >= a.R_cap) {
            if (threadIdx.x == 0)
                raise_status(a.status, kDevErrCapacity);
            return;
        }
        for (int c = threadIdx.x * VEC; c < a.H; c += blockDim.x * VEC)
            store_raw<T, VEC>(rows + (int64_t)r * a.H + c, zero);
    }
}

// One CTA per token; CTAs past the tokens write the padding rows.
template <typename T, int VEC, int KCH, bool DOT>
__global__ void __launch_bounds__(kThreads) scatter_kernel(ScatterArgs a)
{
    __shared__ float part[kThreads / 32][KCH];
    pdl_launch_dependents();
    pdl_wait();
    if ((int)blockIdx.x >= a.T) {
        zero_padding<T, VEC>(a, blockIdx.x - a.T);
        return;
    }
    const int64_t t = blockIdx.x;
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
            if (j0 + j < a.k) {
                d[j] = live_row(__ldg(a.dest + slot0 + j0 + j), a.R_cap, a.status);
                if (a.weights)
                    w[j] = __ldg(a.weights + slot0 + j0 + j);
            }
        }
        for (int c = threadIdx.x * VEC; c < a.H; c += blockDim.x * VEC) {
            const RawOf<T, VEC> raw = load_raw<T, VEC>(src + c);
            RawOf<T, VEC> in[KCH];
            if (DOT) {
#pragma unroll
                for (int j = 0; j < KCH; ++j)
                    if (d[j] >= 0)
                        in[j] = load_raw<T, VEC>(rows_in + (int64_t)d[j] * a.ld_in + c);
            }
            float f[VEC];
            unpack_raw(raw, f);
#pragma unroll
            for (int j = 0; j < KCH; ++j) {
                if (d[j] < 0)
                    continue;
                T *to = rows_out + (int64_t)d[j] * a.H + c;
                if (a.weights) {
                    float o[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        o[i] = w[j] * f[i];
                    store_raw<T, VEC>(to, pack_raw<T, VEC>(o));
                } else {
                    store_raw<T, VEC>(to, raw);
                }
                if (DOT) {
                    float g[VEC];
                    unpack_raw(in[j], g);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        dot[j] = fmaf(f[i], g[i], dot[j]);
                }
            }
        }
        if (DOT) {
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
            for (int j = 0; j < KCH; ++j) {
                float v = dot[j];
                for (int o = 16; o; o >>= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0)
                    part[warp][j] = v;
            }
            __syncthreads();
            if ((int)threadIdx.x < KCH && j0 + (int)threadIdx.x < a.k) {
                float v = 0.0f;
                for (int i = 0; i < warps; ++i)
                    v += part[i][threadIdx.x];
                a.d_weights[slot0 + j0 + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
}

bool multiple_of(const void *p, int64_t ld, int64_t H, int elem, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * elem) % bytes == 0 && (H * elem) % bytes == 0;
}

// Threads for a row of `units` loads: the fewest whole warps that take it in
// the same number of passes as kThreads would.
int block_of(int64_t units)
{
    const int64_t passes = (units + kThreads - 1) / kThreads;
    return (int)(((units + passes - 1) / passes + 31) / 32 * 32);
}

template <typename T, int VEC, int KCH> cudaError_t combine_slots(const LaunchCtx &c, const CombineArgs &a)
{
    const int64_t units = (a.H + VEC - 1) / VEC;
    const int64_t shares = (units + units_in_flight<T, VEC, KCH>() - 1) / units_in_flight<T, VEC, KCH>();
    const int block = block_of(shares);
    const dim3 grid((unsigned)a.T, (unsigned)((shares + block - 1) / block));
    return launch_pdl(combine_kernel<T, VEC, KCH>, grid, dim3(block), 0, c.stream, a);
}

template <typename T, int VEC> cudaError_t combine_vec(const LaunchCtx &c, const CombineArgs &a)
{
    return a.k <= 2 ? combine_slots<T, VEC, 2>(c, a) : combine_slots<T, VEC, 8>(c, a);
}

template <typename T, int VEC, bool DOT> cudaError_t scatter_vec(const LaunchCtx &c, ScatterArgs a)
{
    const int64_t units = (a.H + VEC - 1) / VEC;
    const int block = (int)(units >= kThreads ? kThreads : (units + 31) / 32 * 32);
    a.pad_split = a.E >= 256 ? 8 : 32;
    const dim3 grid((unsigned)(a.T + a.E * a.pad_split));
    return a.k <= 2 ? launch_pdl(scatter_kernel<T, VEC, 2, DOT>, grid, dim3(block), 0, c.stream, a)
                    : launch_pdl(scatter_kernel<T, VEC, 8, DOT>, grid, dim3(block), 0, c.stream, a);
}

template <typename T, int VEC> cudaError_t scatter_dot(const LaunchCtx &c, const ScatterArgs &a)
{
    return a.d_weights ? scatter_vec<T, VEC, true>(c, a) : scatter_vec<T, VEC, false>(c, a);
}

} // namespace

cudaError_t launch_combine(const LaunchCtx &c, const CombineArgs &a, int dtype)
{
    if (a.T == 0)
        return cudaSuccess;
    const int elem = dtype == kF32 ? 4 : 2;
    auto fits = [&](int bytes) {
        return multiple_of(a.rows, a.ld_rows, a.H, elem, bytes) && multiple_of(a.out, a.H, a.H, elem, bytes);
    };
    if (dtype == kF32)
        return fits(16) ? combine_vec<float, 4>(c, a) : combine_vec<float, 1>(c, a);
    return fits(16)  ? combine_vec<uint16_t, 8>(c, a)
           : fits(4) ? combine_vec<uint16_t, 2>(c, a)
                     : combine_vec<uint16_t, 1>(c, a);
}

cudaError_t launch_scatter(const LaunchCtx &c, const ScatterArgs &a, int dtype)
{
    const int elem = dtype == kF32 ? 4 : 2;
    auto fits = [&](int bytes) {
        return multiple_of(a.src, a.ld_src, a.H, elem, bytes) && multiple_of(a.rows_out, a.H, a.H, elem, bytes) &&
               multiple_of(a.rows_in, a.rows_in ? a.ld_in : 0, a.H, elem, bytes);
    };
    if (dtype == kF32)
        return fits(16) ? scatter_dot<float, 4>(c, a) : scatter_dot<float, 1>(c, a);
    return fits(16)  ? scatter_dot<uint16_t, 8>(c, a)
           : fits(4) ? scatter_dot<uint16_t, 2>(c, a)
                     : scatter_dot<uint16_t, 1>(c, a);
}

} // namespace epq
