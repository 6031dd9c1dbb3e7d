// Gated activation between the two expert products, with its input kept for
// the backward pass as MXFP8 (E4M3 elements, one E8M0 scale per 32), and the
// backward pass from that checkpoint.
//
//   forward   act = g s(g) u,  s(g) = 1 / (1 + exp(-g)),  x = [g | u]
//             ckpt = MXFP8(x): per 32 elements e = smallest integer with
//             max|x| <= 448 * 2^e, scale byte e + 127, E4M3_RNE(x / 2^e)
//   backward  with g, u read from ckpt:
//             dg = da u s (1 + g (1 - s)),  du = da g s
//             amax_e = max over the rows of expert e of |dg|, |du| (FP32,
//             before the rounding to BF16)
//
// Both are one pass over the data.  A thread owns 8 consecutive gate columns
// and the 8 up columns beside them (16-byte BF16 loads and stores, 8-byte
// loads and stores of E4M3); the four lanes of a block of 32 share its
// maximum.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 256;
constexpr int kChunkRows = 16;   // rows that a CTA takes at a time

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + expf(-g)); }

__device__ __forceinline__ void unpack8(uint4 r, float (&f)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = u2f(w[i] << 16);
        f[2 * i + 1] = u2f(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}

// Largest |x| (BF16 bits) of 8 elements; `finite`: infinities and NaN left out.
template <bool FINITE>
__device__ __forceinline__ uint32_t absmax8(uint4 r)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (!FINITE || lo < 0x7f80u)
            m = max(m, lo);
        if (!FINITE || hi < 0x7f80u)
            m = max(m, hi);
    }
    return m;
}

__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// 8 elements of a block of 32 held by four neighbouring lanes -> E4M3 codes
// and the scale byte.  Every lane of the warp calls this.  An infinity or NaN
// is stored as E4M3's NaN, under the scale of the block's finite elements, so
// it shows in the backward pass instead of passing for 448.
__device__ __forceinline__ uint2 encode8(uint4 r, const float (&f)[8], uint32_t &sbyte)
{
    uint32_t b = quad_max(absmax8<false>(r));
    const bool bad = b >= 0x7f80u;
    if (__any_sync(0xffffffffu, bad)) {
        const uint32_t fin = quad_max(absmax8<true>(r));
        b = bad ? fin : b;
    }
    // 448 = 1.75 * 2^8: BF16 exponent field 135, mantissa field 96
    const int ef = (int)(b >> 7), mt = (int)(b & 0x7fu);
    const int e = max(-127, ef == 0 ? -127 : ef - 135 + (mt > 96 ? 1 : 0));
    sbyte = (uint32_t)(e + 127);
    const float inv = exp2i(-e);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = f[i] * inv;
        if (bad && (f2u(f[i]) & 0x7f800000u) == 0x7f800000u)
            v[i] = u2f(0x7fffffffu);
    }
    return make_uint2(cvt_e4m3x2(v[0], v[1]) | cvt_e4m3x2(v[2], v[3]) << 16,
                      cvt_e4m3x2(v[4], v[5]) | cvt_e4m3x2(v[6], v[7]) << 16);
}

__device__ __forceinline__ void decode8(uint2 c, uint32_t sbyte, float (&f)[8])
{
    const float s = sbyte ? u2f(sbyte << 23) : u2f(0x00400000u);   // 2^(sbyte - 127)
    const uint32_t two[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(two[i]));
        f[2 * i] = v.x * s;
        f[2 * i + 1] = v.y * s;
    }
}

__device__ __forceinline__ int used_rows(const SwigluArgs &a)
{
    if (!a.offsets)
        return a.R_cap;
    const int R = __ldg(a.offsets + a.E);
    if (R > a.R_cap && blockIdx.x == 0 && threadIdx.x == 0)
        raise_status(a.status, kDevErrCapacity);
    return min(R, a.R_cap);
}

// Threads are cols x (256 / cols): a warp stays within one row.
template <bool CKPT>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluArgs a, int cols)
{
    pdl_launch_dependents();
    pdl_wait();
    const int R = used_rows(a);
    const int nu = a.I / 8;
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, step = kThreads / cols;
    uint8_t *scales = CKPT ? a.ckpt_out + (int64_t)a.R_cap * 2 * a.I : nullptr;
    for (int r0 = blockIdx.x * kChunkRows; r0 < R; r0 += gridDim.x * kChunkRows) {
        const int r1 = min(r0 + kChunkRows, R);
        for (int r = r0 + ty; r < r1; r += step) {
            const uint16_t *x = a.x + (int64_t)r * a.ld;
            for (int q0 = 0; q0 < nu; q0 += cols) {
                const int q = q0 + tx;
                const bool on = q < nu;
                uint4 rg = make_uint4(0, 0, 0, 0), ru = rg;
                if (on) {
                    rg = __ldg(reinterpret_cast<const uint4 *>(x + q * 8));
                    ru = __ldg(reinterpret_cast<const uint4 *>(x + a.I + q * 8));
                }
                float g[8], u[8], o[8];
                unpack8(rg, g);
                unpack8(ru, u);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = g[i] * sigmoid(g[i]) * u[i];
                if (on)
                    *reinterpret_cast<uint4 *>(a.act + (int64_t)r * a.I + q * 8) = pack8(o);
                if (CKPT) {
                    uint32_t sg, su;
                    const uint2 cg = encode8(rg, g, sg), cu = encode8(ru, u, su);
                    if (on) {
                        uint8_t *row = a.ckpt_out + (int64_t)r * 2 * a.I;
                        *reinterpret_cast<uint2 *>(row + q * 8) = cg;
                        *reinterpret_cast<uint2 *>(row + a.I + q * 8) = cu;
                        if ((q & 3) == 0) {
                            uint8_t *sr = scales + (int64_t)r * (a.I / 16);
                            sr[q >> 2] = (uint8_t)sg;
                            sr[a.I / 32 + (q >> 2)] = (uint8_t)su;
                        }
                    }
                }
            }
        }
    }
}

template <bool ACT>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(SwigluArgs a, int cols)
{
    pdl_launch_dependents();
    pdl_wait();
    const int R = used_rows(a);
    const int nu = a.I / 8;
    const int tx = threadIdx.x % cols, ty = threadIdx.x / cols, step = kThreads / cols;
    const uint8_t *scales = a.ckpt + (int64_t)a.R_cap * 2 * a.I;
    int cur = -1;         // expert whose rows `top` covers (the same in all lanes of a warp)
    uint32_t top = 0;     // its largest |dg|, |du| so far, as bits (NaN is the largest)
    auto flush = [&]() {
        const uint32_t m = __reduce_max_sync(0xffffffffu, top);
        if (cur >= 0 && (threadIdx.x & 31) == 0 && m)
            red_max_nonneg(a.expert_amax + cur, u2f(m));
        top = 0;
    };
    for (int r0 = blockIdx.x * kChunkRows; r0 < R; r0 += gridDim.x * kChunkRows) {
        const int r1 = min(r0 + kChunkRows, R);
        for (int r = r0 + ty; r < r1; r += step) {
            if (a.expert_amax) {
                const int e = a.offsets ? expert_of_dest(a.offsets, a.E, r) : 0;
                if (e != cur) {
                    flush();
                    cur = e;
                }
            }
            const uint8_t *row = a.ckpt + (int64_t)r * 2 * a.I;
            const uint8_t *sr = scales + (int64_t)r * (a.I / 16);
            for (int q = tx; q < nu; q += cols) {
                const uint4 rd = __ldg(reinterpret_cast<const uint4 *>(a.d_act + (int64_t)r * a.ld + q * 8));
                const uint2 cg = __ldg(reinterpret_cast<const uint2 *>(row + q * 8));
                const uint2 cu = __ldg(reinterpret_cast<const uint2 *>(row + a.I + q * 8));
                const uint32_t sg = __ldg(sr + (q >> 2)), su = __ldg(sr + a.I / 32 + (q >> 2));
                float d[8], g[8], u[8], dg[8], du[8], o[8];
                unpack8(rd, d);
                decode8(cg, sg, g);
                decode8(cu, su, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = sigmoid(g[i]);
                    const float silu = g[i] * s;
                    du[i] = d[i] * silu;
                    dg[i] = d[i] * u[i] * fmaf(silu, 1.0f - s, s);
                    o[i] = silu * u[i];
                    top = max(top, max(f2u(dg[i]) & 0x7fffffffu, f2u(du[i]) & 0x7fffffffu));
                }
                uint16_t *dx = a.d_x + (int64_t)r * 2 * a.I;
                *reinterpret_cast<uint4 *>(dx + q * 8) = pack8(dg);
                *reinterpret_cast<uint4 *>(dx + a.I + q * 8) = pack8(du);
                if (ACT)
                    *reinterpret_cast<uint4 *>(a.act + (int64_t)r * a.I + q * 8) = pack8(o);
            }
        }
    }
    if (a.expert_amax)
        flush();
}

int column_threads(int I)
{
    const int nu = I / 8;
    return nu <= 32 ? 32 : nu <= 64 ? 64 : nu <= 128 ? 128 : 256;
}

int grid_of(const LaunchCtx &c, int R_cap)
{
    const int64_t chunks = ((int64_t)R_cap + kChunkRows - 1) / kChunkRows;
    const int64_t most = (int64_t)c.num_sms * 8;
    return (int)(chunks < most ? chunks : most);
}

} // namespace

cudaError_t launch_swiglu(const LaunchCtx &c, const SwigluArgs &a)
{
    if (a.R_cap == 0)
        return cudaSuccess;
    const dim3 grid(grid_of(c, a.R_cap));
    const int cols = column_threads(a.I);
    return a.ckpt_out ? launch_pdl(swiglu_kernel<true>, grid, dim3(kThreads), 0, c.stream, a, cols)
                      : launch_pdl(swiglu_kernel<false>, grid, dim3(kThreads), 0, c.stream, a, cols);
}

cudaError_t launch_swiglu_backward(const LaunchCtx &c, const SwigluArgs &a)
{
    if (a.R_cap == 0)
        return cudaSuccess;
    const dim3 grid(grid_of(c, a.R_cap));
    const int cols = column_threads(a.I);
    return a.act ? launch_pdl(swiglu_backward_kernel<true>, grid, dim3(kThreads), 0, c.stream, a, cols)
                 : launch_pdl(swiglu_backward_kernel<false>, grid, dim3(kThreads), 0, c.stream, a, cols);
}

} // namespace epq
