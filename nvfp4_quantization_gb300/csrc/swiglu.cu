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
// Both are one pass over the data, and what bounds them is how many
// instructions a pair (g, u) costs beside its 8 bytes of traffic: arithmetic
// runs on FP32 pairs, maxima on BF16 pairs, and the sigmoid is one ex2 and one
// reciprocal.  A thread owns 8 consecutive gate columns and the 8 up columns
// beside them (16-byte BF16 loads and stores, 8-byte loads and stores of
// E4M3); the four lanes of a block of 32 share its maximum.  A CTA walks a
// contiguous range of (rows, columns) blocks, and the next block's loads are
// in flight while the current one is computed.
//
// Measured on GB300, 64 experts top-6, 16384 tokens, I = 2048: forward and
// backward with the activation again 599 us (6.1 TB/s, 6.3 with the padding
// rows); 8 experts top-2, 8192 tokens, I = 4096: 183 us (5.9 TB/s, 6.1).  Where
// I / 8 does not fill the threads side by side, those past the row's end compute
// along with the others: I = 1536 5.2 TB/s, 2560 4.9, 2112 4.3 (73 % of the issue
// slots in the forward pass, nearly half of them for nothing).  Far gates (below
// -86) cost under 1 % up to one in 10^4; one in 100 takes the forward pass of 17000
// x 4096 from 92 to 129 us and the backward pass from 91 to 194.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// log2 e as the sum of two FP32 numbers.
constexpr float kLog2eHi = 1.44269504088896340736f;
constexpr float kLog2eLo = (float)(1.44269504088896340736 - (double)kLog2eHi);

// 1 / (1 + exp(-g)) of two values up to 2^127 in size, so that g log2 e stays
// finite.  exp(-g) = 2^t (1 + r ln 2) with t = RN(-g log2 e) and r what the
// product lost: its rounding error (exact by a fused multiply-add; Dekker, "A
// floating-point technique for extending the available precision", 1971) and
// the part of log2 e below FP32.  Without r the result would lose as many bits
// as |t| has.  Below g = -87.3 the result, under 2^-126, is taken to 0: a far
// gate, which the kernels look for and hand to the functions below.
__device__ __forceinline__ float2 sigmoid2(float2 g)
{
    const float2 t = mul2(g, both(-kLog2eHi));
    float2 r = fma2(g, both(-kLog2eHi), make_float2(-t.x, -t.y));
    r = fma2(g, both(-kLog2eLo), r);
    const float2 c = fma2(r, both(0.69314718055994530942f), both(1.0f));
    const float2 e = mul2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), c);
    const float2 d = add2(e, both(1.0f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) { return make_float2(u2f(w << 16), u2f(w & 0xffff0000u)); }

__device__ __forceinline__ uint32_t to_bf16_pair(float2 v) { return cvt_bf16x2(v.x, v.y); }

// ---------------------------------------------------------------- far gates
// Below kFar the sigmoid leaves FP32's normal range, but its products with a
// large u or gradient need not: there s = exp(g) = p 2^n to well below a
// rounding, and the products are taken apart into fractions and exponents.
constexpr float kFar = -86.0f;
constexpr uint32_t kFarBits = 0x42acu;      // |kFar| as BF16

// p and n for g in [-1024, kFar]; p is about 2^-1/2 to 2^1/2.
__device__ __forceinline__ float exp_parts(float g, int &n)
{
    const float k = rintf(g * kLog2eHi);
    n = (int)k;
    return ex2_approx(fmaf(g, kLog2eLo, fmaf(g, kLog2eHi, -k)));
}

// a b c 2^n, rounded to FP32's range at the end alone; c is of ordinary size.
__device__ __forceinline__ float product(float a, float b, float c, int n)
{
    int ea, eb;
    const float m = frexpf(a, &ea) * frexpf(b, &eb) * c;
    return ldexpf(m, n + ea + eb);
}

// The products of the backward pass, in the order in which the interface
// states them; c: the sigmoid's argument.
__device__ __forceinline__ void gradients(float2 d, float2 g, float2 c, float2 u, float2 &dg, float2 &du, float2 &act)
{
    const float2 s = sigmoid2(c);
    const float2 silu = mul2(g, s);
    const float2 slope = fma2(silu, fma2(s, both(-1.0f), both(1.0f)), s);
    du = mul2(d, silu);
    dg = mul2(mul2(d, u), slope);
    act = mul2(silu, u);
}

// The same for one far gate.  Beyond -1024 every result is 0.
__device__ __forceinline__ void gradients_far(float d, float g, float u, float &dg, float &du, float &act)
{
    g = fmaxf(g, -1024.0f);
    int n;
    const float p = exp_parts(g, n);
    dg = product(d, u, (1.0f + g) * p, n);
    du = product(d, 1.0f, g * p, n);
    act = product(u, 1.0f, g * p, n);
}

// E4M3 times 2^120 reaches 2^128, which passes for FLT_MAX.
__device__ __forceinline__ float finite(float v) { return fabsf(v) > FLT_MAX ? copysignf(FLT_MAX, v) : v; }
__device__ __forceinline__ float2 finite2(float2 v) { return make_float2(finite(v.x), finite(v.y)); }

// The sigmoid of +-256 is that of +-infinity; a NaN comes back with the product.
__device__ __forceinline__ float near(float g) { return fminf(fmaxf(g, -256.0f), 256.0f); }

// max(|a|, |b|) per BF16 half; a NaN in either wins (signs are meaningless).
__device__ __forceinline__ uint32_t absmax_pair(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// max(m, |a|, |b|), NaN if one of them is.
__device__ __forceinline__ float max_abs_nan(float m, float2 v)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(v.x)), "f"(fabsf(v.y)));
    return d;
}

__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Exponent of a block whose largest |x| has BF16 bits b (finite): the smallest
// e >= -127 with max <= 448 * 2^e; 448 = 1.75 * 2^8 is exponent field 135,
// mantissa field 96, so e = field - 135, plus 1 above that mantissa.
__device__ __forceinline__ int block_exponent(uint32_t b)
{
    const int e = (int)((b + 31u) >> 7) - 135;
    return b < 0x80u ? -127 : max(-127, e);
}

// Blocks with an infinity or a NaN: those elements become E4M3's NaN, under
// the scale of the block's finite elements, so they show in the backward pass
// instead of passing for 448.  Kept out of line: it is rare.  Codes in x and y,
// scale byte in z.
__device__ __noinline__ uint3 encode8_nonfinite(uint4 r)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        b = max(b, m < 0x7f80u ? m : 0u);
    }
    b = quad_max(b);
    const int e = block_exponent(b);
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
        const float v = (h & 0x7f80u) == 0x7f80u ? u2f(0x7fffffffu) : u2f(h << 16) * exp2i(-e);
        o[i >> 2] |= (cvt_e4m3x2(v, 0.0f) & 0xffu) << (8 * (i & 3));
    }
    return make_uint3(o[0], o[1], (uint32_t)(e + 127));
}

// 8 elements of a block of 32 held by four neighbouring lanes -> E4M3 codes
// and the scale byte.  Every lane of the warp calls this.
__device__ __forceinline__ uint2 encode8(uint4 r, uint32_t &sbyte)
{
    const uint32_t m = absmax_pair(absmax_pair(r.x, r.y), absmax_pair(r.z, r.w));
    const uint32_t b = quad_max(max(m & 0x7fffu, (m >> 16) & 0x7fffu));
    if (__any_sync(0xffffffffu, b >= 0x7f80u)) {
        const uint3 v = encode8_nonfinite(r);
        sbyte = v.z;
        return make_uint2(v.x, v.y);
    }
    const int e = block_exponent(b);
    sbyte = (uint32_t)(e + 127);
    const float2 inv = both(exp2i(-e));
    const float2 v0 = mul2(bf16_pair(r.x), inv), v1 = mul2(bf16_pair(r.y), inv);
    const float2 v2 = mul2(bf16_pair(r.z), inv), v3 = mul2(bf16_pair(r.w), inv);
    return make_uint2(cvt_e4m3x2(v0.x, v0.y) | cvt_e4m3x2(v1.x, v1.y) << 16,
                      cvt_e4m3x2(v2.x, v2.y) | cvt_e4m3x2(v3.x, v3.y) << 16);
}

// Two E4M3 codes times 2^(sbyte - 127).
__device__ __forceinline__ float2 decode2(uint32_t two, float2 s)
{
    return mul2(f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(two)), s);
}

__device__ __forceinline__ float2 scale_of(uint32_t sbyte)
{
    return both(sbyte ? u2f(sbyte << 23) : u2f(0x00400000u));
}

// Whether a gate of a block with this scale can lie below kFar (448 * 2^-3 = 56
// is the largest element of the scale before), or an element of either at 2^128.
__device__ __forceinline__ bool has_far(uint32_t sbyte_g, uint32_t sbyte_u)
{
    return sbyte_g >= 125u || sbyte_u >= 247u;
}

// The results of 8 columns with far gates or elements of 2^128 among them.
// Kept out of line: it is rare.
struct Results {
    uint4 dg, du, act;
    float top;
};

__device__ __noinline__ Results backward8_far(uint4 d, uint2 cg, uint2 cu, uint32_t sbyte_g, uint32_t sbyte_u,
                                              float top)
{
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
    const uint32_t gw[4] = {cg.x & 0xffffu, cg.x >> 16, cg.y & 0xffffu, cg.y >> 16};
    const uint32_t uw[4] = {cu.x & 0xffffu, cu.x >> 16, cu.y & 0xffffu, cu.y >> 16};
    uint32_t og[4], ou[4], oa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 dv = bf16_pair(dw[i]);
        const float2 g = finite2(decode2(gw[i], scale_of(sbyte_g))), u = finite2(decode2(uw[i], scale_of(sbyte_u)));
        float2 dg, du, act;
        gradients(dv, g, make_float2(near(g.x), near(g.y)), u, dg, du, act);
        if (g.x < kFar)
            gradients_far(dv.x, g.x, u.x, dg.x, du.x, act.x);
        if (g.y < kFar)
            gradients_far(dv.y, g.y, u.y, dg.y, du.y, act.y);
        top = max_abs_nan(max_abs_nan(top, dg), du);
        og[i] = to_bf16_pair(dg);
        ou[i] = to_bf16_pair(du);
        oa[i] = to_bf16_pair(act);
    }
    return {make_uint4(og[0], og[1], og[2], og[3]), make_uint4(ou[0], ou[1], ou[2], ou[3]),
            make_uint4(oa[0], oa[1], oa[2], oa[3]), top};
}

// Activations `o` of 8 gates with those of far gates put right (beyond -256
// they are 0 as they stand, and an infinity's is NaN).  Out of line like the
// one above.
__device__ __noinline__ uint4 forward8_far(uint4 g, uint4 u, uint4 o)
{
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
    uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int up = 16 * (i & 1);
        const float gv = u2f(gw[i >> 1] >> up << 16);
        if (!(gv >= -256.0f && gv < kFar))
            continue;
        int n;
        const float p = exp_parts(gv, n);
        const uint32_t v = cvt_bf16x2(product(u2f(uw[i >> 1] >> up << 16), 1.0f, gv * p, n), 0.0f);
        ow[i >> 1] = (ow[i >> 1] & 0xffff0000u >> up) | (v & 0xffffu) << up;
    }
    return make_uint4(ow[0], ow[1], ow[2], ow[3]);
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

// A CTA's walk over blocks of (256 / cols) rows x cols units of 8 columns, in
// row order; the four lanes of a block of 32 elements stay together.
struct Walk {
    int nu, cols, tx, ty, step, blocks, r, qb;
    int64_t left;

    __device__ __forceinline__ Walk(const SwigluArgs &a, int cols_, int R)
        : nu(a.I / 8), cols(cols_), tx(threadIdx.x % cols_), ty(threadIdx.x / cols_), step(kThreads / cols_)
    {
        blocks = (nu + cols - 1) / cols;
        const int64_t total = ((int64_t)R + step - 1) / step * blocks;
        const int64_t from = total * blockIdx.x / gridDim.x;
        left = total * (blockIdx.x + 1) / gridDim.x - from;
        r = (int)(from / blocks) * step + ty;
        qb = (int)(from % blocks);
    }
    __device__ __forceinline__ int unit() const { return qb * cols + tx; }
    __device__ __forceinline__ void next()
    {
        --left;
        if (++qb == blocks) {
            qb = 0;
            r += step;
        }
    }
};

template <bool CKPT>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluArgs a, int cols)
{
    pdl_launch_dependents();
    pdl_wait();
    const int R = used_rows(a);
    uint8_t *scales = CKPT ? a.ckpt_out + (int64_t)a.R_cap * 2 * a.I : nullptr;
    Walk at(a, cols, R);
    uint4 rg = make_uint4(0, 0, 0, 0), ru = rg;
    auto fetch = [&]() {
        if (at.left > 0 && at.r < R && at.unit() < at.nu) {
            const uint16_t *x = a.x + (int64_t)at.r * a.ld + at.unit() * 8;
            rg = __ldg(reinterpret_cast<const uint4 *>(x));
            ru = __ldg(reinterpret_cast<const uint4 *>(x + a.I));
        }
    };
    fetch();
    while (at.left > 0) {
        const uint4 g = rg, u = ru;
        const int r = at.r, q = at.unit();
        const bool on = r < R && q < at.nu;
        at.next();
        fetch();
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c;                 // what near() makes of the pair
            asm("{\n\t.reg .b32 m;\n\tmin.bf16x2 m, %1, %2;\n\tmax.bf16x2 %0, m, %3;\n\t}"
                : "=r"(c) : "r"(gw[i]), "r"(0x43804380u), "r"(0xc380c380u));
            o[i] = to_bf16_pair(mul2(mul2(bf16_pair(gw[i]), sigmoid2(bf16_pair(c))), bf16_pair(uw[i])));
        }
        uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
        const uint32_t m = absmax_pair(absmax_pair(g.x, g.y), absmax_pair(g.z, g.w)) & 0x7fff7fffu;
        if (max(m & 0xffffu, m >> 16) > kFarBits)
            out = forward8_far(g, u, out);
        if (on)
            *reinterpret_cast<uint4 *>(a.act + (int64_t)r * a.I + q * 8) = out;
        if (CKPT) {
            uint32_t sg, su;
            const uint2 cg = encode8(g, sg), cu = encode8(u, su);
            if (on) {
                uint8_t *row = a.ckpt_out + (int64_t)r * 2 * a.I + q * 8;
                *reinterpret_cast<uint2 *>(row) = cg;
                *reinterpret_cast<uint2 *>(row + a.I) = cu;
                if ((q & 3) == 0) {
                    uint8_t *sr = scales + (int64_t)r * (a.I / 16) + (q >> 2);
                    sr[0] = (uint8_t)sg;
                    sr[a.I / 32] = (uint8_t)su;
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
    const uint8_t *scales = a.ckpt + (int64_t)a.R_cap * 2 * a.I;
    Walk at(a, cols, R);
    uint4 rd = make_uint4(0, 0, 0, 0);
    uint2 rg = make_uint2(0, 0), ru = rg;
    uint32_t rsg = 0, rsu = 0;
    auto fetch = [&]() {
        if (at.left > 0 && at.r < R && at.unit() < at.nu) {
            const int q = at.unit();
            const uint8_t *row = a.ckpt + (int64_t)at.r * 2 * a.I + q * 8;
            const uint8_t *sr = scales + (int64_t)at.r * (a.I / 16) + (q >> 2);
            rd = __ldg(reinterpret_cast<const uint4 *>(a.d_act + (int64_t)at.r * a.ld + q * 8));
            rg = __ldg(reinterpret_cast<const uint2 *>(row));
            ru = __ldg(reinterpret_cast<const uint2 *>(row + a.I));
            rsg = __ldg(sr);
            rsu = __ldg(sr + a.I / 32);
        }
    };
    int cur = -1;         // expert whose rows `top` covers ...
    int cur_end = 0;      // ... and where they end
    float top = 0.0f;     // its largest |dg|, |du| so far
    auto flush = [&]() {
        if (__all_sync(0xffffffffu, cur == __shfl_sync(0xffffffffu, cur, 0))) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, f2u(top));
            if (cur >= 0 && (threadIdx.x & 31) == 0 && m)
                red_max_nonneg(a.expert_amax + cur, u2f(m));
        } else if (cur >= 0 && f2u(top)) {      // short rows: the warp's rows lie on both sides of a boundary
            red_max_nonneg(a.expert_amax + cur, top);
        }
        top = 0.0f;
    };
    fetch();
    while (at.left > 0) {
        const uint4 d = rd;
        const uint2 cg = rg, cu = ru;
        const uint32_t sbyte_g = rsg, sbyte_u = rsu;
        const int r = at.r, q = at.unit();
        const bool on = r < R && q < at.nu;
        at.next();
        fetch();
        const bool turn = r < R && (cur < 0 || r >= cur_end);
        if (a.expert_amax && __any_sync(0xffffffffu, turn)) {
            flush();
            if (turn) {
                cur = a.offsets ? expert_of_dest(a.offsets, a.E, r) : 0;
                cur_end = a.offsets ? __ldg(a.offsets + cur + 1) : R;
            }
        }
        if (on) {
            Results o;
            if (has_far(sbyte_g, sbyte_u)) {
                o = backward8_far(d, cg, cu, sbyte_g, sbyte_u, top);
                top = o.top;
            } else {
                const float2 sg = scale_of(sbyte_g), su = scale_of(sbyte_u);
                const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
                const uint32_t gw[4] = {cg.x & 0xffffu, cg.x >> 16, cg.y & 0xffffu, cg.y >> 16};
                const uint32_t uw[4] = {cu.x & 0xffffu, cu.x >> 16, cu.y & 0xffffu, cu.y >> 16};
                uint32_t og[4], ou[4], oa[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 g = decode2(gw[i], sg);
                    float2 dg, du, act;
                    gradients(bf16_pair(dw[i]), g, g, decode2(uw[i], su), dg, du, act);
                    top = max_abs_nan(max_abs_nan(top, dg), du);
                    og[i] = to_bf16_pair(dg);
                    ou[i] = to_bf16_pair(du);
                    oa[i] = to_bf16_pair(act);
                }
                o.dg = make_uint4(og[0], og[1], og[2], og[3]);
                o.du = make_uint4(ou[0], ou[1], ou[2], ou[3]);
                o.act = make_uint4(oa[0], oa[1], oa[2], oa[3]);
            }
            uint16_t *dx = a.d_x + (int64_t)r * 2 * a.I + q * 8;
            *reinterpret_cast<uint4 *>(dx) = o.dg;
            *reinterpret_cast<uint4 *>(dx + a.I) = o.du;
            if (ACT)
                *reinterpret_cast<uint4 *>(a.act + (int64_t)r * a.I + q * 8) = o.act;
        }
    }
    if (a.expert_amax)
        flush();
}

// Threads side by side along a row: the least power of two that covers it, 4
// (one block of 32) to 256.  (With no fewer than a warp, 6022 x 6 rows of I = 96
// took 29 us.)
int column_threads(int I)
{
    int n = 4;
    while (n < I / 8 && n < kThreads)
        n *= 2;
    return n;
}

// One wave of resident CTAs (or fewer, if there is less work).
template <void (*kernel)(SwigluArgs, int)> cudaError_t launch_walk(const LaunchCtx &c, const SwigluArgs &a)
{
    static std::atomic<int> resident{0};    // CTAs per SM, asked for once
    const int cols = column_threads(a.I), step = kThreads / cols;
    const int64_t blocks = ((int64_t)a.R_cap + step - 1) / step * ((a.I / 8 + cols - 1) / cols);
    int per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
        if (e != cudaSuccess)
            return e;
        per_sm = per_sm < 1 ? 1 : per_sm;
        resident.store(per_sm, std::memory_order_relaxed);
    }
    const int64_t wave = (int64_t)c.num_sms * per_sm;
    return launch_pdl(kernel, dim3((unsigned)(blocks < wave ? blocks : wave)), dim3(kThreads), 0, c.stream, a, cols);
}

} // namespace

cudaError_t launch_swiglu(const LaunchCtx &c, const SwigluArgs &a)
{
    if (a.R_cap == 0)
        return cudaSuccess;
    return a.ckpt_out ? launch_walk<swiglu_kernel<true>>(c, a) : launch_walk<swiglu_kernel<false>>(c, a);
}

cudaError_t launch_swiglu_backward(const LaunchCtx &c, const SwigluArgs &a)
{
    if (a.R_cap == 0)
        return cudaSuccess;
    return a.act ? launch_walk<swiglu_backward_kernel<true>>(c, a) : launch_walk<swiglu_backward_kernel<false>>(c, a);
}

} // namespace epq
