// Device-side building blocks shared by the epq kernels: format conversions
// (inline PTX cvt forms of sm_100-family GPUs), packed FP32 pair arithmetic,
// mbarrier / TMA / programmatic-dependent-launch wrappers, and the
// Philox4x32-10 generator used for stochastic rounding.
#pragma once

#include <cuda.h>
#include <float.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace epq {

constexpr uint32_t kDevErrBadExpert = 1u;
constexpr uint32_t kDevErrDupExpert = 2u;
constexpr uint32_t kDevErrTimeout = 4u;
constexpr uint32_t kDevErrCapacity = 8u;

// ---------------------------------------------------------------- bit casts
__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

// 2^k as FP32 for k in [-126, 127].
__device__ __forceinline__ float exp2i(int k) { return u2f((uint32_t)(k + 127) << 23); }

// ---------------------------------------------------------------- E2M1 / E4M3
// Two FP32 values -> one byte holding two E2M1 codes, round to nearest even,
// saturating at +-6.  `lo` lands in the low nibble (the even element).
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi)
{
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u16.u8 %0, t;\n\t}"
        : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight FP32 values -> one word of eight E2M1 codes (round to nearest even,
// saturating); a[0] in the lowest nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(float a0, float a1, float a2, float a3, float a4, float a5,
                                               float a6, float a7)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a0), "f"(a1), "f"(a2), "f"(a3), "f"(a4), "f"(a5), "f"(a6), "f"(a7));
    return r;
}

// One byte of two E2M1 codes -> f16x2 (exact); the low nibble goes to the low
// half.
__device__ __forceinline__ uint32_t cvt_f16x2_from_e2m1x2(uint32_t byte)
{
    uint32_t r;
    uint16_t b = (uint16_t)byte;
    asm("{\n\t.reg .b8 t;\n\t"
        "mov.b16 {t, _}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(r) : "h"(b));
    return r;
}

// Two FP32 values -> two E4M3 codes (round to nearest even, saturating at
// +-448); `lo` in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E4M3 codes (low byte first) -> f16x2, exact.
__device__ __forceinline__ uint32_t cvt_f16x2_from_e4m3x2(uint32_t two)
{
    uint32_t r;
    uint16_t b = (uint16_t)two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h)
{
    __half2 v = *reinterpret_cast<__half2 *>(&h);
    return __half22float2(v);
}

// E4M3 code -> FP32 (exact).
__device__ __forceinline__ float e4m3_to_f32(uint32_t code)
{
    return f16x2_to_f32x2(cvt_f16x2_from_e4m3x2(code & 0xffu)).x;
}

// Two FP32 -> packed f16x2, round to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two FP32 -> packed bf16x2, round to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four bytes (each in the low byte of its word) -> one word, b0 lowest.
__device__ __forceinline__ uint32_t pack4(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3)
{
    return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
}

// ---------------------------------------------------------------- FP32 pairs
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
// a - b, one rounding: fma(b, -1, a).
__device__ __forceinline__ float2 sub2(float2 a, float2 b)
{
    return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// ---------------------------------------------------------------- PDL
// Programmatic dependent launch: wait until the preceding kernel in the
// stream has completed and its writes are visible; allow the next kernel to be
// scheduled.  Both are no-ops when the launch carries no programmatic edge.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Loads of what an earlier kernel may have written just before.  A kernel that is
// launched early is running while that one still writes, so its inputs do not stay
// the same for its whole lifetime, which loads through the read-only path (__ldg,
// ld.global.nc, and plain loads of const __restrict__ parameters) rely on, and the
// compiler could move such a load ahead of the wait.  These stay behind it: volatile
// statements keep their order among themselves.  They claim no other memory, since no
// kernel writes its own inputs.
__device__ __forceinline__ uint32_t ld_word(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ int ld_word(const int32_t *p)
{
    return (int)ld_word(reinterpret_cast<const uint32_t *>(p));
}

__device__ __forceinline__ float ld_word(const float *p)
{
    return u2f(ld_word(reinterpret_cast<const uint32_t *>(p)));
}

__device__ __forceinline__ uint32_t ld_half_word(const uint16_t *p)
{
    uint16_t v;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_byte(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 ld_8bytes(const void *p)
{
    uint2 v;
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 ld_16bytes(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ---------------------------------------------------------------- gpu-scope loads
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// ---------------------------------------------------------------- status
__device__ __forceinline__ void raise_status(uint32_t *st, uint32_t bits)
{
    if (st)
        atomicOr(st, bits);
}

// ---------------------------------------------------------------- per-expert amax
// Max-reduction of a non-negative FP32 value into *p, done on the bit
// patterns: for non-negative floats the unsigned order of the bits is the
// numeric order.  Fire-and-forget (no value comes back).
__device__ __forceinline__ void red_max_nonneg(float *p, float v)
{
    asm volatile("red.relaxed.gpu.global.max.u32 [%0], %1;" ::"l"(p), "r"(__float_as_uint(v)) : "memory");
}

// The expert whose slot holds row d: the last e with offsets[e] <= d (empty
// slots before it share its offset and are skipped by taking the last).
__device__ __forceinline__ int expert_of_dest(const int32_t *offsets, int E, int d)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ld_word(offsets + mid) <= d)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Columnwise metadata of an expert from its rowwise amax A_e (reading R11):
// amax_col = fl32(4 A_e), S_enc = min(fl32(2688 / amax_col), FLT_MAX), and
// S_enc = 1 for an expert whose amax is 0 (no rows, or all-zero rows).
__device__ __forceinline__ float colwise_encode_scale(float amax_row, float &amax_col)
{
    amax_col = 4.0f * amax_row;
    return amax_col > 0.0f ? fminf(__fdiv_rn(2688.0f, amax_col), FLT_MAX) : 1.0f;
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}"
                 ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\t"
                 "mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                 ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Raise the transaction count of the current phase without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Bounded wait on a phase of an mbarrier.  Gives up after roughly a second
// (the try_wait instruction itself suspends for a while on each attempt) and
// returns false; the caller records EP_DEV_ERR_TIMEOUT and unwinds.
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (i > 64)
            __nanosleep(256);
    }
    return false;
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory");
}

// 2-D tiled load global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_2d(void *smem_dst, const CUtensorMap *m, int x, int y,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(smem_dst)), "l"((uint64_t)m), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}

// 1-D bulk copy global -> shared (src, dst 16-byte aligned, bytes % 16 == 0),
// completion counted on `bar`.
__device__ __forceinline__ void bulk_load(void *smem_dst, const void *gsrc, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(smem_dst)), "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Bring [gsrc, gsrc + bytes) into L2 (16-byte aligned, bytes % 16 == 0).  L2 is
// the point of coherence, so a prefetch issued before the data's producer has
// finished cannot return stale data to later loads.
__device__ __forceinline__ void bulk_prefetch_l2(const void *gsrc, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(gsrc), "r"(bytes) : "memory");
}

// Order this thread's earlier generic-proxy shared-memory accesses before
// later async-proxy (bulk copy) accesses.
__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 2-D tiled store shared -> global (elements outside the tensor are skipped).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, int x, int y, const void *smem_src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"((uint64_t)m), "r"(x), "r"(y), "r"(smem_u32(smem_src)) : "memory");
}

__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// Wait until every committed bulk store has finished reading shared memory.
__device__ __forceinline__ void tma_store_wait_read0()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Wait until every committed bulk store has completed.
__device__ __forceinline__ void tma_store_wait0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Named barrier over a subset of the CTA's warps.
__device__ __forceinline__ void named_bar_sync(uint32_t id, uint32_t nthreads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// Named barrier that also ORs a predicate over the participating threads;
// every participant gets the same result.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t nthreads, bool pred)
{
    uint32_t out;
    asm volatile("{\n\t.reg .pred pi, po;\n\t"
                 "setp.ne.u32 pi, %1, 0;\n\t"
                 "bar.red.or.pred po, %2, %3, pi;\n\t"
                 "selp.u32 %0, 1, 0, po;\n\t}"
                 : "=r"(out) : "r"((uint32_t)pred), "r"(id), "r"(nthreads) : "memory");
    return out != 0;
}

// RN(a * b + c) with a, b the halves H_A, H_B (0 = low, 1 = high) of two
// packed f16 pairs and c, the result FP32: one mixed-precision FMA (the
// product of two f16 values is exact in FP32, so this rounds once).
template <int HA, int HB>
__device__ __forceinline__ float fma_f16h(uint32_t a, uint32_t b, float c)
{
    float d;
    if (HA == 0 && HB == 0)
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.f16 %0, a0, b0, %3;\n\t}" : "=f"(d) : "r"(a), "r"(b), "f"(c));
    else if (HA == 1 && HB == 0)
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.f16 %0, a1, b0, %3;\n\t}" : "=f"(d) : "r"(a), "r"(b), "f"(c));
    else if (HA == 0 && HB == 1)
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.f16 %0, a0, b1, %3;\n\t}" : "=f"(d) : "r"(a), "r"(b), "f"(c));
    else
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.f16 %0, a1, b1, %3;\n\t}" : "=f"(d) : "r"(a), "r"(b), "f"(c));
    return d;
}

// Thread-block cluster: barrier over all threads of all CTAs of the cluster,
// with release / acquire ordering of the shared-memory writes before it.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A 32-bit word at the same shared-memory offset as `p`, in the CTA of the
// cluster with rank `rank`.
__device__ __forceinline__ uint32_t ld_dsmem_u32(const void *p, uint32_t rank)
{
    uint32_t remote, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}

// Packed f16 product, round to nearest even.
__device__ __forceinline__ uint32_t hmul2_rn(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// max(m, |a|, |b|) in one three-input maximum (finite inputs).
__device__ __forceinline__ float max3_abs(float m, float a, float b)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}

// ---------------------------------------------------------------- Philox
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC'11): ten rounds, each two 32x32->64-bit products of words 0
// and 2 with the round multipliers, the high halves XORed with the other two
// words and the round key; the key is advanced by the Weyl constants between
// rounds.
struct Philox4 {
    uint32_t x, y, z, w;
};

// The ten round keys of one seed, (k0 + r W0, k1 + r W1) for r = 0..9 with
// (k0, k1) the low and high words of the seed and (W0, W1) the Weyl
// constants, computed once on the host and passed as a kernel parameter so
// the rounds read them straight from the constant bank.
struct PhiloxKey {
    uint32_t k[10][2];
};

__host__ __device__ inline PhiloxKey philox_key(uint64_t seed)
{
    PhiloxKey K;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int r = 0; r < 10; ++r) {
        K.k[r][0] = k0;
        K.k[r][1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return K;
}

__device__ __forceinline__ Philox4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                                 const PhiloxKey &K)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0;
        const uint64_t p1 = (uint64_t)0xCD9E8D57u * c2;
        const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c1 ^ K.k[r][0];
        const uint32_t n2 = (uint32_t)(p0 >> 32) ^ c3 ^ K.k[r][1];
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        c0 = n0;
        c2 = n2;
    }
    return Philox4{c0, c1, c2, c3};
}

// The Philox output for the aligned group of 16 elements starting at element
// index idx0 (idx0 % 16 == 0) of stream `stream`: word q (x, y, z, w for
// q = 0..3) carries the random numbers of elements idx0 + 4q .. idx0 + 4q + 3
// (see cvt_e2m1x8_sr).
__device__ __forceinline__ Philox4 sr_bytes16(const PhiloxKey &K, uint32_t stream, uint64_t idx0)
{
    const uint64_t n = idx0 >> 4;
    return philox4x32_10((uint32_t)n, (uint32_t)(n >> 32), stream, 0u, K);
}

// sr_bytes16 for an element index below 2^36 (the grouped operands: offsets,
// columns and rows address at most R_cap * H < 2^36 elements), whose counter's
// second word is 0.  With that word a literal, the product of round 2 that
// involves only the key is loop-invariant: 18 wide products per call, not 19.
__device__ __forceinline__ Philox4 sr_bytes16_36(const PhiloxKey &K, uint32_t stream, uint64_t idx0)
{
    return philox4x32_10((uint32_t)(idx0 >> 4), 0u, stream, 0u, K);
}

// Eight FP32 values -> one word of eight E2M1 codes by stochastic rounding,
// a[0] in the lowest nibble; a[0..3] take the random word r_lo, a[4..7] r_hi.
// Within a word with bytes b0..b3 (b0 least significant), A = b2:b0 and
// B = b3:b1 (16-bit numbers, high byte first): the four values take A, A
// bit-reversed, B, B bit-reversed; a value rounds up iff R + 65536 f >= 65536
// with f its position between the neighbouring grid values, sign kept,
// saturating at 6.
//
// Hardware: cvt.rs.satfinite.e2m1x4.f32 d, {a, b, c, e}, rbits puts e in bits
// 3:0 of d, c in 7:4, b in 11:8, a in 15:12, and rounds e with the 16-bit
// number rbits[23:16]:rbits[7:0], b with rbits[31:24]:rbits[15:8], c and a
// with the bit reverses of those two; a value rounds up iff its fraction plus
// R 2^-16 reaches 1 (measured on GB300 over 8.4 M values with random words
// and boundary fractions: 0 mismatches).  So the rule above is exactly one
// conversion per four values with the Philox word as rbits.
__device__ __forceinline__ uint32_t cvt_e2m1x8_sr(float a0, float a1, float a2, float a3, float a4, float a5,
                                                  float a6, float a7, uint32_t r_lo, uint32_t r_hi)
{
    uint32_t out;
    asm("{\n\t.reg .b16 h0, h1;\n\t"
        "cvt.rs.satfinite.e2m1x4.f32 h0, {%4, %3, %2, %1}, %9;\n\t"
        "cvt.rs.satfinite.e2m1x4.f32 h1, {%8, %7, %6, %5}, %10;\n\t"
        "mov.b32 %0, {h0, h1};\n\t}"
        : "=r"(out)
        : "f"(a0), "f"(a1), "f"(a2), "f"(a3), "f"(a4), "f"(a5), "f"(a6), "f"(a7), "r"(r_lo), "r"(r_hi));
    return out;
}

} // namespace epq
