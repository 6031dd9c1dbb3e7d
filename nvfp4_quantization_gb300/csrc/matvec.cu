// Products of a few tokens with NVFP4 expert weights (decode batches).
//
//   y[s] = W_e(s) x(s),  W[n][i] = code(n, i) * s_b(n, i / 16) * S(n)
//
// The weights are packed NVFP4 rows as the pack writes them (E2M1 codes, an
// E4M3 scale per 16 elements, an FP32 row scale in the trailer): one row per
// output feature.  Products and sums are FP32; the row scale is applied to the
// finished sum, which is rounded once.
#include "epq_device.cuh"
#include "epq_internal.h"

namespace epq {

namespace {

constexpr int kThreads = 256;

// One warp per (slot, output feature).
__global__ void __launch_bounds__(kThreads) matvec_kernel(MatvecArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int blocks = (a.N + kThreads / 32 - 1) / (kThreads / 32);
    const int n = blockIdx.x % blocks * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t s = blockIdx.x / blocks;
    if (n >= a.N)
        return;
    int e = a.topk ? __ldg(a.topk + s) : 0;
    if (e < -1 || e >= a.E) {
        if (lane == 0)
            raise_status(a.status, kDevErrBadExpert);
        e = -1;
    }
    float acc = 0.0f, row_scale = 0.0f;
    if (e >= 0) {
        const uint8_t *row = a.w + ((int64_t)e * a.N + n) * a.S;
        const uint16_t *x = a.x + (a.per_slot ? s : s / a.k) * a.ld_x;
        row_scale = __ldg(reinterpret_cast<const float *>(row + a.S - 16));
        for (int q = lane; q < a.K / 8; q += 32) {
            const uint32_t cw = __ldg(reinterpret_cast<const uint32_t *>(row) + q);
            const float sc = e4m3_to_f32(__ldg(row + a.K / 2 + (q >> 1)));
            float part = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float2 v = f16x2_to_f32x2(cvt_f16x2_from_e2m1x2((cw >> (8 * b)) & 0xffu));
                part = fmaf(v.x, u2f((uint32_t)__ldg(x + q * 8 + 2 * b) << 16), part);
                part = fmaf(v.y, u2f((uint32_t)__ldg(x + q * 8 + 2 * b + 1) << 16), part);
            }
            acc = fmaf(part, sc, acc);
        }
    }
    for (int o = 16; o; o >>= 1)
        acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0)
        a.y[s * a.N + n] = (uint16_t)cvt_bf16x2(e >= 0 ? acc * row_scale : 0.0f, 0.0f);
}

} // namespace

cudaError_t launch_matvec(const LaunchCtx &c, const MatvecArgs &a)
{
    const int64_t slots = (int64_t)a.T * a.k;
    if (slots == 0)
        return cudaSuccess;
    const int64_t grid = slots * ((a.N + kThreads / 32 - 1) / (kThreads / 32));
    if (grid > (int64_t)INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_pdl(matvec_kernel, dim3((unsigned)grid), dim3(kThreads), 0, c.stream, a);
}

} // namespace epq
