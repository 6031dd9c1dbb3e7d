// BF16 matrix products grouped by expert (the kernel is in grouped.cuh).
#include "grouped.cuh"

namespace epq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A matrix [outer][inner] of BF16, copied in boxes of 64 x `rows`.
bool bf16_map(CUtensorMap *m, const void *p, int64_t inner, int64_t outer, int64_t pitch, int64_t experts, int rows)
{
    return make_map_3d(m, MapType::Bf16, p, {(uint64_t)inner, (uint64_t)outer, (uint64_t)experts},
                       {(uint64_t)pitch * 2, (uint64_t)(pitch * outer) * 2}, {64, (uint32_t)rows, 1}, 128);
}

template <bool kAmn, int kCtas> cudaError_t gemm(const LaunchCtx &c, const GroupedGemmArgs &a)
{
    using C = GroupedCfg<false, false, kAmn, kCtas, false>;
    GroupedParams p = {};
    // without rows there is nothing to copy: the kernel only looks at the offsets
    const bool ok = a.R_cap == 0 ||
                    ((kAmn ? bf16_map(&p.map[kMapA], a.w, a.N, a.K, a.N, a.E, 64)
                           : bf16_map(&p.map[kMapA], a.w, a.K, a.N, a.K, a.E, 128)) &&
                     bf16_map(&p.map[kMapB], a.x, a.K, a.R_cap, a.ld_x, 1, 64) &&
                     make_map_3d(&p.out, MapType::Bf16, a.out, {(uint64_t)a.N, (uint64_t)a.R_cap, 1},
                                 {(uint64_t)a.N * 2, (uint64_t)a.N * 2 * a.R_cap}, {32, 32, 1}, 64));
    if (!ok)
        return cudaErrorInvalidValue;
    p.offsets = a.offsets;
    p.status = a.status;
    p.R_cap = a.R_cap;
    p.E = a.E;
    p.M = p.N = a.N;
    p.K = a.K;
    return launch_grouped<C>(c, p, ceil_div(a.N, C::kSpan) * (ceil_div(a.R_cap, C::kTileN) + a.E));
}

template <bool kF32, int kCtas> cudaError_t wgrad(const LaunchCtx &c, const GroupedWgradArgs &a)
{
    using C = GroupedCfg<false, true, true, kCtas, kF32>;
    GroupedParams p = {};
    // without rows there is nothing to copy from
    if (a.R_cap > 0 && (!bf16_map(&p.map[kMapA], a.dy, a.N, a.R_cap, a.ld_dy, 1, 64) ||
                        !bf16_map(&p.map[kMapB], a.x, a.K, a.R_cap, a.ld_x, 1, 64)))
        return cudaErrorInvalidValue;
    const uint64_t size = kF32 ? 4 : 2;
    if (!make_map_3d(&p.out, kF32 ? MapType::F32 : MapType::Bf16, a.d_w, {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E},
                     {a.K * size, a.K * size * a.N}, {(uint32_t)C::kChunk, 32, 1}, 128))
        return cudaErrorInvalidValue;
    p.offsets = a.offsets;
    p.counts = a.counts;
    p.status = a.status;
    p.R_cap = a.R_cap;
    p.E = a.E;
    p.M = a.N;
    p.N = a.K;
    p.add = a.add;
    return launch_grouped<C>(c, p, a.E * ceil_div(a.N, C::kSpan) * ceil_div(a.K, C::kTileN));
}

} // namespace

cudaError_t launch_grouped_gemm(const LaunchCtx &c, const GroupedGemmArgs &a)
{
    if (a.R_cap == 0 && !a.offsets)
        return cudaSuccess;
    using One = GroupedCfg<false, false, false, 1, false>;
    if (single_ctas<One>(c, a.N, ceil_div(a.R_cap, One::kTileN)))
        return a.transposed ? gemm<true, 1>(c, a) : gemm<false, 1>(c, a);
    return a.transposed ? gemm<true, 2>(c, a) : gemm<false, 2>(c, a);
}

cudaError_t launch_grouped_wgrad(const LaunchCtx &c, const GroupedWgradArgs &a)
{
    using One = GroupedCfg<false, true, true, 1, false>;
    if (single_ctas<One>(c, a.N, a.E * ceil_div(a.K, One::kTileN)))
        return a.f32 ? wgrad<true, 1>(c, a) : wgrad<false, 1>(c, a);
    return a.f32 ? wgrad<true, 2>(c, a) : wgrad<false, 2>(c, a);
}

} // namespace epq
