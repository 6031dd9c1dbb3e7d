// NVFP4 matrix products grouped by expert (the kernel is in grouped.cuh), and
// what prepares their operands: the tiled scales of packed rows.
#include <algorithm>

#include "grouped.cuh"

namespace epq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- operand
// Block scales of packed rows [row][K / 16] into tiles of 128 rows x 4 (512
// bytes; row m, column b at (m % 32) * 16 + (m % 128 / 32) * 4 + b % 4), and the
// row scales out of the trailers.  A CTA takes 128 rows x 32 tiles: the scales
// come in 16-byte pieces, a row's next to each other, and go out as 16-byte
// pieces of a tile (four rows), a tile's next to each other.
constexpr int kOpThreads = 256;
constexpr int kOpTiles = 32;                      // tiles of a CTA: 128 bytes of every row
constexpr int kOpPitch = kOpTiles * 4 + 4;        // bytes of a row in shared memory: no bank twice

__global__ void __launch_bounds__(kOpThreads) operand_kernel(const __grid_constant__ OperandArgs a, int mt, int kt)
{
    __shared__ __align__(16) uint8_t s[128 * kOpPitch];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    int64_t limit = a.per_group;                  // rows of a group
    if (a.offsets) {
        const int R = ld_word(a.offsets + a.E);
        if (R > limit && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
            raise_status(a.status, kDevErrCapacity);
        limit = R < limit ? R : limit;
    }
    const int64_t g = blockIdx.x / mt, m0 = (int64_t)(blockIdx.x % mt) * 128;
    if (a.offsets && m0 >= limit)
        return;
    const int t0 = blockIdx.y * kOpTiles, nt = min(kOpTiles, kt - t0);
    const int Kb = a.K / 16;
    const uint8_t *rows = a.rows + (g * a.per_group + m0) * a.S;
    const int pieces = (nt + 3) / 4;              // 16-byte pieces of a row
    for (int i = tid; i < 128 * pieces; i += kOpThreads) {
        const int m = i / pieces, q = i - m * pieces;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (m0 + m < limit) {
            const uint4 u = *reinterpret_cast<const uint4 *>(rows + m * a.S + a.K / 2 + 4 * t0 + 16 * q);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int left = Kb - 4 * (t0 + 4 * q + j);     // columns from here on
                v[j] = left >= 4 ? w[j] : left <= 0 ? 0u : w[j] & ((1u << (8 * left)) - 1u);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint32_t *>(s + m * kOpPitch + 16 * q + 4 * j) = v[j];
    }
    if (blockIdx.y == 0 && tid < 128 && m0 + tid < limit)
        a.row_scale[g * a.per_group + m0 + tid] = *reinterpret_cast<const float *>(rows + tid * a.S + a.S - 16);
    if (a.codes) {                                // the same tiles' codes: 32 bytes a tile and row
        const int c0 = 32 * t0, units = (min(a.K / 2, c0 + 32 * nt) - c0) / 16, n = (int)min((int64_t)128, limit - m0);
        uint8_t *to = a.codes + (g * a.per_group + m0) * (a.K / 2) + c0;
        for (int i = tid; i < n * units; i += kOpThreads) {
            const int m = i / units, q = i - m * units;
            *reinterpret_cast<uint4 *>(to + (int64_t)m * (a.K / 2) + 16 * q) =
                *reinterpret_cast<const uint4 *>(rows + m * a.S + c0 + 16 * q);
        }
    }
    __syncthreads();
    uint8_t *out = a.scales + ((g * mt + m0 / 128) * kt + t0) * 512;
    for (int i = tid; i < 32 * nt; i += kOpThreads) {
        const int t = i >> 5, l = i & 31;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = *reinterpret_cast<const uint32_t *>(s + (l + 32 * j) * kOpPitch + 4 * t);
        *reinterpret_cast<uint4 *>(out + 512 * t + 16 * l) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// ---------------------------------------------------------------- products
// Codes [outer][inner bytes], copied in boxes of 128 bytes x `rows`.
bool code_map(CUtensorMap *m, const void *p, int64_t inner, int64_t outer, int64_t pitch, int64_t experts, int rows)
{
    return make_map_3d(m, MapType::U8, p, {(uint64_t)inner, (uint64_t)outer, (uint64_t)experts},
                       {(uint64_t)pitch, (uint64_t)(pitch * outer)}, {128, (uint32_t)rows, 1}, 128);
}

// Tiled scales: blocks of 128 rows, each of `tiles` tiles of 512 bytes; copied
// four tiles at a time of `blocks` blocks, as pieces of 128 bytes.
bool scale_map(CUtensorMap *m, const void *p, int64_t tiles, int64_t count, int blocks)
{
    return make_map_3d(m, MapType::U8, p, {128, (uint64_t)tiles * 4, (uint64_t)count}, {128, (uint64_t)tiles * 512},
                       {128, 16, (uint32_t)blocks}, 0);
}

template <int kCtas> cudaError_t gemm(const LaunchCtx &c, const Nvfp4GemmArgs &a)
{
    using C = GroupedCfg<true, false, false, kCtas, false>;
    GroupedParams p = {};
    const int64_t kt = ceil_div(a.K, 64);
    // slots are whole blocks of 128 rows, so that rows past the last whole block are
    // past the capacity; without slots the last block may be cut
    const int64_t blocks = a.offsets ? a.R_cap / 128 : ceil_div(a.R_cap, 128);
    // without whole blocks there is nothing to copy: the kernel only looks at the offsets
    const bool ok = blocks == 0 ||
                    (code_map(&p.map[kMapA], a.w, a.K / 2, a.N, a.ld_w, a.E, 128) &&
                     code_map(&p.map[kMapB], a.x, a.K / 2, a.R_cap, a.ld_x, 1, 64) &&
                     scale_map(&p.map[kMapSa], a.w_scales, kt, ceil_div(a.N, 128) * a.E, 1) &&
                     scale_map(&p.map[kMapSb], a.x_scales, kt, blocks, C::kTileN / 128) &&
                     make_map_3d(&p.out, MapType::Bf16, a.out, {(uint64_t)a.N, (uint64_t)a.R_cap, 1},
                                 {(uint64_t)a.N * 2, (uint64_t)a.N * 2 * a.R_cap}, {32, 32, 1}, 64));
    if (!ok)
        return cudaErrorInvalidValue;
    p.offsets = a.offsets;
    p.m_scale = a.w_row;
    p.n_scale = a.x_row;
    p.status = a.status;
    p.R_cap = a.offsets ? (int)(128 * blocks) : a.R_cap;
    p.E = a.E;
    p.M = p.N = a.N;
    p.K = a.K;
    return launch_grouped<C>(c, p, ceil_div(a.N, C::kSpan) * (ceil_div(a.R_cap, C::kTileN) + a.E));
}

template <bool kF32, int kCtas> cudaError_t wgrad(const LaunchCtx &c, const Nvfp4WgradArgs &a)
{
    using C = GroupedCfg<true, true, false, kCtas, kF32>;
    GroupedParams p = {};
    const uint64_t size = kF32 ? 4 : 2;
    if (!make_map_3d(&p.out, kF32 ? MapType::F32 : MapType::Bf16, a.d_w, {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E},
                     {a.K * size, a.K * size * a.N}, {(uint32_t)C::kChunk, 32, 1}, 128))
        return cudaErrorInvalidValue;
    p.col[kMapA] = a.dy;
    p.col[kMapB] = a.x;
    p.col[kMapSa] = a.dy_scales;
    p.col[kMapSb] = a.x_scales;
    p.offsets = a.offsets;
    p.m_scale = a.dy_enc;
    p.n_scale = a.x_enc;
    p.status = a.status;
    p.R_cap = a.R_cap;
    p.E = a.E;
    p.M = a.N;
    p.N = a.K;
    p.add = a.add;
    return launch_grouped<C>(c, p, a.E * ceil_div(a.N, C::kSpan) * ceil_div(a.K, C::kTileN));
}

} // namespace

cudaError_t launch_operand(const LaunchCtx &c, const OperandArgs &a)
{
    // (without any rows a CTA still looks at the offsets)
    const int64_t mt = a.offsets ? std::max<int64_t>(1, ceil_div(a.per_group, 128)) : ceil_div(a.per_group, 128);
    const int64_t kt = ceil_div(a.K, 64);
    if (a.groups * mt == 0)
        return cudaSuccess;
    return launch_pdl(operand_kernel, dim3((unsigned)(a.groups * mt), (unsigned)ceil_div(kt, kOpTiles)),
                      dim3(kOpThreads), 0, c.stream, a, (int)mt, (int)kt);
}

cudaError_t launch_nvfp4_gemm(const LaunchCtx &c, const Nvfp4GemmArgs &a)
{
    if (a.R_cap == 0 && !a.offsets)
        return cudaSuccess;
    using One = GroupedCfg<true, false, false, 1, false>;
    if (single_ctas<One>(c, a.N, ceil_div(a.R_cap, One::kTileN)))
        return gemm<1>(c, a);
    return gemm<2>(c, a);
}

cudaError_t launch_nvfp4_wgrad(const LaunchCtx &c, const Nvfp4WgradArgs &a)
{
    using One = GroupedCfg<true, true, false, 1, false>;
    if (single_ctas<One>(c, a.N, a.E * ceil_div(a.K, One::kTileN)))
        return a.f32 ? wgrad<true, 1>(c, a) : wgrad<false, 1>(c, a);
    return a.f32 ? wgrad<true, 2>(c, a) : wgrad<false, 2>(c, a);
}

} // namespace epq
