// extern "C" boundary of libepq.so (declared and documented in include/epq.h):
// argument validation on the host, the device guard, and the kernel launches.
// Nothing here allocates, frees or synchronises.
#include <stdint.h>
#include <string.h>

#include "../../include/epq.h"
#include "epq_internal.h"

namespace {

using epq::LaunchCtx;

// Makes `dev` current for the lifetime of the guard and restores the caller's
// current device afterwards (TE PR #3753, commit "guard the NVFP4 EP bindings
// with the input tensor's device").
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess)
            return;
        ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard()
    {
        if (ok && prev >= 0)
            cudaSetDevice(prev);
    }
};

// Device that owns `p`, or -1 if `p` is not device (or managed) memory.
int device_of(const void *p)
{
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return -1;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
        return -1;
    return a.device;
}

bool on_device(const void *p, int dev) { return p == nullptr || device_of(p) == dev; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count(int dev)
{
    static std::atomic<int> cache[64] = {};
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0)
            return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 1;
    if (dev >= 0 && dev < 64)
        cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

ep_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess)
        return EP_OK;
    (void)cudaGetLastError();
    return EP_ERR_CUDA;
}

bool shape_ok(int64_t T, int64_t H, int k, int E)
{
    if (T < 0 || T > (int64_t)INT32_MAX / 32 || H < 32 || H % 32 != 0 || H > (1 << 20))
        return false;
    if (k < 1 || k > 32 || E < 1 || E > 1024)
        return false;
    return true;
}

} // namespace

extern "C" {

size_t ep_nvfp4_row_bytes(int64_t H) { return H > 0 ? (size_t)epq::row_bytes(H) : 0; }

int64_t ep_rows_capacity(int64_t T, int k, int E, int A)
{
    if (T < 0 || k < 1 || E < 1 || A < 1)
        return 0;
    return T * (int64_t)k + (int64_t)E * (int64_t)(A - 1);
}

size_t ep_route_workspace_bytes(int64_t T, int k, int E)
{
    (void)k;
    return epq::route_workspace_bytes(T < 0 ? 0 : T, E < 1 ? 1 : E);
}

const char *ep_status_string(int s)
{
    switch (s) {
    case EP_OK: return "EP_OK";
    case EP_ERR_NULL: return "EP_ERR_NULL: a required pointer is NULL";
    case EP_ERR_SHAPE: return "EP_ERR_SHAPE: size out of range (H % 32, k in [1,32], E in [1,1024])";
    case EP_ERR_ALIGN: return "EP_ERR_ALIGN: alignment A must be a positive multiple of 128 and buffers 16-byte aligned";
    case EP_ERR_CAPACITY: return "EP_ERR_CAPACITY: R_cap or workspace too small";
    case EP_ERR_ARG: return "EP_ERR_ARG: bad argument";
    case EP_ERR_DEVICE: return "EP_ERR_DEVICE: pointer is not device memory of the input's device";
    case EP_ERR_CUDA: return "EP_ERR_CUDA: a CUDA call failed";
    default: return "unknown ep_status";
    }
}

ep_status ep_route_plan(const int32_t *topk_idx, int64_t T, int k, int E, int A, int64_t R_cap,
                        int32_t *expert_offsets, int32_t *expert_counts, int32_t *dest,
                        void *workspace, size_t ws_bytes, uint32_t *dev_status, void *stream)
{
    if (!expert_offsets || !expert_counts || !workspace || !dev_status || (T > 0 && (!topk_idx || !dest)))
        return EP_ERR_NULL;
    if (T < 0 || T * (int64_t)k > (int64_t)INT32_MAX || k < 1 || k > 32 || E < 1 || E > 1024)
        return EP_ERR_SHAPE;
    if (A <= 0 || A % 128 != 0)
        return EP_ERR_ALIGN;
    if (R_cap < ep_rows_capacity(T, k, E, A) || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (ws_bytes < ep_route_workspace_bytes(T, k, E))
        return EP_ERR_CAPACITY;
    const int dev = device_of(expert_offsets);
    if (dev < 0 || !on_device(topk_idx, dev) || !on_device(expert_counts, dev) || !on_device(dest, dev) ||
        !on_device(workspace, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    return cuda_status(epq::launch_route_plan(c, topk_idx, (int)T, k, E, A, expert_offsets, expert_counts,
                                              dest, (int32_t *)workspace, dev_status));
}

static ep_status pack_common_checks(const void *tokens, int64_t T, int64_t H, const int32_t *dest, int k,
                                    const int32_t *offsets, const int32_t *counts, int E, const uint8_t *out,
                                    int64_t R_cap, const uint32_t *dev_status, int *dev_out)
{
    if (!offsets || !counts || !out || !dev_status || (T > 0 && (!tokens || !dest)))
        return EP_ERR_NULL;
    if (!shape_ok(T, H, k, E))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (!aligned16(tokens) || !aligned16(out))
        return EP_ERR_ALIGN;
    const int dev = device_of(T > 0 ? tokens : (const void *)offsets);
    if (dev < 0 || !on_device(dest, dev) || !on_device(offsets, dev) || !on_device(counts, dev) ||
        !on_device(out, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    *dev_out = dev;
    return EP_OK;
}

ep_status ep_nvfp4_pack(const void *tokens_bf16, int64_t T, int64_t H, const int32_t *dest, int k,
                        const int32_t *expert_offsets, const int32_t *expert_counts, int E, uint8_t *rows,
                        int64_t R_cap, float *expert_amax, int rounding, uint64_t seed, uint32_t *dev_status,
                        void *stream)
{
    int dev = -1;
    ep_status st = pack_common_checks(tokens_bf16, T, H, dest, k, expert_offsets, expert_counts, E, rows,
                                      R_cap, dev_status, &dev);
    if (st != EP_OK)
        return st;
    if (!on_device(expert_amax, dev))
        return EP_ERR_DEVICE;
    if ((reinterpret_cast<uintptr_t>(expert_amax) & 3u) != 0)
        return EP_ERR_ALIGN;
    if (rounding != EP_ROUND_RNE && rounding != EP_ROUND_SR)
        return EP_ERR_ARG;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::PackAmax am;
    am.amax = expert_amax;
    return cuda_status(epq::launch_nvfp4_pack(c, (const uint16_t *)tokens_bf16, (int)T, (int)H, dest, k,
                                              expert_offsets, expert_counts, E, rows, (int)R_cap, rounding,
                                              seed, dev_status, false, am));
}

ep_status ep_nvfp4_dispatch(const int32_t *topk_idx, const void *tokens_bf16, int64_t T, int64_t H, int k, int E,
                            int A, int64_t R_cap, int32_t *expert_offsets, int32_t *expert_counts, int32_t *dest,
                            void *workspace, size_t ws_bytes, uint8_t *rows, float *expert_amax, int rounding,
                            uint64_t seed, uint32_t *dev_status, void *stream)
{
    if (!expert_offsets || !expert_counts || !workspace || !dev_status || !rows ||
        (T > 0 && (!topk_idx || !dest || !tokens_bf16)))
        return EP_ERR_NULL;
    if (T < 0 || T * (int64_t)k > (int64_t)INT32_MAX || k < 1 || k > 32 || E < 1 || E > 1024 ||
        !shape_ok(T, H, k, E))
        return EP_ERR_SHAPE;
    if (A <= 0 || A % 128 != 0 || !aligned16(tokens_bf16) || !aligned16(rows) ||
        (reinterpret_cast<uintptr_t>(expert_amax) & 3u) != 0)
        return EP_ERR_ALIGN;
    if (R_cap < ep_rows_capacity(T, k, E, A) || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (ws_bytes < ep_route_workspace_bytes(T, k, E))
        return EP_ERR_CAPACITY;
    if (rounding != EP_ROUND_RNE && rounding != EP_ROUND_SR)
        return EP_ERR_ARG;
    const int dev = device_of(expert_offsets);
    if (dev < 0 || !on_device(topk_idx, dev) || !on_device(tokens_bf16, dev) || !on_device(expert_counts, dev) ||
        !on_device(dest, dev) || !on_device(workspace, dev) || !on_device(rows, dev) || !on_device(dev_status, dev) ||
        !on_device(expert_amax, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    // the routing kernel zeroes expert_amax; the pack max-reduces into it,
    // taking each slot's expert straight from topk_idx
    cudaError_t err = epq::launch_route_plan(c, topk_idx, (int)T, k, E, A, expert_offsets, expert_counts, dest,
                                             (int32_t *)workspace, dev_status, expert_amax);
    epq::PackAmax am;
    am.topk = topk_idx;
    am.amax = expert_amax;
    if (err == cudaSuccess)
        err = epq::launch_nvfp4_pack(c, (const uint16_t *)tokens_bf16, (int)T, (int)H, dest, k, expert_offsets,
                                     expert_counts, E, rows, (int)R_cap, rounding, seed, dev_status, true, am);
    return cuda_status(err);
}

static ep_status colwise_rht_bf16_common(const void *x_bf16, int64_t R_cap, int64_t H, const int32_t *expert_offsets,
                                    int E, const float *amax_in, uint8_t *cw_codes, uint8_t *cw_scales,
                                    float *amax_row, float *amax_col, float *cw_scale_enc, int rounding,
                                    uint64_t seed, uint16_t rht_sign_mask, uint32_t *dev_status, void *stream,
                                    bool tiled)
{
    if (!x_bf16 || !expert_offsets || !amax_in || !cw_codes || !cw_scales || !amax_row || !amax_col ||
        !cw_scale_enc || !dev_status)
        return EP_ERR_NULL;
    if (!shape_ok(0, H, 1, E) || (tiled && H % 128 != 0))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || R_cap * H / 2 > (int64_t)INT32_MAX * 16)
        return EP_ERR_CAPACITY;
    if (rounding != EP_ROUND_RNE && rounding != EP_ROUND_SR)
        return EP_ERR_ARG;
    if (!aligned16(x_bf16) || !aligned16(cw_codes) || !aligned16(cw_scales))
        return EP_ERR_ALIGN;
    const int dev = device_of(x_bf16);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(amax_in, dev) || !on_device(cw_codes, dev) ||
        !on_device(cw_scales, dev) || !on_device(amax_row, dev) || !on_device(amax_col, dev) ||
        !on_device(cw_scale_enc, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    return cuda_status(epq::launch_colwise_rht_bf16(c, (const uint16_t *)x_bf16, (int)R_cap, (int)H, expert_offsets,
                                                    E, amax_in, cw_codes, cw_scales, amax_row, amax_col,
                                                    cw_scale_enc, rounding, seed, rht_sign_mask, dev_status, tiled));
}

ep_status ep_nvfp4_colwise_rht_bf16(const void *x_bf16, int64_t R_cap, int64_t H, const int32_t *expert_offsets,
                                    int E, const float *amax_in, uint8_t *cw_codes, uint8_t *cw_scales,
                                    float *amax_row, float *amax_col, float *cw_scale_enc, int rounding,
                                    uint64_t seed, uint16_t rht_sign_mask, uint32_t *dev_status, void *stream)
{
    return colwise_rht_bf16_common(x_bf16, R_cap, H, expert_offsets, E, amax_in, cw_codes, cw_scales, amax_row,
                                   amax_col, cw_scale_enc, rounding, seed, rht_sign_mask, dev_status, stream, false);
}

ep_status ep_nvfp4_colwise_rht_bf16_swizzled(const void *x_bf16, int64_t R_cap, int64_t H,
                                             const int32_t *expert_offsets, int E, const float *amax_in,
                                             uint8_t *cw_codes, uint8_t *cw_scales, float *amax_row, float *amax_col,
                                             float *cw_scale_enc, int rounding, uint64_t seed, uint16_t rht_sign_mask,
                                             uint32_t *dev_status, void *stream)
{
    return colwise_rht_bf16_common(x_bf16, R_cap, H, expert_offsets, E, amax_in, cw_codes, cw_scales, amax_row,
                                   amax_col, cw_scale_enc, rounding, seed, rht_sign_mask, dev_status, stream, true);
}

ep_status ep_mxfp8_colwise(const void *x_bf16, int64_t R_cap, int64_t H, const int32_t *expert_offsets, int E,
                           uint8_t *buf, uint32_t *dev_status, void *stream)
{
    if (!x_bf16 || !expert_offsets || !buf || !dev_status)
        return EP_ERR_NULL;
    if (!shape_ok(0, H, 1, E))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || R_cap * H > (int64_t)INT32_MAX * 32)
        return EP_ERR_CAPACITY;
    if (!aligned16(x_bf16) || !aligned16(buf))
        return EP_ERR_ALIGN;
    const int dev = device_of(x_bf16);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(buf, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    return cuda_status(epq::launch_mxfp8_colwise(c, (const uint16_t *)x_bf16, (int)R_cap, (int)H, expert_offsets, E,
                                                 buf, dev_status));
}

ep_status ep_mxfp8_pack(const void *tokens_bf16, int64_t T, int64_t H, const int32_t *dest, int k,
                        const int32_t *expert_offsets, const int32_t *expert_counts, int E, uint8_t *buf,
                        int64_t R_cap, uint32_t *dev_status, void *stream)
{
    int dev = -1;
    ep_status st = pack_common_checks(tokens_bf16, T, H, dest, k, expert_offsets, expert_counts, E, buf,
                                      R_cap, dev_status, &dev);
    if (st != EP_OK)
        return st;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    return cuda_status(epq::launch_mxfp8_pack(c, (const uint16_t *)tokens_bf16, (int)T, (int)H, dest, k,
                                              expert_offsets, expert_counts, E, buf, (int)R_cap, dev_status));
}

ep_status ep_nvfp4_unpack(const uint8_t *rows, int64_t R_cap, int64_t H, const int32_t *expert_offsets, int E,
                          void *out_bf16, uint32_t *dev_status, void *stream)
{
    if (!rows || !expert_offsets || !out_bf16 || !dev_status)
        return EP_ERR_NULL;
    if (!shape_ok(0, H, 1, E))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (!aligned16(rows) || !aligned16(out_bf16))
        return EP_ERR_ALIGN;
    const int dev = device_of(rows);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(out_bf16, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    return cuda_status(epq::launch_nvfp4_unpack(c, rows, (int)R_cap, (int)H, expert_offsets, E,
                                                (uint16_t *)out_bf16, dev_status));
}

static ep_status direct_receive_common(const uint8_t *rows, int64_t R_cap, int64_t H,
                                       const int32_t *expert_offsets, int E, const float *expert_amax,
                                       const ep_nvfp4_grouped *out,
                                       int rounding, uint64_t seed, uint16_t rht_sign_mask, uint32_t *dev_status,
                                       void *stream, bool swz)
{
    if (!rows || !expert_offsets || !out || !dev_status)
        return EP_ERR_NULL;
    if (!out->cw_codes || !out->cw_scales || !out->amax_row || !out->amax_col || !out->cw_scale_enc)
        return EP_ERR_NULL;
    const bool rw_any = out->rw_codes || out->rw_scales || out->rw_row_scale;
    const bool rw_all = out->rw_codes && out->rw_scales && out->rw_row_scale;
    if (rw_any && !rw_all)
        return EP_ERR_NULL;
    if (!shape_ok(0, H, 1, E) || (swz && H % 128 != 0))
        return EP_ERR_SHAPE;
    // element positions (the SR counters) below 2^36
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || R_cap * H > ((int64_t)1 << 36))
        return EP_ERR_CAPACITY;
    if (rounding != EP_ROUND_RNE && rounding != EP_ROUND_SR)
        return EP_ERR_ARG;
    if (!aligned16(rows) || !aligned16(out->cw_codes) || !aligned16(out->cw_scales) ||
        (rw_all && (!aligned16(out->rw_codes) || !aligned16(out->rw_scales))) ||
        (reinterpret_cast<uintptr_t>(expert_amax) & 3u) != 0)
        return EP_ERR_ALIGN;
    const int dev = device_of(rows);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(dev_status, dev) ||
        !on_device(out->rw_codes, dev) || !on_device(out->rw_scales, dev) || !on_device(out->rw_row_scale, dev) ||
        !on_device(out->cw_codes, dev) || !on_device(out->cw_scales, dev) || !on_device(out->amax_row, dev) ||
        !on_device(out->amax_col, dev) || !on_device(out->cw_scale_enc, dev) || !on_device(expert_amax, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::GroupedOut o{out->rw_codes, out->rw_scales, out->rw_row_scale, out->cw_codes,
                      out->cw_scales, out->amax_row, out->amax_col, out->cw_scale_enc};
    return cuda_status(epq::launch_direct_receive(c, rows, (int)R_cap, (int)H, expert_offsets, E, o, rounding,
                                                  seed, rht_sign_mask, dev_status, swz, expert_amax));
}

ep_status ep_nvfp4_direct_receive(const uint8_t *rows, int64_t R_cap, int64_t H, const int32_t *expert_offsets,
                                  int E, const float *expert_amax, const ep_nvfp4_grouped *out, int rounding,
                                  uint64_t seed, uint16_t rht_sign_mask, uint32_t *dev_status, void *stream)
{
    return direct_receive_common(rows, R_cap, H, expert_offsets, E, expert_amax, out, rounding, seed, rht_sign_mask,
                                 dev_status, stream, false);
}

ep_status ep_nvfp4_direct_receive_swizzled(const uint8_t *rows, int64_t R_cap, int64_t H,
                                           const int32_t *expert_offsets, int E, const float *expert_amax,
                                           const ep_nvfp4_grouped *out, int rounding, uint64_t seed,
                                           uint16_t rht_sign_mask, uint32_t *dev_status, void *stream)
{
    return direct_receive_common(rows, R_cap, H, expert_offsets, E, expert_amax, out, rounding, seed, rht_sign_mask,
                                 dev_status, stream, true);
}

// Checks of the unquantised [rows, H] buffers (elements of 2 or 4 bytes).
static bool dtype_ok(int dtype) { return dtype == EP_DTYPE_BF16 || dtype == EP_DTYPE_F32; }

static bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0; }

static bool layer_shape_ok(int64_t T, int64_t H, int k, int E)
{
    return T >= 0 && T <= (int64_t)INT32_MAX / 32 && H >= 1 && H <= (1 << 20) && k >= 1 && k <= 32 && E >= 1 &&
           E <= 1024;
}

static bool pitch_ok(int64_t ld, int64_t H) { return ld >= H && ld <= (int64_t)INT32_MAX; }

static ep_status scatter_common(const void *src, int dtype, int64_t T, int64_t H, int64_t ld_src, const void *rows_in,
                                int64_t ld_in, const int32_t *dest, const float *weights, int k,
                                const int32_t *offsets, const int32_t *counts, int E, void *rows_out, int64_t R_cap,
                                float *d_weights, uint32_t *dev_status, void *stream)
{
    if (!offsets || !counts || !dev_status || (T > 0 && (!src || !dest)) || (R_cap > 0 && !rows_out) ||
        (T > 0 && R_cap > 0 && d_weights && !rows_in))
        return EP_ERR_NULL;
    if (!layer_shape_ok(T, H, k, E) || !pitch_ok(ld_src, H) || (rows_in && !pitch_ok(ld_in, H)))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (!dtype_ok(dtype))
        return EP_ERR_ARG;
    const int elem = dtype == EP_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(src, elem) || !aligned_to(rows_in, elem) || !aligned_to(rows_out, elem) ||
        !aligned_to(weights, 4) || !aligned_to(d_weights, 4))
        return EP_ERR_ALIGN;
    const int dev = device_of(T > 0 ? src : (const void *)offsets);
    if (dev < 0 || !on_device(rows_in, dev) || !on_device(dest, dev) || !on_device(weights, dev) ||
        !on_device(offsets, dev) || !on_device(counts, dev) || !on_device(rows_out, dev) ||
        !on_device(d_weights, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::ScatterArgs a = {};
    a.src = src;
    a.ld_src = ld_src;
    a.rows_in = d_weights ? rows_in : nullptr;
    a.ld_in = ld_in;
    a.dest = dest;
    a.offsets = offsets;
    a.counts = counts;
    a.weights = weights;
    a.rows_out = rows_out;
    a.d_weights = d_weights;
    a.T = (int)T;
    a.k = k;
    a.H = (int)H;
    a.E = E;
    a.R_cap = (int)R_cap;
    a.status = dev_status;
    return cuda_status(epq::launch_scatter(c, a, dtype));
}

ep_status ep_pack(const void *tokens, int dtype, int64_t T, int64_t H, int64_t ld_tokens, const int32_t *dest, int k,
                  const int32_t *expert_offsets, const int32_t *expert_counts, int E, void *rows, int64_t R_cap,
                  uint32_t *dev_status, void *stream)
{
    return scatter_common(tokens, dtype, T, H, ld_tokens, nullptr, H, dest, nullptr, k, expert_offsets, expert_counts,
                          E, rows, R_cap, nullptr, dev_status, stream);
}

ep_status ep_combine_backward(const void *d_out, int dtype, int64_t T, int64_t H, int64_t ld_out, const void *rows,
                              int64_t ld_rows, const int32_t *dest, const float *weights, int k,
                              const int32_t *expert_offsets, const int32_t *expert_counts, int E, void *d_rows,
                              int64_t R_cap, float *d_weights, uint32_t *dev_status, void *stream)
{
    return scatter_common(d_out, dtype, T, H, ld_out, rows, ld_rows, dest, weights, k, expert_offsets, expert_counts,
                          E, d_rows, R_cap, d_weights, dev_status, stream);
}

ep_status ep_combine(const void *rows, int dtype, int64_t R_cap, int64_t H, int64_t ld_rows, const int32_t *index,
                     int slot_order, const float *weights, int64_t T, int k, void *out, uint32_t *dev_status,
                     void *stream)
{
    if (!dev_status || (T > 0 && (!out || (R_cap > 0 && !rows) || (!index && !slot_order))))
        return EP_ERR_NULL;
    if (!layer_shape_ok(T, H, k, 1) || !pitch_ok(ld_rows, H))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || (slot_order && R_cap < T * (int64_t)k))
        return EP_ERR_CAPACITY;
    if (!dtype_ok(dtype))
        return EP_ERR_ARG;
    const int elem = dtype == EP_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(rows, elem) || !aligned_to(out, elem) || !aligned_to(weights, 4))
        return EP_ERR_ALIGN;
    const int dev = device_of(R_cap > 0 && T > 0 ? rows : (const void *)dev_status);
    if (dev < 0 || !on_device(index, dev) || !on_device(weights, dev) || !on_device(out, dev) ||
        !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::CombineArgs a = {};
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.index = index;
    a.slot_order = slot_order != 0;
    a.weights = weights;
    a.out = out;
    a.T = (int)T;
    a.k = k;
    a.H = (int)H;
    a.R_cap = (int)R_cap;
    a.status = dev_status;
    return cuda_status(epq::launch_combine(c, a, dtype));
}

// Checks shared by the two passes of the gated activation, on their strided
// input (`width` columns).
static ep_status swiglu_checks(const void *in, int64_t ld, int64_t width, int64_t R_cap, int64_t I,
                               const int32_t *offsets, int E, const uint32_t *dev_status)
{
    if (!dev_status || (R_cap > 0 && !in))
        return EP_ERR_NULL;
    if (I < 32 || I % 32 != 0 || I > (1 << 19) || E < 1 || E > 1024 || (!offsets && E != 1) || !pitch_ok(ld, width))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (!aligned16(in) || ld % 8 != 0)
        return EP_ERR_ALIGN;
    return EP_OK;
}

ep_status ep_swiglu(const void *x_bf16, int64_t ld_x, int64_t R_cap, int64_t I, const int32_t *expert_offsets, int E,
                    void *act_bf16, uint8_t *ckpt, uint32_t *dev_status, void *stream)
{
    ep_status st = swiglu_checks(x_bf16, ld_x, 2 * I, R_cap, I, expert_offsets, E, dev_status);
    if (st != EP_OK)
        return st;
    if (R_cap > 0 && !act_bf16)
        return EP_ERR_NULL;
    if (!aligned16(act_bf16) || !aligned16(ckpt))
        return EP_ERR_ALIGN;
    const int dev = device_of(R_cap > 0 ? x_bf16 : (const void *)dev_status);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(act_bf16, dev) || !on_device(ckpt, dev) ||
        !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::SwigluArgs a = {};
    a.x = (const uint16_t *)x_bf16;
    a.ld = ld_x;
    a.ckpt_out = ckpt;
    a.offsets = expert_offsets;
    a.R_cap = (int)R_cap;
    a.I = (int)I;
    a.E = E;
    a.act = (uint16_t *)act_bf16;
    a.status = dev_status;
    return cuda_status(epq::launch_swiglu(c, a));
}

ep_status ep_swiglu_backward(const void *d_act_bf16, int64_t ld_act, const uint8_t *ckpt, int64_t R_cap, int64_t I,
                             const int32_t *expert_offsets, int E, void *d_x_bf16, void *act_bf16, float *expert_amax,
                             uint32_t *dev_status, void *stream)
{
    ep_status st = swiglu_checks(d_act_bf16, ld_act, I, R_cap, I, expert_offsets, E, dev_status);
    if (st != EP_OK)
        return st;
    if (R_cap > 0 && (!ckpt || !d_x_bf16))
        return EP_ERR_NULL;
    if (!aligned16(ckpt) || !aligned16(d_x_bf16) || !aligned16(act_bf16) || !aligned_to(expert_amax, 4))
        return EP_ERR_ALIGN;
    const int dev = device_of(R_cap > 0 ? d_act_bf16 : (const void *)dev_status);
    if (dev < 0 || !on_device(ckpt, dev) || !on_device(expert_offsets, dev) || !on_device(d_x_bf16, dev) ||
        !on_device(act_bf16, dev) || !on_device(expert_amax, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::SwigluArgs a = {};
    a.d_act = (const uint16_t *)d_act_bf16;
    a.ld = ld_act;
    a.ckpt = ckpt;
    a.offsets = expert_offsets;
    a.R_cap = (int)R_cap;
    a.I = (int)I;
    a.E = E;
    a.act = (uint16_t *)act_bf16;
    a.d_x = (uint16_t *)d_x_bf16;
    a.expert_amax = expert_amax;
    a.status = dev_status;
    return cuda_status(epq::launch_swiglu_backward(c, a));
}

// Sizes of the grouped products: their row tiles and output tiles are counted
// in 32 bits.
static bool product_ok(int64_t N, int64_t K, int E, int unit_n, int unit_k)
{
    return N >= unit_n && N <= (1 << 20) && N % unit_n == 0 && K >= unit_k && K <= (1 << 20) && K % unit_k == 0 &&
           E >= 1 && E <= 1024;
}

static bool tiles_ok(int64_t M, int64_t N_tiles) { return (M + 127) / 128 * N_tiles <= (int64_t)INT32_MAX; }

ep_status ep_grouped_gemm(const void *x_bf16, int64_t R_cap, int64_t K, int64_t ld_x, const void *w_bf16, int E,
                          int64_t N, int transposed, const int32_t *expert_offsets, void *out_bf16,
                          uint32_t *dev_status, void *stream)
{
    if (!dev_status || (R_cap > 0 && (!x_bf16 || !w_bf16 || !out_bf16)))
        return EP_ERR_NULL;
    if (!product_ok(N, K, E, 8, 8) || !pitch_ok(ld_x, K) || (!expert_offsets && E != 1))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || !tiles_ok(N, (R_cap + 255) / 256 + E))
        return EP_ERR_CAPACITY;
    if (!aligned16(x_bf16) || ld_x % 8 != 0 || !aligned16(w_bf16) || !aligned16(out_bf16))
        return EP_ERR_ALIGN;
    const int dev = device_of(R_cap > 0 ? x_bf16 : (const void *)dev_status);
    if (dev < 0 || !on_device(w_bf16, dev) || !on_device(expert_offsets, dev) || !on_device(out_bf16, dev) ||
        !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::GroupedGemmArgs a = {};
    a.x = x_bf16;
    a.ld_x = ld_x;
    a.w = w_bf16;
    a.transposed = transposed != 0;
    a.offsets = expert_offsets;
    a.out = out_bf16;
    a.R_cap = (int)R_cap;
    a.E = E;
    a.K = (int)K;
    a.N = (int)N;
    a.status = dev_status;
    return cuda_status(epq::launch_grouped_gemm(c, a));
}

// Checks that the weight gradients share.
static ep_status wgrad_checks(int64_t R_cap, int64_t N, int64_t K, int E, int unit, const int32_t *offsets,
                              const void *d_w, int dtype, int accumulate, const uint32_t *dev_status)
{
    if (!dev_status || !d_w)
        return EP_ERR_NULL;
    if (!product_ok(N, K, E, unit, unit) || (!offsets && E != 1))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || !tiles_ok(N, E * ((K + 255) / 256)))
        return EP_ERR_CAPACITY;
    if (!dtype_ok(dtype) || (accumulate && dtype != EP_DTYPE_F32))
        return EP_ERR_ARG;
    return aligned16(d_w) ? EP_OK : EP_ERR_ALIGN;
}

ep_status ep_grouped_wgrad(const void *dy_bf16, int64_t ld_dy, const void *x_bf16, int64_t ld_x, int64_t R_cap,
                           int64_t N, int64_t K, const int32_t *expert_offsets, const int32_t *expert_counts, int E,
                           void *d_w, int dtype, int accumulate, uint32_t *dev_status, void *stream)
{
    if (R_cap > 0 && (!dy_bf16 || !x_bf16))
        return EP_ERR_NULL;
    const ep_status st = wgrad_checks(R_cap, N, K, E, 8, expert_offsets, d_w, dtype, accumulate, dev_status);
    if (st != EP_OK)
        return st;
    if (!pitch_ok(ld_dy, N) || !pitch_ok(ld_x, K))
        return EP_ERR_SHAPE;
    if (!aligned16(dy_bf16) || ld_dy % 8 != 0 || !aligned16(x_bf16) || ld_x % 8 != 0 || !aligned_to(expert_counts, 4))
        return EP_ERR_ALIGN;
    const int dev = device_of(d_w);
    if (dev < 0 || !on_device(dy_bf16, dev) || !on_device(x_bf16, dev) || !on_device(expert_offsets, dev) ||
        !on_device(expert_counts, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::GroupedWgradArgs a = {};
    a.dy = dy_bf16;
    a.ld_dy = ld_dy;
    a.x = x_bf16;
    a.ld_x = ld_x;
    a.offsets = expert_offsets;
    a.counts = expert_counts;
    a.d_w = d_w;
    a.R_cap = (int)R_cap;
    a.E = E;
    a.N = (int)N;
    a.K = (int)K;
    a.f32 = dtype == EP_DTYPE_F32;
    a.add = accumulate != 0;
    a.status = dev_status;
    return cuda_status(epq::launch_grouped_wgrad(c, a));
}

size_t ep_nvfp4_scale_bytes(int64_t rows, int64_t H)
{
    return rows > 0 && H > 0 ? (size_t)((rows + 127) / 128 * ((H + 63) / 64) * 512) : 0;
}

ep_status ep_nvfp4_operand(const uint8_t *rows, int64_t groups, int64_t rows_per_group, int64_t H,
                           const int32_t *expert_offsets, int E, uint8_t *scales, float *row_scale, uint8_t *codes,
                           uint32_t *dev_status, void *stream)
{
    const bool any = groups > 0 && rows_per_group > 0;
    if (!dev_status || (any && (!rows || !scales || !row_scale)))
        return EP_ERR_NULL;
    if (!shape_ok(0, H, 1, E) || (expert_offsets ? groups != 1 : E != 1))
        return EP_ERR_SHAPE;
    if (groups < 0 || rows_per_group < 0 || rows_per_group > (int64_t)INT32_MAX ||
        (groups > 0 && rows_per_group > (int64_t)INT32_MAX / groups) ||
        groups * ((rows_per_group + 127) / 128) > (int64_t)INT32_MAX)
        return EP_ERR_CAPACITY;
    if (!aligned16(rows) || !aligned16(scales) || !aligned_to(row_scale, 4) || !aligned16(codes))
        return EP_ERR_ALIGN;
    const int dev = device_of(any ? (const void *)rows : (const void *)dev_status);
    if (dev < 0 || !on_device(expert_offsets, dev) || !on_device(scales, dev) || !on_device(row_scale, dev) ||
        !on_device(codes, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::OperandArgs a = {};
    a.rows = rows;
    a.S = epq::row_bytes(H);
    a.groups = groups;
    a.per_group = rows_per_group;
    a.offsets = expert_offsets;
    a.E = E;
    a.K = (int)H;
    a.scales = scales;
    a.row_scale = row_scale;
    a.codes = codes;
    a.status = dev_status;
    return cuda_status(epq::launch_operand(c, a));
}

ep_status ep_nvfp4_grouped_gemm(const uint8_t *x_codes, int64_t ld_x, const uint8_t *x_scales,
                                const float *x_row_scale, int64_t R_cap, int64_t K, const uint8_t *w_codes,
                                int64_t ld_w, const uint8_t *w_scales, const float *w_row_scale, int E, int64_t N,
                                const int32_t *expert_offsets, void *out_bf16, uint32_t *dev_status, void *stream)
{
    if (!dev_status || (R_cap > 0 && (!x_codes || !x_scales || !x_row_scale || !w_codes || !w_scales || !w_row_scale ||
                                      !out_bf16)))
        return EP_ERR_NULL;
    if (!product_ok(N, K, E, 8, 32) || !pitch_ok(ld_x, K / 2) || !pitch_ok(ld_w, K / 2) ||
        (!expert_offsets && E != 1))
        return EP_ERR_SHAPE;
    if (R_cap < 0 || R_cap > (int64_t)INT32_MAX || !tiles_ok(N, (R_cap + 255) / 256 + E))
        return EP_ERR_CAPACITY;
    if (!aligned16(x_codes) || ld_x % 16 != 0 || !aligned16(x_scales) || !aligned_to(x_row_scale, 4) ||
        !aligned16(w_codes) || ld_w % 16 != 0 || !aligned16(w_scales) || !aligned_to(w_row_scale, 4) ||
        !aligned16(out_bf16))
        return EP_ERR_ALIGN;
    const int dev = device_of(R_cap > 0 ? (const void *)x_codes : (const void *)dev_status);
    if (dev < 0 || !on_device(x_scales, dev) || !on_device(x_row_scale, dev) || !on_device(w_codes, dev) ||
        !on_device(w_scales, dev) || !on_device(w_row_scale, dev) || !on_device(expert_offsets, dev) ||
        !on_device(out_bf16, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::Nvfp4GemmArgs a = {};
    a.x = x_codes;
    a.x_scales = x_scales;
    a.x_row = x_row_scale;
    a.ld_x = ld_x;
    a.w = w_codes;
    a.w_scales = w_scales;
    a.w_row = w_row_scale;
    a.ld_w = ld_w;
    a.offsets = expert_offsets;
    a.out = out_bf16;
    a.R_cap = (int)R_cap;
    a.E = E;
    a.K = (int)K;
    a.N = (int)N;
    a.status = dev_status;
    return cuda_status(epq::launch_nvfp4_gemm(c, a));
}

ep_status ep_nvfp4_grouped_wgrad(const uint8_t *dy_codes, const uint8_t *dy_scales, const float *dy_scale_enc,
                                 const uint8_t *x_codes, const uint8_t *x_scales, const float *x_scale_enc,
                                 int64_t R_cap, int64_t N, int64_t K, const int32_t *expert_offsets, int E,
                                 void *d_w, int dtype, int accumulate, uint32_t *dev_status, void *stream)
{
    if (!dy_scale_enc || !x_scale_enc ||
        (R_cap > 0 && (!dy_codes || !dy_scales || !x_codes || !x_scales)))
        return EP_ERR_NULL;
    const ep_status st = wgrad_checks(R_cap, N, K, E, 128, expert_offsets, d_w, dtype, accumulate, dev_status);
    if (st != EP_OK)
        return st;
    if (!expert_offsets && R_cap % 128 != 0)
        return EP_ERR_SHAPE;
    if (!aligned16(dy_codes) || !aligned16(dy_scales) || !aligned_to(dy_scale_enc, 4) || !aligned16(x_codes) ||
        !aligned16(x_scales) || !aligned_to(x_scale_enc, 4))
        return EP_ERR_ALIGN;
    const int dev = device_of(d_w);
    if (dev < 0 || !on_device(dy_codes, dev) || !on_device(dy_scales, dev) || !on_device(dy_scale_enc, dev) ||
        !on_device(x_codes, dev) || !on_device(x_scales, dev) || !on_device(x_scale_enc, dev) ||
        !on_device(expert_offsets, dev) || !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::Nvfp4WgradArgs a = {};
    a.dy = dy_codes;
    a.dy_scales = dy_scales;
    a.dy_enc = dy_scale_enc;
    a.x = x_codes;
    a.x_scales = x_scales;
    a.x_enc = x_scale_enc;
    a.offsets = expert_offsets;
    a.d_w = d_w;
    a.R_cap = (int)R_cap;
    a.E = E;
    a.N = (int)N;
    a.K = (int)K;
    a.f32 = dtype == EP_DTYPE_F32;
    a.add = accumulate != 0;
    a.status = dev_status;
    return cuda_status(epq::launch_nvfp4_wgrad(c, a));
}

ep_status ep_nvfp4_matvec(const void *x_bf16, int64_t T, int64_t K, int64_t ld_x, int x_per_slot,
                          const uint8_t *w_rows, int E, int64_t N, const int32_t *topk_idx, int k, void *y_bf16,
                          uint32_t *dev_status, void *stream)
{
    if (!w_rows || !dev_status || (T > 0 && (!x_bf16 || !y_bf16)))
        return EP_ERR_NULL;
    if (!shape_ok(T, K, k, E) || K > 32768 || N < 1 || N > (1 << 20) || !pitch_ok(ld_x, K) ||
        (T > 0 && !topk_idx && (E != 1 || k != 1)))
        return EP_ERR_SHAPE;
    // every group of slots is looked for among all of them: past this the call
    // would take seconds, and it is not the call for such batches
    if (T * (int64_t)k > (1 << 20))
        return EP_ERR_CAPACITY;
    if (!aligned16(x_bf16) || ld_x % 8 != 0 || !aligned16(w_rows) || !aligned_to(y_bf16, 2))
        return EP_ERR_ALIGN;
    const int dev = device_of(w_rows);
    if (dev < 0 || !on_device(x_bf16, dev) || !on_device(topk_idx, dev) || !on_device(y_bf16, dev) ||
        !on_device(dev_status, dev))
        return EP_ERR_DEVICE;
    DeviceGuard g(dev);
    if (!g.ok)
        return EP_ERR_DEVICE;
    LaunchCtx c{(cudaStream_t)stream, dev, sm_count(dev)};
    epq::MatvecArgs a = {};
    a.x = (const uint16_t *)x_bf16;
    a.ld_x = ld_x;
    a.per_slot = x_per_slot != 0;
    a.w = w_rows;
    a.S = epq::row_bytes(K);
    a.topk = topk_idx;
    a.y = (uint16_t *)y_bf16;
    a.T = (int)T;
    a.k = k;
    a.K = (int)K;
    a.N = (int)N;
    a.E = E;
    a.status = dev_status;
    return cuda_status(epq::launch_matvec(c, a));
}

} // extern "C"
