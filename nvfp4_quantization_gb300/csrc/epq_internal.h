// Host-side declarations shared by the epq translation units: kernel
// launchers (one per kernel family) and launch helpers.  The extern "C"
// boundary that validates arguments lives in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

namespace epq {

struct LaunchCtx {
    cudaStream_t stream;
    int device;
    int num_sms;
};

// Launch `kernel` with programmatic stream serialization (PDL) so that its
// launch latency overlaps the tail of the preceding kernel; every epq kernel
// calls griddepcontrol.wait before it reads memory another kernel wrote.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Sets the dynamic shared-memory limit of `kernel` once per device (it is a
// per-function attribute; setting it again inside a stream capture is avoided).
// The per-device flags are atomic: calls from several host threads may race to
// set the same attribute, which is harmless.
template <typename K>
cudaError_t ensure_smem_limit(K kernel, int device, int bytes, std::atomic<uint32_t> *done_mask_words /*[2]*/)
{
    const int w = device >> 5;
    const uint32_t bit = 1u << (device & 31);
    if (device >= 0 && device < 64 && (done_mask_words[w].load(std::memory_order_acquire) & bit))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && device >= 0 && device < 64)
        done_mask_words[w].fetch_or(bit, std::memory_order_release);
    return e;
}

size_t route_workspace_bytes(int64_t T, int E);
// Launched without programmatic dependency: it starts only once every earlier
// kernel on the stream has finished (launch_nvfp4_pack's `early` relies on it).
// amax_zero (optional, f32 [E]): set to 0 by the kernel, for a pack that
// max-reduces the per-expert amax into it.
cudaError_t launch_route_plan(const LaunchCtx &c, const int32_t *topk, int T, int k, int E, int A,
                              int32_t *offsets, int32_t *counts, int32_t *dest, int32_t *hist,
                              uint32_t *status, float *amax_zero = nullptr);

// The pack's optional per-expert amax: every written row's token amax A_t is
// max-reduced into amax[e] of its expert e (the array holds zeros, or an
// earlier partial max, when the pack starts).  topk, when given, names the
// expert of each (token, slot) directly; otherwise it is found from the row
// index and the expert offsets.
struct PackAmax {
    const int32_t *topk = nullptr;
    float *amax = nullptr;
};

// early: the launch directly follows launch_route_plan on the same stream,
// so the tokens may be read before the wait for the routing kernel.
cudaError_t launch_nvfp4_pack(const LaunchCtx &c, const uint16_t *tokens, int T, int H,
                              const int32_t *dest, int k, const int32_t *offsets,
                              const int32_t *counts, int E, uint8_t *rows, int R_cap,
                              int rounding, uint64_t seed, uint32_t *status, bool early = false,
                              PackAmax am = PackAmax());

cudaError_t launch_mxfp8_pack(const LaunchCtx &c, const uint16_t *tokens, int T, int H,
                              const int32_t *dest, int k, const int32_t *offsets,
                              const int32_t *counts, int E, uint8_t *buf, int R_cap,
                              uint32_t *status);

cudaError_t launch_nvfp4_unpack(const LaunchCtx &c, const uint8_t *rows, int R_cap, int H,
                                const int32_t *offsets, int E, uint16_t *out, uint32_t *status);

struct GroupedOut {
    uint8_t *rw_codes;
    uint8_t *rw_scales;
    float *rw_row_scale;
    uint8_t *cw_codes;
    uint8_t *cw_scales;
    float *amax_row;
    float *amax_col;
    float *scale_enc;
};

// tiled: the scales in the layout of block-scaled GEMM operands (H % 128 == 0,
// checked by the caller).
cudaError_t launch_colwise_rht_bf16(const LaunchCtx &c, const uint16_t *x, int R_cap, int H, const int32_t *offsets,
                                    int E, const float *amax_in, uint8_t *cw_codes, uint8_t *cw_scales,
                                    float *amax_row, float *amax_col, float *scale_enc, int rounding, uint64_t seed,
                                    uint32_t sign_mask, uint32_t *status, bool tiled = false);

cudaError_t launch_mxfp8_colwise(const LaunchCtx &c, const uint16_t *x, int R_cap, int H, const int32_t *offsets,
                                 int E, uint8_t *buf, uint32_t *status);

// swz: both scale tensors in the tiled layout of block-scaled GEMM operands
// (H % 128 == 0, checked by the caller).
cudaError_t launch_direct_receive(const LaunchCtx &c, const uint8_t *rows, int R_cap, int H,
                                  const int32_t *offsets, int E, const GroupedOut &out,
                                  int rounding, uint64_t seed, uint32_t sign_mask,
                                  uint32_t *status, bool swz = false, const float *amax_in = nullptr);

// Element types of the unquantised row buffers (EP_DTYPE_* of the C ABI).
constexpr int kBf16 = 0;
constexpr int kF32 = 1;

struct CombineArgs {
    const void *rows;        // [R_cap, H], row pitch ld_rows elements
    int64_t ld_rows;
    const int32_t *index;    // [T * k]: row of the slot, or (slot_order) negative = dropped; NULL: none dropped
    bool slot_order;         // slot (t, j) is row t * k + j
    const float *weights;    // [T * k] or NULL (1)
    void *out;               // [T, H]
    int T, k, H, R_cap;
    uint32_t *status;
};

cudaError_t launch_combine(const LaunchCtx &c, const CombineArgs &a, int dtype);

// ep_pack (weights, rows_in, d_weights NULL) and ep_combine_backward.
struct ScatterArgs {
    const void *src;         // [T, H], row pitch ld_src elements
    int64_t ld_src;
    const void *rows_in;     // [R_cap, H], row pitch ld_in; with d_weights only
    int64_t ld_in;
    const int32_t *dest, *offsets, *counts;
    const float *weights;    // [T * k] or NULL (1)
    void *rows_out;          // [R_cap, H]
    float *d_weights;        // [T * k] or NULL
    int T, k, H, E, R_cap;
    int pad_split;           // CTAs that share an expert's padding rows (set by the launcher)
    uint32_t *status;
};

cudaError_t launch_scatter(const LaunchCtx &c, const ScatterArgs &a, int dtype);

struct SwigluArgs {
    const uint16_t *x;       // forward: [R_cap, 2I], row pitch ld
    const uint16_t *d_act;   // backward: [R_cap, I], row pitch ld
    int64_t ld;
    const uint8_t *ckpt;     // backward: data [R_cap, 2I], then scales [R_cap, 2I/32]
    uint8_t *ckpt_out;       // forward: the same, or NULL
    const int32_t *offsets;  // [E + 1] or NULL: all R_cap rows, one expert
    int R_cap, I, E;
    uint16_t *act;           // [R_cap, I]; backward: or NULL
    uint16_t *d_x;           // backward: [R_cap, 2I]
    float *expert_amax;      // backward: [E] or NULL
    uint32_t *status;
};

cudaError_t launch_swiglu(const LaunchCtx &c, const SwigluArgs &a);
cudaError_t launch_swiglu_backward(const LaunchCtx &c, const SwigluArgs &a);

struct MatvecArgs {
    const uint16_t *x;       // [T or T * k, K], row pitch ld_x
    int64_t ld_x;
    bool per_slot;           // x has a row per slot, not per token
    const uint8_t *w;        // packed NVFP4 rows [E * N, S]
    int64_t S;
    const int32_t *topk;     // [T * k] or NULL: expert 0
    uint16_t *y;             // [T * k, N]
    int T, k, K, N, E;
    uint32_t *status;
};

cudaError_t launch_matvec(const LaunchCtx &c, const MatvecArgs &a);

// Tensor map of a 2-D byte tensor [outer][inner] with a row pitch of `pitch`
// bytes and a box of box_outer rows x box_inner bytes (no swizzle, L2
// promotion 256 B); false if the driver refuses it.  elem = 2: inner and
// box_inner count 16-bit units instead.
bool make_map(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint64_t pitch,
              uint32_t box_inner, uint32_t box_outer, int elem = 1);

// Tensor map of a 3-D tensor (dims[0] contiguous, pitches of the other two in
// bytes), with a swizzle of 0, 64 or 128 bytes.
enum class MapType { U8, Bf16, F32 };
bool make_map_3d(CUtensorMap *m, MapType type, const void *base, const uint64_t (&dims)[3],
                 const uint64_t (&pitches)[2], const uint32_t (&box)[3], int swizzle);

// y[r] = W_e x[r] for the rows of expert e; `transposed`: w is [E, K, N].
struct GroupedGemmArgs {
    const void *x;           // BF16 [R_cap, K], row pitch ld_x elements
    int64_t ld_x;
    const void *w;           // BF16 [E, N, K] or [E, K, N]
    bool transposed;
    const int32_t *offsets;  // [E + 1] or NULL: all R_cap rows, one expert
    void *out;               // BF16 [R_cap, N]
    int R_cap, E, K, N;
    uint32_t *status;
};

cudaError_t launch_grouped_gemm(const LaunchCtx &c, const GroupedGemmArgs &a);

// d_w[e] = sum over e's rows of dy[r] x[r]^T.
struct GroupedWgradArgs {
    const void *dy, *x;      // BF16 [R_cap, N] and [R_cap, K], row pitches ld_dy and ld_x elements
    int64_t ld_dy, ld_x;
    const int32_t *offsets;  // [E + 1] or NULL
    const int32_t *counts;   // [E] or NULL: all rows of a slot
    void *d_w;               // [E, N, K], FP32 or BF16
    int R_cap, E, N, K;
    bool f32, add;
    uint32_t *status;
};

cudaError_t launch_grouped_wgrad(const LaunchCtx &c, const GroupedWgradArgs &a);

// Packed rows -> tiled block scales and row scales.
struct OperandArgs {
    const uint8_t *rows;     // [groups * per_group, S]
    int64_t S;
    int64_t groups, per_group;
    const int32_t *offsets;  // with one group: [E + 1] or NULL
    int E, K;
    uint8_t *scales;         // [groups][ceil(per_group / 128)][ceil(K / 64)][512]
    float *row_scale;        // [groups * per_group]
    uint8_t *codes;          // [groups * per_group, K / 2] or NULL
    uint32_t *status;
};

cudaError_t launch_operand(const LaunchCtx &c, const OperandArgs &a);

struct Nvfp4GemmArgs {
    const uint8_t *x, *x_scales;   // codes, row pitch ld_x bytes; tiled scales
    const float *x_row;            // [R_cap]
    int64_t ld_x;
    const uint8_t *w, *w_scales;   // codes [E][N], row pitch ld_w bytes; tiled scales
    const float *w_row;            // [E * N]
    int64_t ld_w;
    const int32_t *offsets;
    void *out;                     // BF16 [R_cap, N]
    int R_cap, E, K, N;
    uint32_t *status;
};

cudaError_t launch_nvfp4_gemm(const LaunchCtx &c, const Nvfp4GemmArgs &a);

struct Nvfp4WgradArgs {
    const uint8_t *dy, *dy_scales, *x, *x_scales;   // columnwise operands, tiled scales
    const float *dy_enc, *x_enc;                    // [E]
    const int32_t *offsets;                         // or NULL
    void *d_w;                                      // [E, N, K]
    int R_cap, E, N, K;
    bool f32, add;
    uint32_t *status;
};

cudaError_t launch_nvfp4_wgrad(const LaunchCtx &c, const Nvfp4WgradArgs &a);

// Bytes of a packed NVFP4 row: roundup16(9H/16 + 16).
inline int64_t row_bytes(int64_t H) { return (9 * H / 16 + 16 + 15) / 16 * 16; }

} // namespace epq
