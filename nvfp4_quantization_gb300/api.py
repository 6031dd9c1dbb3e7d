"""Python binding of libepq.so: argument marshalling only.

Each function takes torch CUDA tensors, allocates outputs the caller did not
pass (torch is the allocator; the library never allocates), and calls the C
entry point of the same name on the current torch stream.  Every step of the
path runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import EP_DTYPE_BF16, EP_DTYPE_F32, EP_ROUND_RNE, EP_ROUND_SR, EpGrouped, check

DEFAULT_ALIGNMENT = 128
DEFAULT_SIGN_MASK = 0xA53C


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def row_bytes(H: int) -> int:
    return int(_lib.lib().ep_nvfp4_row_bytes(int(H)))


def rows_capacity(T: int, k: int, E: int, A: int = DEFAULT_ALIGNMENT) -> int:
    return int(_lib.lib().ep_rows_capacity(int(T), int(k), int(E), int(A)))


@dataclass
class RoutePlan:
    """Device-resident routing plan (all int32 CUDA tensors)."""
    offsets: torch.Tensor     # [E+1]
    counts: torch.Tensor      # [E]
    dest: torch.Tensor        # [T*k]
    T: int
    k: int
    E: int
    A: int
    R_cap: int
    status: torch.Tensor      # uint32-valued int32 [1], EP_DEV_ERR_* bits


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def new_route_workspace(T: int, k: int, E: int, device) -> torch.Tensor:
    """A zero-filled workspace for ep_route_plan (reusable across calls)."""
    nbytes = int(_lib.lib().ep_route_workspace_bytes(int(T), int(k), int(E)))
    return torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)


def ep_route_plan(topk_idx: torch.Tensor, E: int, A: int = DEFAULT_ALIGNMENT, R_cap: int | None = None,
                  plan: RoutePlan | None = None, workspace: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, stream=None) -> RoutePlan:
    """Place every (token, slot) of ``topk_idx`` [T, k] (int32, -1 = dropped)
    in expert-contiguous, A-aligned row order."""
    _need_cuda(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    dev = topk_idx.device
    if R_cap is None:
        R_cap = rows_capacity(T, k, E, A)
    if plan is None:
        plan = RoutePlan(torch.empty(E + 1, dtype=torch.int32, device=dev),
                         torch.empty(E, dtype=torch.int32, device=dev),
                         torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
                         T, k, E, A, R_cap, status if status is not None else new_status(dev))
    if workspace is None:
        workspace = new_route_workspace(T, k, E, dev)
    st = _lib.lib().ep_route_plan(_ptr(topk_idx), T, k, E, A, R_cap, _ptr(plan.offsets), _ptr(plan.counts),
                                  _ptr(plan.dest), _ptr(workspace), workspace.numel() * 4, _ptr(plan.status),
                                  _stream(stream))
    check("ep_route_plan", st)
    return plan


def ep_route_plan_noalloc(topk_idx: torch.Tensor, plan: RoutePlan, stream=None) -> RoutePlan:
    """ep_route_plan into a caller-allocated ``plan``, with no workspace: the
    C entry point uses a fixed scratch array inside the library and allocates
    nothing (for hosts that own all device memory themselves).  Calls whose
    work may overlap on one GPU share that scratch and race."""
    _need_cuda(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    st = _lib.lib().ep_route_plan_noalloc(_ptr(topk_idx), T, k, plan.E, plan.A, plan.R_cap, _ptr(plan.offsets),
                                          _ptr(plan.counts), _ptr(plan.dest), _ptr(plan.status), _stream(stream))
    check("ep_route_plan_noalloc", st)
    return plan


def _need_amax(expert_amax, E: int):
    if expert_amax is not None:
        _need_cuda(expert_amax, "expert_amax", torch.float32)
        if expert_amax.numel() < E:
            raise ValueError("expert_amax needs E entries")


def ep_nvfp4_pack(tokens: torch.Tensor, plan: RoutePlan, rows: torch.Tensor | None = None,
                  rounding: int = EP_ROUND_RNE, seed: int = 0, expert_amax: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """BF16 tokens [T, H] -> packed NVFP4 rows [R_cap, row_bytes(H)] (uint8).
    ``expert_amax`` (f32 [E], filled by the caller, e.g. with zeros) receives
    the max of the token amaxes of each expert's rows."""
    _need_cuda(tokens, "tokens", torch.bfloat16)
    _need_amax(expert_amax, plan.E)
    T, H = tokens.shape
    S = row_bytes(H)
    if rows is None:
        rows = torch.empty((plan.R_cap, S), dtype=torch.uint8, device=tokens.device)
    _need_cuda(rows, "rows", torch.uint8)
    st = _lib.lib().ep_nvfp4_pack(_ptr(tokens), T, H, _ptr(plan.dest), plan.k, _ptr(plan.offsets),
                                  _ptr(plan.counts), plan.E, _ptr(rows), rows.shape[0], _ptr(expert_amax),
                                  int(rounding), int(seed) & ((1 << 64) - 1), _ptr(plan.status), _stream(stream))
    check("ep_nvfp4_pack", st)
    return rows


def ep_nvfp4_dispatch(tokens: torch.Tensor, topk_idx: torch.Tensor, E: int, A: int = DEFAULT_ALIGNMENT,
                      R_cap: int | None = None, plan: RoutePlan | None = None,
                      workspace: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                      rounding: int = EP_ROUND_RNE, seed: int = 0, status: torch.Tensor | None = None,
                      expert_amax: torch.Tensor | None = None, stream=None) -> tuple[RoutePlan, torch.Tensor]:
    """ep_route_plan then ep_nvfp4_pack in one C call (the pack overlaps the
    routing kernel); returns (plan, rows).  ``expert_amax`` (f32 [E]) is
    zeroed and then receives each expert's amax, for ep_nvfp4_direct_receive."""
    _need_cuda(tokens, "tokens", torch.bfloat16)
    _need_amax(expert_amax, E)
    _need_cuda(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    if tokens.shape[0] != T:
        raise ValueError("tokens and topk_idx disagree on T")
    H = tokens.shape[1]
    dev = topk_idx.device
    if R_cap is None:
        R_cap = plan.R_cap if plan is not None else rows_capacity(T, k, E, A)
    if plan is None:
        plan = RoutePlan(torch.empty(E + 1, dtype=torch.int32, device=dev),
                         torch.empty(E, dtype=torch.int32, device=dev),
                         torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
                         T, k, E, A, R_cap, status if status is not None else new_status(dev))
    if workspace is None:
        workspace = new_route_workspace(T, k, E, dev)
    if rows is None:
        rows = torch.empty((R_cap, row_bytes(H)), dtype=torch.uint8, device=dev)
    _need_cuda(rows, "rows", torch.uint8)
    if rows.shape[0] < R_cap:
        raise ValueError("rows has fewer than R_cap rows")
    st = _lib.lib().ep_nvfp4_dispatch(_ptr(topk_idx), _ptr(tokens), T, H, k, E, A, R_cap, _ptr(plan.offsets),
                                      _ptr(plan.counts), _ptr(plan.dest), _ptr(workspace), workspace.numel() * 4,
                                      _ptr(rows), _ptr(expert_amax), int(rounding), int(seed) & ((1 << 64) - 1),
                                      _ptr(plan.status), _stream(stream))
    check("ep_nvfp4_dispatch", st)
    return plan, rows


def ep_nvfp4_unpack(rows: torch.Tensor, H: int, offsets: torch.Tensor, E: int,
                    out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Packed rows -> BF16 [R_cap, H]; rows [0, offsets[E]) are written."""
    _need_cuda(rows, "rows", torch.uint8)
    R_cap = rows.shape[0]
    if out is None:
        out = torch.empty((R_cap, H), dtype=torch.bfloat16, device=rows.device)
    if status is None:
        status = new_status(rows.device)
    st = _lib.lib().ep_nvfp4_unpack(_ptr(rows), R_cap, H, _ptr(offsets), E, _ptr(out), _ptr(status),
                                    _stream(stream))
    check("ep_nvfp4_unpack", st)
    return out


def alloc_grouped(R_cap: int, H: int, E: int, device, rowwise: bool = True) -> dict:
    """Output tensors of the direct receive.  amax_row, amax_col and
    cw_scale_enc are the three rows of one [3, E] tensor, ``metadata``, so a
    single copy moves all three."""
    u8, f32 = torch.uint8, torch.float32
    meta = torch.empty((3, E), dtype=f32, device=device)
    g = dict(cw_codes=torch.empty(R_cap * H // 2, dtype=u8, device=device),
             cw_scales=torch.empty(R_cap * H // 16, dtype=u8, device=device),
             amax_row=meta[0], amax_col=meta[1], cw_scale_enc=meta[2], metadata=meta)
    if rowwise:
        g.update(rw_codes=torch.empty((R_cap, H // 2), dtype=u8, device=device),
                 rw_scales=torch.empty((R_cap, H // 16), dtype=u8, device=device),
                 rw_row_scale=torch.empty(R_cap, dtype=f32, device=device))
    return g


def grouped_struct(g: dict) -> EpGrouped:
    return EpGrouped(*[ctypes.c_void_p(g[n].data_ptr()) if g.get(n) is not None else None
                       for n, _ in EpGrouped._fields_])


def ep_nvfp4_direct_receive(rows: torch.Tensor, H: int, offsets: torch.Tensor, E: int,
                            out: dict | None = None, rounding: int = EP_ROUND_RNE, seed: int = 0,
                            sign_mask: int = DEFAULT_SIGN_MASK, status: torch.Tensor | None = None,
                            rowwise: bool = True, swizzled: bool = False, expert_amax: torch.Tensor | None = None,
                            stream=None) -> dict:
    """Packed rows -> grouped rowwise + columnwise-RHT NVFP4 operands (dict of
    tensors, see ep_nvfp4_grouped in include/epq.h).  ``swizzled`` calls
    ep_nvfp4_direct_receive_swizzled: both scale tensors in the tiled layout
    of block-scaled GEMM operands (H % 128 == 0).  ``expert_amax`` (f32 [E]):
    each expert's amax as the pack or dispatch reduced it; the call then
    skips its own pass over the row trailers."""
    _need_cuda(rows, "rows", torch.uint8)
    _need_amax(expert_amax, E)
    R_cap = rows.shape[0]
    if out is None:
        out = alloc_grouped(R_cap, H, E, rows.device, rowwise)
    if status is None:
        status = new_status(rows.device)
    desc = grouped_struct(out)
    name = "ep_nvfp4_direct_receive_swizzled" if swizzled else "ep_nvfp4_direct_receive"
    st = getattr(_lib.lib(), name)(_ptr(rows), R_cap, H, _ptr(offsets), E, _ptr(expert_amax), ctypes.byref(desc),
                                   int(rounding),
                                   int(seed) & ((1 << 64) - 1), int(sign_mask) & 0xFFFF, _ptr(status),
                                   _stream(stream))
    check(name, st)
    return out


def ep_nvfp4_colwise_rht_bf16(x: torch.Tensor, offsets: torch.Tensor, E: int, amax: torch.Tensor,
                              out: dict | None = None, rounding: int = EP_ROUND_RNE, seed: int = 0,
                              sign_mask: int = DEFAULT_SIGN_MASK, status: torch.Tensor | None = None,
                              stream=None) -> dict:
    """Expert-grouped BF16 rows [R_cap, H] + supplied per-expert amax [E]
    (f32) -> the columnwise RHT operand and its metadata (keys cw_codes,
    cw_scales, amax_row, amax_col, cw_scale_enc)."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(amax, "amax", torch.float32)
    R_cap, H = x.shape
    dev = x.device
    if out is None:
        out = {"cw_codes": torch.empty(R_cap * H // 2, dtype=torch.uint8, device=dev),
               "cw_scales": torch.empty(R_cap * H // 16, dtype=torch.uint8, device=dev),
               "amax_row": torch.empty(E, dtype=torch.float32, device=dev),
               "amax_col": torch.empty(E, dtype=torch.float32, device=dev),
               "cw_scale_enc": torch.empty(E, dtype=torch.float32, device=dev)}
    if status is None:
        status = new_status(dev)
    st = _lib.lib().ep_nvfp4_colwise_rht_bf16(_ptr(x), R_cap, H, _ptr(offsets), E, _ptr(amax), _ptr(out["cw_codes"]),
                                              _ptr(out["cw_scales"]), _ptr(out["amax_row"]), _ptr(out["amax_col"]),
                                              _ptr(out["cw_scale_enc"]), int(rounding), int(seed) & ((1 << 64) - 1),
                                              int(sign_mask) & 0xFFFF, _ptr(status), _stream(stream))
    check("ep_nvfp4_colwise_rht_bf16", st)
    return out


def ep_mxfp8_colwise(x: torch.Tensor, offsets: torch.Tensor, E: int, buf: torch.Tensor | None = None,
                     status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert-grouped BF16 rows [R_cap, H] -> one uint8 buffer: the columnwise
    MXFP8 data (expert e: [H][n_e]) then scales (expert e: [H][n_e/32])."""
    _need_cuda(x, "x", torch.bfloat16)
    R_cap, H = x.shape
    if buf is None:
        buf = torch.empty(R_cap * H + R_cap * (H // 32), dtype=torch.uint8, device=x.device)
    if status is None:
        status = new_status(x.device)
    st = _lib.lib().ep_mxfp8_colwise(_ptr(x), R_cap, H, _ptr(offsets), E, _ptr(buf), _ptr(status), _stream(stream))
    check("ep_mxfp8_colwise", st)
    return buf


def ep_mxfp8_pack(tokens: torch.Tensor, plan: RoutePlan, buf: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """BF16 tokens -> one uint8 buffer: data [R_cap, H] then scales [R_cap, H/32]."""
    _need_cuda(tokens, "tokens", torch.bfloat16)
    T, H = tokens.shape
    if buf is None:
        buf = torch.empty(plan.R_cap * H + plan.R_cap * (H // 32), dtype=torch.uint8, device=tokens.device)
    st = _lib.lib().ep_mxfp8_pack(_ptr(tokens), T, H, _ptr(plan.dest), plan.k, _ptr(plan.offsets),
                                  _ptr(plan.counts), plan.E, _ptr(buf), plan.R_cap, _ptr(plan.status),
                                  _stream(stream))
    check("ep_mxfp8_pack", st)
    return buf


# ---------------------------------------------------------------------------
# around the expert products: rows without quantisation, combine, activation,
# products of a few tokens
# ---------------------------------------------------------------------------
# With `stream`, outputs and scratch made here belong to that stream; inputs made
# on another one are the caller's to order (wait_stream) and keep (record_stream).
#
# What a kernel finds wrong it reports in `status` (new_status; EP_DEV_ERR_* bits)
# or in the plan's word.  A call without either makes a word of its own, which
# costs a fill and which nobody sees.
#
# These calls are made for single tokens too, where a call's host time is its
# time: operands go to the library as plain addresses, and the current stream's
# handle is read without building a Stream object (3 us of a 10 us call).
_DTYPE = {torch.bfloat16: EP_DTYPE_BF16, torch.float32: EP_DTYPE_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _at(t):
    return None if t is None else t.data_ptr()


def _stream_of(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need_dense(t: torch.Tensor, name: str, shape: tuple, dtype):
    """A contiguous operand of exactly this shape and type.  (That it is on the
    input's device is the library's own check, on the addresses.)"""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}")


def _need_rows(t: torch.Tensor, name: str, dtypes) -> int:
    """A 2-D CUDA input whose rows are contiguous; returns its row pitch in elements."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    n, width = t.shape
    pitch, unit = t.stride()
    if width > 1 and unit != 1:
        raise ValueError(f"{name} must have contiguous rows (its last stride is {unit})")
    if n <= 1:
        return max(width, 1)
    if pitch < width:
        raise ValueError(f"{name} must not have overlapping rows (row stride {pitch}, width {width})")
    return pitch


def _need_int32(t: torch.Tensor, name: str, n: int):
    if t.dtype != torch.int32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor with at least {n} entries")


def _need_plan(plan: RoutePlan, T: int):
    if plan.T != T:
        raise ValueError(f"the plan is for {plan.T} tokens, got {T}")
    _need_int32(plan.dest, "plan.dest", T * plan.k)
    _need_int32(plan.offsets, "plan.offsets", plan.E + 1)
    _need_int32(plan.counts, "plan.counts", plan.E)
    _need_int32(plan.status, "plan.status", 1)


def _empty(shape, dtype, device, stream):
    """An output on `stream` (the allocator must know where it is used)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status_or_new(status, device, stream):
    if status is None:
        if stream is None:
            return new_status(device)
        with torch.cuda.stream(stream):
            return new_status(device)
    _need_int32(status, "status", 1)
    return status


def ep_pack(tokens: torch.Tensor, plan: RoutePlan, rows: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """BF16 or FP32 tokens [T, H] -> expert rows [R_cap, H], copied as they
    are; padding rows are zeroed.  The gradient is ``ep_combine(d_rows, plan)``."""
    ld = _need_rows(tokens, "tokens", _DTYPE)
    T, H = tokens.shape
    _need_plan(plan, T)
    if rows is None:
        rows = _empty((plan.R_cap, H), tokens.dtype, tokens.device, stream)
    else:
        _need_dense(rows, "rows", (plan.R_cap, H), tokens.dtype)
    st = _lib.lib().ep_pack(tokens.data_ptr(), _DTYPE[tokens.dtype], T, H, ld, plan.dest.data_ptr(), plan.k,
                            plan.offsets.data_ptr(), plan.counts.data_ptr(), plan.E, rows.data_ptr(), plan.R_cap,
                            plan.status.data_ptr(), _stream_of(stream, tokens.device))
    if st:
        check("ep_pack", st)
    return rows


def ep_combine(rows: torch.Tensor, plan: RoutePlan | None = None, weights: torch.Tensor | None = None,
               topk_idx: torch.Tensor | None = None, out: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert rows -> tokens [T, H]: ``out[t] = sum_j weights[t, j] * row(t, j)``.

    With ``plan`` the rows are in its order ([R_cap, H]); with ``topk_idx``
    (int32 [T, k]) they are in slot order ([T*k, H], as ep_nvfp4_matvec writes
    them) and slots whose id is negative are left out.  ``weights`` f32 [T, k],
    None = 1.  Errors are reported in ``status``, or in the plan's word."""
    ld = _need_rows(rows, "rows", _DTYPE)
    n, H = rows.shape
    dev = rows.device
    if (plan is None) == (topk_idx is None):
        raise ValueError("ep_combine takes either plan or topk_idx")
    if plan is not None:
        T, k, index = plan.T, plan.k, plan.dest
        _need_plan(plan, T)
        if status is None:
            status = plan.status
    else:
        if topk_idx.dim() != 2:
            raise ValueError("topk_idx must have two dimensions")
        T, k = topk_idx.shape
        _need_dense(topk_idx, "topk_idx", (T, k), torch.int32)
        if n != T * k:
            raise ValueError(f"rows in slot order must be {T * k}, got {n}")
        index = topk_idx
    status = _status_or_new(status, dev, stream)
    if weights is not None:
        _need_dense(weights, "weights", (T, k), torch.float32)
    if out is None:
        out = _empty((T, H), rows.dtype, dev, stream)
    else:
        _need_dense(out, "out", (T, H), rows.dtype)
    st = _lib.lib().ep_combine(rows.data_ptr(), _DTYPE[rows.dtype], n, H, ld, index.data_ptr(), int(plan is None),
                               _at(weights), T, k, out.data_ptr(), status.data_ptr(), _stream_of(stream, dev))
    if st:
        check("ep_combine", st)
    return out


def ep_combine_backward(d_out: torch.Tensor, plan: RoutePlan, weights: torch.Tensor | None = None,
                        rows: torch.Tensor | None = None, d_rows: torch.Tensor | None = None,
                        d_weights: torch.Tensor | None = None,
                        stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradients of ``ep_combine(rows, plan, weights)`` from d_out [T, H]:
    (d_rows [R_cap, H], d_weights f32 [T, k]).  Without ``rows`` the weights'
    gradient is not computed (None)."""
    ld = _need_rows(d_out, "d_out", _DTYPE)
    T, H = d_out.shape
    dev, dt = d_out.device, d_out.dtype
    _need_plan(plan, T)
    k, R_cap = plan.k, plan.R_cap
    ld_rows = H
    if weights is not None:
        _need_dense(weights, "weights", (T, k), torch.float32)
    if rows is not None:
        ld_rows = _need_rows(rows, "rows", (dt,))
        if rows.shape != (R_cap, H):
            raise ValueError(f"rows must have shape {(R_cap, H)}, got {tuple(rows.shape)}")
        if d_weights is None:
            d_weights = _empty((T, k), torch.float32, dev, stream)
        else:
            _need_dense(d_weights, "d_weights", (T, k), torch.float32)
    elif d_weights is not None:
        raise ValueError("d_weights needs rows")
    if d_rows is None:
        d_rows = _empty((R_cap, H), dt, dev, stream)
    else:
        _need_dense(d_rows, "d_rows", (R_cap, H), dt)
    st = _lib.lib().ep_combine_backward(d_out.data_ptr(), _DTYPE[dt], T, H, ld, _at(rows), ld_rows,
                                        plan.dest.data_ptr(), _at(weights), k, plan.offsets.data_ptr(),
                                        plan.counts.data_ptr(), plan.E, d_rows.data_ptr(), R_cap, _at(d_weights),
                                        plan.status.data_ptr(), _stream_of(stream, dev))
    if st:
        check("ep_combine_backward", st)
    return d_rows, d_weights


def swiglu_checkpoint_bytes(R_cap: int, I: int) -> int:
    """Bytes of ep_swiglu's checkpoint: E4M3 data [R_cap, 2I], then E8M0 scales [R_cap, 2I/32]."""
    return R_cap * 2 * I + R_cap * (2 * I // 32)


def _need_offsets(offsets, E: int):
    if offsets is not None:
        _need_int32(offsets, "offsets", E + 1)
    elif E != 1:
        raise ValueError("E must be 1 without offsets")


def ep_swiglu(x: torch.Tensor, offsets: torch.Tensor | None = None, E: int = 1, act: torch.Tensor | None = None,
              ckpt: torch.Tensor | None = None, checkpoint: bool = True, status: torch.Tensor | None = None,
              stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gated activation of x [R_cap, 2I] (gate columns, then up columns), BF16:
    (act [R_cap, I], checkpoint).  The checkpoint (uint8,
    swiglu_checkpoint_bytes) holds x in MXFP8 for ep_swiglu_backward;
    ``checkpoint=False`` leaves it out (None).  With ``offsets`` (int32 [E+1])
    only rows [0, offsets[E]) are processed; more than R_cap of them are
    reported in ``status`` (not seen without it)."""
    ld = _need_rows(x, "x", (torch.bfloat16,))
    R_cap, width = x.shape
    if width % 64:
        raise ValueError(f"x needs two halves of a multiple of 32 columns, got {width}")
    I, dev = width // 2, x.device
    _need_offsets(offsets, E)
    if act is None:
        act = _empty((R_cap, I), torch.bfloat16, dev, stream)
    else:
        _need_dense(act, "act", (R_cap, I), torch.bfloat16)
    if ckpt is not None:
        _need_dense(ckpt, "ckpt", (swiglu_checkpoint_bytes(R_cap, I),), torch.uint8)
    elif checkpoint:
        ckpt = _empty((swiglu_checkpoint_bytes(R_cap, I),), torch.uint8, dev, stream)
    status = _status_or_new(status, dev, stream)
    st = _lib.lib().ep_swiglu(x.data_ptr(), ld, R_cap, I, _at(offsets), E, act.data_ptr(), _at(ckpt),
                              status.data_ptr(), _stream_of(stream, dev))
    if st:
        check("ep_swiglu", st)
    return act, ckpt


def ep_swiglu_backward(d_act: torch.Tensor, ckpt: torch.Tensor, offsets: torch.Tensor | None = None, E: int = 1,
                       d_x: torch.Tensor | None = None, act: torch.Tensor | None = None, recompute: bool = False,
                       expert_amax: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradient of ep_swiglu from its checkpoint: (d_x [R_cap, 2I], act).  The
    activation is written again (from the checkpoint's values) into ``act``, or
    into a new tensor with ``recompute=True``; else None.  ``expert_amax`` (f32
    [E], filled by the caller, e.g. with zeros) receives the max of each
    expert's |d_x| before rounding: the amax of ep_nvfp4_colwise_rht_bf16.
    ``status`` as in ep_swiglu."""
    ld = _need_rows(d_act, "d_act", (torch.bfloat16,))
    R_cap, I = d_act.shape
    dev = d_act.device
    if I % 32:
        raise ValueError(f"d_act needs a multiple of 32 columns, got {I}")
    _need_offsets(offsets, E)
    _need_dense(ckpt, "ckpt", (swiglu_checkpoint_bytes(R_cap, I),), torch.uint8)
    if d_x is None:
        d_x = _empty((R_cap, 2 * I), torch.bfloat16, dev, stream)
    else:
        _need_dense(d_x, "d_x", (R_cap, 2 * I), torch.bfloat16)
    if act is not None:
        _need_dense(act, "act", (R_cap, I), torch.bfloat16)
    elif recompute:
        act = _empty((R_cap, I), torch.bfloat16, dev, stream)
    if expert_amax is not None:
        _need_dense(expert_amax, "expert_amax", (E,), torch.float32)
    status = _status_or_new(status, dev, stream)
    st = _lib.lib().ep_swiglu_backward(d_act.data_ptr(), ld, ckpt.data_ptr(), R_cap, I, _at(offsets), E,
                                       d_x.data_ptr(), _at(act), _at(expert_amax), status.data_ptr(),
                                       _stream_of(stream, dev))
    if st:
        check("ep_swiglu_backward", st)
    return d_x, act


def ep_nvfp4_pack_weights(w: torch.Tensor, rounding: int = EP_ROUND_RNE, seed: int = 0, stream=None) -> torch.Tensor:
    """BF16 weights [E, N, K] -> packed NVFP4 rows [E, N, row_bytes(K)] for
    ep_nvfp4_matvec: ep_nvfp4_pack with every row in its own place."""
    _need_cuda(w, "w", torch.bfloat16)
    if w.dim() != 3:
        raise ValueError("w must have three dimensions [E, N, K]")
    E, N, K = w.shape
    n = E * N

    def pack():
        offsets = torch.tensor([0, n], dtype=torch.int32, device=w.device)
        plan = RoutePlan(offsets, offsets[1:], torch.arange(max(n, 1), dtype=torch.int32, device=w.device), n, 1, 1,
                         DEFAULT_ALIGNMENT, n, new_status(w.device))
        return ep_nvfp4_pack(w.view(n, K), plan, rounding=rounding, seed=seed)

    if stream is None:
        rows = pack()
    else:
        with torch.cuda.stream(stream):
            rows = pack()
    return rows.view(E, N, rows.shape[1])


def ep_nvfp4_matvec(x: torch.Tensor, w_rows: torch.Tensor, topk_idx: torch.Tensor | None = None,
                    y: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Products of a few tokens with NVFP4 expert weights, for decode batches:
    ``y[t*k + j] = W[topk_idx[t, j]] @ x``, BF16 [T*k, N].

    ``w_rows`` uint8 [E, N, row_bytes(K)] (ep_nvfp4_pack_weights); ``x`` BF16
    [T, K] (one row for all slots of a token) or [T*k, K] (one per slot).
    Slots whose id is -1 give zero rows.  Without ``topk_idx`` E must be 1 and
    the call is a dense layer on x [T, K].  An id out of range (its rows are
    zero too) and a wait that gave up (rows of y left as they were) are reported
    in ``status`` and not seen without it."""
    ld = _need_rows(x, "x", (torch.bfloat16,))
    n, K = x.shape
    dev = x.device
    if w_rows.dim() != 3:
        raise ValueError("w_rows must have three dimensions [E, N, row_bytes(K)]")
    E, N, S = w_rows.shape
    _need_dense(w_rows, "w_rows", (E, N, (9 * K // 16 + 31) // 16 * 16), torch.uint8)   # row_bytes(K)
    if topk_idx is None:
        if E != 1:
            raise ValueError("w_rows of several experts needs topk_idx")
        T, k = n, 1
    else:
        if topk_idx.dim() != 2:
            raise ValueError("topk_idx must have two dimensions")
        T, k = topk_idx.shape
        _need_dense(topk_idx, "topk_idx", (T, k), torch.int32)
        if n != T and n != T * k:
            raise ValueError(f"x must have {T} or {T * k} rows, got {n}")
    if y is None:
        y = _empty((T * k, N), torch.bfloat16, dev, stream)
    else:
        _need_dense(y, "y", (T * k, N), torch.bfloat16)
    status = _status_or_new(status, dev, stream)
    st = _lib.lib().ep_nvfp4_matvec(x.data_ptr(), T, K, ld, int(n != T), w_rows.data_ptr(), E, N, _at(topk_idx), k,
                                    y.data_ptr(), status.data_ptr(), _stream_of(stream, dev))
    if st:
        check("ep_nvfp4_matvec", st)
    return y
