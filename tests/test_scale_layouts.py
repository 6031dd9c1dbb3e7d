"""The products read block scales in tiles; operands whose scales lie row after
row have the same names, shapes and sizes, and are refused.
"""
import pytest
import torch

import nvfp4_quantization_gb300 as nq
from nvfp4_quantization_gb300 import api


def test_the_note_on_a_tensor():
    out = dict(cw_scales=torch.zeros(8, dtype=torch.uint8), rw_scales=torch.zeros(8, dtype=torch.uint8), rw_codes=None)
    for name in ("cw_scales", "rw_scales"):
        api._need_tiled(out[name], name)              # nobody knows: taken as it is
    api._set_layout(out, False)
    for name in ("cw_scales", "rw_scales"):
        with pytest.raises(ValueError, match="swizzled=True"):
            api._need_tiled(out[name], name)
        with pytest.raises(ValueError, match="swizzled=True"):
            api._need_tiled(dict(out, K=64)[name], name)
    api._set_layout(dict(cw_scales=out["cw_scales"]), True)
    api._need_tiled(out["cw_scales"], "cw_scales")
    with pytest.raises(ValueError):
        api._need_tiled(out["rw_scales"], "rw_scales")


@pytest.mark.gpu
def test_products_refuse_scales_that_lie_row_after_row():
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    E, K, N, R = 2, 256, 128, 384
    offsets = torch.tensor([0, 128, R], dtype=torch.int32, device="cuda")
    x, dy = (torch.randn(R, h, generator=g, device="cuda").to(torch.bfloat16) for h in (K, N))
    rows = nq.ep_nvfp4_pack_weights(x.unsqueeze(0))[0]
    w = nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(torch.randn(E, N, K, generator=g, device="cuda").to(torch.bfloat16)), K)
    amax = torch.full((E,), 5.0, device="cuda")
    receive = lambda **kw: nq.ep_nvfp4_direct_receive(rows, K, offsets, E, **kw)             # noqa: E731
    columns = lambda t, **kw: nq.ep_nvfp4_colwise_rht_bf16(t, offsets, E, amax, **kw)        # noqa: E731
    gemm = lambda x: nq.ep_nvfp4_grouped_gemm(x, w, offsets)                                 # noqa: E731
    wgrad = lambda dy, x: nq.ep_nvfp4_grouped_wgrad(dy, x, N, K, offsets, E)                 # noqa: E731
    tiled, flat = receive(swizzled=True), receive()
    dyt, dyf = columns(dy, swizzled=True), columns(dy)
    y, d_w = gemm(tiled), wgrad(dyt, tiled)
    for bad in (lambda: gemm(flat), lambda: gemm(dict(flat)), lambda: wgrad(dyt, flat), lambda: wgrad(dyf, tiled),
                lambda: wgrad(dyt, columns(x))):
        with pytest.raises(ValueError, match="swizzled=True"):
            bad()
    # buffers that are used again: what counts is what the last call wrote
    receive(out=flat, swizzled=True)
    columns(dy, out=dyf, swizzled=True)
    assert torch.equal(gemm(flat), y) and torch.equal(wgrad(dyf, flat), d_w)
    receive(out=flat)
    with pytest.raises(ValueError, match="swizzled=True"):
        gemm(flat)
    # a tensor of the caller's own carries no note
    own = dict(tiled, rw_scales=tiled["rw_scales"].clone(), cw_scales=tiled["cw_scales"].clone())
    assert torch.equal(gemm(own), y) and torch.equal(wgrad(dyt, own), d_w)
