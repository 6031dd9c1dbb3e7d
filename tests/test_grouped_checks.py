"""Refusals of the grouped products: the C entries' host checks (no call here
reaches CUDA) and the Python binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_quantization_gb300 as nq

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
HALF = ctypes.c_void_p(0x10008)   # 8-byte aligned only
ODD = ctypes.c_void_p(0x10002)


def _gemm(**kw):
    a = dict(x=FAKE, R=600, K=64, ld=64, w=FAKE, E=4, N=40, tr=0, off=FAKE, out=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_grouped_gemm(a["x"], a["R"], a["K"], a["ld"], a["w"], a["E"], a["N"], a["tr"], a["off"],
                                    a["out"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(st=None), -1), (dict(off=None), -2),
    (dict(K=60, ld=64), -2), (dict(K=0, ld=8), -2), (dict(N=41), -2), (dict(N=0), -2), (dict(N=(1 << 20) + 8), -2),
    (dict(K=(1 << 20) + 8, ld=1 << 21), -2), (dict(ld=56), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(R=-1), -4),
    (dict(R=1 << 31), -4), (dict(R=(1 << 31) - 1, N=1 << 20), -4), (dict(x=HALF), -3), (dict(ld=68), -3),
    (dict(w=HALF), -3), (dict(out=HALF), -3)])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


def _wgrad(**kw):
    a = dict(dy=FAKE, ldy=40, x=FAKE, ldx=64, R=600, N=40, K=64, off=FAKE, cnt=FAKE, E=4, dw=FAKE, dt=1, acc=0, st=FAKE)
    a.update(kw)
    return nq.lib().ep_grouped_wgrad(a["dy"], a["ldy"], a["x"], a["ldx"], a["R"], a["N"], a["K"], a["off"], a["cnt"],
                                     a["E"], a["dw"], a["dt"], a["acc"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(dy=None), -1), (dict(x=None), -1), (dict(dw=None), -1), (dict(st=None), -1), (dict(off=None), -2),
    (dict(N=36), -2), (dict(K=4), -2), (dict(ldy=32), -2), (dict(ldx=56), -2), (dict(E=0), -2), (dict(E=1025), -2),
    (dict(R=-1), -4), (dict(R=1 << 31), -4), (dict(E=1024, N=1 << 20, K=1 << 20, ldy=1 << 20, ldx=1 << 20), -4),
    (dict(dt=2), -5), (dict(dt=0, acc=1), -5), (dict(dy=HALF), -3), (dict(x=HALF), -3), (dict(ldy=44), -3),
    (dict(ldx=68), -3), (dict(dw=HALF), -3), (dict(cnt=ODD), -3)])
def test_wgrad_refusals(kw, status):
    assert _wgrad(**kw) == status


def _operand(**kw):
    a = dict(rows=FAKE, g=1, n=600, H=64, off=FAKE, E=4, sc=FAKE, rs=FAKE, co=None, st=FAKE)
    a.update(kw)
    return nq.lib().ep_nvfp4_operand(a["rows"], a["g"], a["n"], a["H"], a["off"], a["E"], a["sc"], a["rs"], a["co"],
                                     a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(rows=None), -1), (dict(sc=None), -1), (dict(rs=None), -1), (dict(st=None), -1), (dict(H=48), -2),
    (dict(H=0), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(off=None), -2), (dict(g=2), -2),
    (dict(n=-1), -4), (dict(n=1 << 31), -4), (dict(g=4, n=1 << 30, off=None, E=1), -4), (dict(rows=HALF), -3),
    (dict(sc=HALF), -3), (dict(rs=ODD), -3), (dict(co=HALF), -3)])
def test_operand_refusals(kw, status):
    assert _operand(**kw) == status


def _ngemm(**kw):
    a = dict(x=FAKE, ldx=32, xs=FAKE, xr=FAKE, R=600, K=64, w=FAKE, ldw=32, ws=FAKE, wr=FAKE, E=4, N=40, off=FAKE,
             out=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_nvfp4_grouped_gemm(a["x"], a["ldx"], a["xs"], a["xr"], a["R"], a["K"], a["w"], a["ldw"],
                                          a["ws"], a["wr"], a["E"], a["N"], a["off"], a["out"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), -1), (dict(xs=None), -1), (dict(xr=None), -1), (dict(w=None), -1), (dict(ws=None), -1),
    (dict(wr=None), -1), (dict(out=None), -1), (dict(st=None), -1), (dict(K=48), -2), (dict(N=41), -2),
    (dict(ldx=16), -2), (dict(ldw=16), -2), (dict(off=None), -2), (dict(E=1025), -2), (dict(R=-1), -4),
    (dict(R=1 << 31), -4), (dict(x=HALF), -3), (dict(ldx=40), -3), (dict(xs=HALF), -3), (dict(xr=ODD), -3),
    (dict(w=HALF), -3), (dict(ldw=40), -3), (dict(ws=HALF), -3), (dict(wr=ODD), -3), (dict(out=HALF), -3)])
def test_nvfp4_gemm_refusals(kw, status):
    assert _ngemm(**kw) == status


def _nwgrad(**kw):
    a = dict(y=FAKE, ys=FAKE, ye=FAKE, x=FAKE, xs=FAKE, xe=FAKE, R=640, N=128, K=256, off=FAKE, E=4,
             dw=FAKE, dt=1, acc=0, st=FAKE)
    a.update(kw)
    return nq.lib().ep_nvfp4_grouped_wgrad(a["y"], a["ys"], a["ye"], a["x"], a["xs"], a["xe"], a["R"], a["N"], a["K"],
                                           a["off"], a["E"], a["dw"], a["dt"], a["acc"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(y=None), -1), (dict(ys=None), -1), (dict(ye=None), -1), (dict(x=None), -1), (dict(xs=None), -1),
    (dict(xe=None), -1), (dict(dw=None), -1), (dict(st=None), -1), (dict(N=64), -2),
    (dict(K=192), -2), (dict(off=None), -2), (dict(off=None, E=1, R=600), -2), (dict(E=1025), -2),
    (dict(R=-1), -4), (dict(dt=3), -5), (dict(dt=0, acc=1), -5), (dict(y=HALF), -3),
    (dict(ys=HALF), -3), (dict(ye=ODD), -3), (dict(x=HALF), -3), (dict(xs=HALF), -3), (dict(xe=ODD), -3),
    (dict(dw=HALF), -3)])
def test_nvfp4_wgrad_refusals(kw, status):
    assert _nwgrad(**kw) == status


def test_colwise_in_tiles_refuses_partial_tiles():
    f = nq.lib().ep_nvfp4_colwise_rht_bf16_swizzled
    assert f(FAKE, 256, 96, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 0, FAKE, None) == -2
    assert f(None, 256, 128, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 0, FAKE, None) == -1


def test_host_memory_is_refused_with_ep_err_device():
    buf = np.zeros(1 << 16, np.int32)
    h = ctypes.c_void_p((buf.ctypes.data + 127) // 128 * 128)
    assert _gemm(x=h, w=h, off=h, out=h, st=h) == -6
    assert _wgrad(dy=h, x=h, off=h, cnt=h, dw=h, st=h) == -6
    assert _operand(rows=h, off=h, sc=h, rs=h, st=h) == -6
    assert _ngemm(x=h, xs=h, xr=h, w=h, ws=h, wr=h, off=h, out=h, st=h) == -6
    assert _nwgrad(y=h, ys=h, ye=h, x=h, xs=h, xe=h, off=h, dw=h, st=h) == -6
    assert buf.sum() == 0


def test_sizes():
    L = nq.lib()
    for rows, H in ((0, 64), (1, 32), (128, 64), (129, 96), (1000, 7168)):
        assert L.ep_nvfp4_scale_bytes(rows, H) == nq.nvfp4_scale_bytes(rows, H) == -(-rows // 128) * -(-H // 64) * 512


def test_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)      # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_grouped_gemm(bf(8, 64), bf(1, 16, 64))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_grouped_wgrad(bf(8, 64), bf(8, 16))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_nvfp4_operand(u8(8, nq.row_bytes(64)), 64)
    op = dict(rw_codes=u8(8, 32), rw_scales=u8(512), rw_row_scale=torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_nvfp4_grouped_gemm(op, op)
    cw = dict(cw_codes=u8(128 * 64), cw_scales=u8(128 * 8), cw_scale_enc=torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_nvfp4_grouped_wgrad(cw, cw, 128, 128)
