"""Refusals of the operators around the expert products: the C entries' host
checks (no call here reaches CUDA) and the Python binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_quantization_gb300 as nq

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)   # 8-byte aligned only


def _pack(**kw):
    a = dict(tok=FAKE, dt=0, T=4, H=100, ld=100, dest=FAKE, k=2, off=FAKE, cnt=FAKE, E=4, rows=FAKE, R=600, st=FAKE)
    a.update(kw)
    return nq.lib().ep_pack(a["tok"], a["dt"], a["T"], a["H"], a["ld"], a["dest"], a["k"], a["off"], a["cnt"], a["E"],
                            a["rows"], a["R"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(tok=None), -1), (dict(dest=None), -1), (dict(off=None), -1), (dict(cnt=None), -1), (dict(rows=None), -1),
    (dict(st=None), -1), (dict(T=-1), -2), (dict(H=0, ld=1), -2), (dict(H=(1 << 20) + 1, ld=1 << 21), -2),
    (dict(ld=99), -2), (dict(ld=1 << 31), -2), (dict(k=0), -2), (dict(k=33), -2), (dict(E=0), -2), (dict(E=1025), -2),
    (dict(R=-1), -4), (dict(R=1 << 31), -4), (dict(dt=2), -5), (dict(tok=ODD), -3), (dict(rows=ODD), -3),
    (dict(dt=1, tok=ctypes.c_void_p(0x10002)), -3)])
def test_pack_refusals(kw, status):
    assert _pack(**kw) == status


def _back(**kw):
    a = dict(d=FAKE, dt=0, T=4, H=100, ld=100, rows=FAKE, ldr=100, dest=FAKE, w=FAKE, k=2, off=FAKE, cnt=FAKE, E=4,
             dr=FAKE, R=600, dw=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_combine_backward(a["d"], a["dt"], a["T"], a["H"], a["ld"], a["rows"], a["ldr"], a["dest"],
                                        a["w"], a["k"], a["off"], a["cnt"], a["E"], a["dr"], a["R"], a["dw"], a["st"],
                                        None)


@pytest.mark.parametrize("kw, status", [
    (dict(d=None), -1), (dict(rows=None), -1), (dict(dr=None), -1), (dict(st=None), -1), (dict(ldr=99), -2),
    (dict(ld=99), -2), (dict(k=33), -2), (dict(R=-1), -4), (dict(dt=7), -5), (dict(w=ctypes.c_void_p(0x10002)), -3),
    (dict(dw=ctypes.c_void_p(0x10002)), -3), (dict(rows=ODD), -3)])
def test_combine_backward_refusals(kw, status):
    assert _back(**kw) == status


def _combine(**kw):
    a = dict(rows=FAKE, dt=0, R=600, H=100, ld=100, ix=FAKE, so=0, w=FAKE, T=4, k=2, out=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_combine(a["rows"], a["dt"], a["R"], a["H"], a["ld"], a["ix"], a["so"], a["w"], a["T"], a["k"],
                               a["out"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(rows=None), -1), (dict(ix=None), -1), (dict(out=None), -1), (dict(st=None), -1), (dict(H=0, ld=1), -2),
    (dict(ld=99), -2), (dict(k=0), -2), (dict(T=-1), -2), (dict(so=1, R=7), -4), (dict(R=-1), -4), (dict(dt=-1), -5),
    (dict(out=ODD), -3), (dict(w=ctypes.c_void_p(0x10002)), -3)])
def test_combine_refusals(kw, status):
    assert _combine(**kw) == status


def _swiglu(**kw):
    a = dict(x=FAKE, ld=128, R=256, I=64, off=FAKE, E=4, act=FAKE, ck=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_swiglu(a["x"], a["ld"], a["R"], a["I"], a["off"], a["E"], a["act"], a["ck"], a["st"], None)


def _swiglu_back(**kw):
    a = dict(d=FAKE, ld=64, ck=FAKE, R=256, I=64, off=FAKE, E=4, dx=FAKE, act=FAKE, am=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_swiglu_backward(a["d"], a["ld"], a["ck"], a["R"], a["I"], a["off"], a["E"], a["dx"], a["act"],
                                       a["am"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), -1), (dict(act=None), -1), (dict(st=None), -1), (dict(I=48), -2), (dict(I=0), -2), (dict(ld=127), -2),
    (dict(E=0), -2), (dict(E=1025), -2), (dict(off=None), -2), (dict(R=-1), -4), (dict(x=HALF), -3),
    (dict(ld=130), -3), (dict(ck=HALF), -3), (dict(act=HALF), -3)])
def test_swiglu_refusals(kw, status):
    assert _swiglu(**kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(d=None), -1), (dict(ck=None), -1), (dict(dx=None), -1), (dict(st=None), -1), (dict(I=48), -2),
    (dict(ld=63), -2), (dict(off=None), -2), (dict(R=-1), -4), (dict(ld=66), -3), (dict(dx=HALF), -3),
    (dict(act=HALF), -3), (dict(am=ctypes.c_void_p(0x10002)), -3)])
def test_swiglu_backward_refusals(kw, status):
    assert _swiglu_back(**kw) == status


def _matvec(**kw):
    a = dict(x=FAKE, T=4, K=64, ld=64, ps=0, w=FAKE, E=4, N=10, tk=FAKE, k=2, y=FAKE, st=FAKE)
    a.update(kw)
    return nq.lib().ep_nvfp4_matvec(a["x"], a["T"], a["K"], a["ld"], a["ps"], a["w"], a["E"], a["N"], a["tk"], a["k"],
                                    a["y"], a["st"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(st=None), -1), (dict(K=48, ld=48), -2), (dict(K=32800, ld=32800), -2),
    (dict(ld=56), -2), (dict(N=0), -2), (dict(N=(1 << 20) + 1), -2), (dict(tk=None), -2), (dict(tk=None, E=1), -2),
    (dict(E=0), -2), (dict(k=33), -2), (dict(T=-1), -2), (dict(T=(1 << 19) + 1), -4), (dict(x=HALF), -3), (dict(w=HALF), -3), (dict(ld=66), -3),
    (dict(y=ODD), -3)])
def test_matvec_refusals(kw, status):
    assert _matvec(**kw) == status


def test_host_memory_is_refused_with_ep_err_device():
    buf = np.zeros(1 << 16, np.int32)
    at = (buf.ctypes.data + 15) // 16 * 16
    h = ctypes.c_void_p(at)
    assert _pack(tok=h, dest=h, off=h, cnt=h, rows=h, st=h) == -6
    assert _back(d=h, rows=h, dest=h, w=h, off=h, cnt=h, dr=h, dw=h, st=h) == -6
    assert _combine(rows=h, ix=h, w=h, out=h, st=h) == -6
    assert _swiglu(x=h, off=h, act=h, ck=h, st=h) == -6
    assert _swiglu_back(d=h, ck=h, off=h, dx=h, act=h, am=h, st=h) == -6
    assert _matvec(x=h, w=h, tk=h, y=h, st=h) == -6
    assert buf.sum() == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    z = lambda n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    plan = nq.RoutePlan(z(5), z(4), z(16), 8, 2, 4, 128, 1024, z(1))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_pack(bf(8, 64), plan)
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_combine(bf(1024, 64), plan)
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_combine_backward(bf(8, 64), plan)
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_swiglu(bf(8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_swiglu_backward(bf(8, 64), torch.zeros(10, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_nvfp4_matvec(bf(1, 64), torch.zeros((1, 4, nq.row_bytes(64)), dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        nq.ep_nvfp4_pack_weights(bf(1, 4, 64))


def test_checkpoint_bytes_follow_the_mxfp8_layout():
    assert nq.swiglu_checkpoint_bytes(0, 64) == 0
    assert nq.swiglu_checkpoint_bytes(256, 96) == 256 * 192 + 256 * 6
