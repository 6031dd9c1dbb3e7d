"""The operators around the expert products against their definitions in 64
bits.

Error bounds (u = 2^-24, half an FP32 ulp; b = 2^-8, half a BF16 ulp):
rounding once to the output type costs b|y| (BF16) or u|y| (FP32); a sum of n
terms in any order with rounding or truncating additions costs at most
2 n u sum|terms|; expf, the sum 1 + e and __fdividef are within 2, 1/2 and 2
ulps, so s = 1/(1+exp(-g)) and the products behind it stay within 32 u
relative, and 1 - s within 32 u absolute.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_gb300 as nq
import oracle

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def ulp(dtype):
    return B if dtype == torch.bfloat16 else U


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def route(T, k, E, g, drop=0.0):
    topk = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1)[1] if T else torch.empty(0, k, device="cuda")
    topk = topk.to(torch.int32)
    if drop and T:
        topk[torch.rand(T, k, generator=g, device="cuda") < drop] = -1
        topk[T // 2] = -1      # a token without any expert
    return topk.contiguous()


def dest_of(plan):
    return plan.dest[: plan.T * plan.k].view(plan.T, plan.k).long()


def within(got, want, bound):
    """|got - want| <= bound, element by element, in 64 bits."""
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (int(bad.sum()), d[bad].max().item(), bound.expand_as(d)[bad].min().item())


def strided(t, extra):
    """The same values with a row pitch `extra` elements wider (None: as it is)."""
    if extra is None:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


SHAPES = [  # T, k, E, H, type, dropped share, extra row pitch
    (1, 1, 1, 1, "bf16", 0.0, None), (1, 8, 16, 7168, "bf16", 0.0, None), (0, 2, 4, 64, "bf16", 0.0, None),
    (130, 2, 4, 1024, "bf16", 0.3, None), (257, 3, 7, 1001, "bf16", 0.2, None), (64, 5, 9, 333, "f32", 0.2, None),
    (300, 8, 64, 4096, "f32", 0.0, None), (90, 11, 40, 258, "bf16", 0.3, None), (33, 32, 48, 96, "bf16", 0.1, 8),
    (50, 4, 8, 128, "bf16", 0.1, 3), (77, 2, 3, 100, "f32", 0.1, 1), (1000, 6, 300, 2056, "bf16", 0.05, None),
    (40, 9, 16, 8200, "f32", 0.0, 4), (5, 2, 1024, 34, "bf16", 0.0, 2)]


@pytest.mark.parametrize("T,k,E,H,dt,drop,extra", SHAPES)
def test_pack(T, k, E, H, dt, drop, extra):
    g = gen(1)
    topk = route(T, k, E, g, drop)
    plan = nq.ep_route_plan(topk, E)
    tok = torch.randn(T, H, generator=g, device="cuda").to(TYPES[dt])
    rows = torch.full((plan.R_cap, H), 7.0, dtype=TYPES[dt], device="cuda")
    assert nq.ep_pack(strided(tok, extra), plan, rows=rows) is rows
    want = torch.full_like(rows, 7.0)
    want[: int(plan.offsets[-1])] = 0
    d = dest_of(plan)
    for j in range(k):
        live = d[:, j] >= 0
        want[d[live, j]] = tok[live]
    assert torch.equal(rows, want)
    assert int(plan.status) == 0


def combine64(rows, index, live, weights):
    out = torch.zeros(index.shape[0], rows.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for j in range(index.shape[1]):
        t = live[:, j].nonzero().reshape(-1)
        v = rows[index[t, j]].double()
        if weights is not None:
            v = v * weights[t, j].double().unsqueeze(1)
        out[t] += v
        mag[t] += v.abs()
    return out, mag


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,dt,drop,extra", SHAPES)
def test_combine(T, k, E, H, dt, drop, extra, weighted):
    g = gen(2)
    topk = route(T, k, E, g, drop)
    plan = nq.ep_route_plan(topk, E)
    rows = torch.randn(plan.R_cap, H, generator=g, device="cuda").to(TYPES[dt])
    weights = torch.randn(T, k, generator=g, device="cuda") if weighted else None
    d = dest_of(plan)
    live = d >= 0
    if weighted:      # nothing of a dropped slot reaches the sum
        weights[~live] = float("nan")
    pad = torch.ones(plan.R_cap, dtype=torch.bool, device="cuda")
    pad[d[live]] = False
    rows[pad] = float("inf")
    out = torch.full((T, H), 7.0, dtype=TYPES[dt], device="cuda")
    assert nq.ep_combine(strided(rows, extra), plan, weights=weights, out=out) is out
    want, mag = combine64(rows, d, live, weights)
    within(out, want, ulp(out.dtype) * want.abs() * (1 + B) + 2 * k * U * mag + 2.0 ** -133)
    assert int(plan.status) == 0
    # the same sum from rows in slot order
    slots = torch.full((T * k, H), float("nan"), dtype=TYPES[dt], device="cuda")
    slots[live.reshape(-1)] = rows[d[live]]
    out2 = nq.ep_combine(strided(slots, extra), topk_idx=topk, weights=weights)
    assert torch.equal(out2, out)


@pytest.mark.parametrize("T,k,E,H,dt,drop,extra", SHAPES)
def test_combine_backward(T, k, E, H, dt, drop, extra):
    g = gen(3)
    topk = route(T, k, E, g, drop)
    plan = nq.ep_route_plan(topk, E)
    d = dest_of(plan)
    live = d >= 0
    rows = torch.full((plan.R_cap, H), float("nan"), dtype=TYPES[dt], device="cuda")
    rows[d[live]] = torch.randn(int(live.sum()), H, generator=g, device="cuda").to(TYPES[dt])
    weights = torch.randn(T, k, generator=g, device="cuda")
    weights[~live] = float("inf")
    d_out = torch.randn(T, H, generator=g, device="cuda").to(TYPES[dt])
    d_rows = torch.full((plan.R_cap, H), 7.0, dtype=TYPES[dt], device="cuda")
    d_w = torch.full((T, k), 7.0, device="cuda")
    nq.ep_combine_backward(strided(d_out, extra), plan, weights=weights, rows=strided(rows, extra), d_rows=d_rows,
                           d_weights=d_w)
    R = int(plan.offsets[-1])
    want = torch.zeros(plan.R_cap, H, dtype=torch.float64, device="cuda")
    want[R:] = 7.0
    want_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    mag_w = torch.zeros_like(want_w)
    for j in range(k):
        t = live[:, j].nonzero().reshape(-1)
        want[d[t, j]] = d_out[t].double() * weights[t, j].double().unsqueeze(1)
        p = d_out[t].double() * rows[d[t, j]].double()
        want_w[t, j], mag_w[t, j] = p.sum(1), p.abs().sum(1)
    within(d_rows, want, (ulp(d_rows.dtype) + 2 * U) * want.abs() + 2.0 ** -133)
    within(d_w, want_w, 2 * H * U * mag_w)
    assert int(plan.status) == 0
    # the weights' gradient does not depend on the weights
    again, d_w2 = nq.ep_combine_backward(d_out, plan, rows=rows, d_rows=torch.full_like(d_rows, 7.0))
    assert torch.equal(d_w2, d_w)
    # without weights, without the weights' gradient
    ones, none = nq.ep_combine_backward(d_out, plan, d_rows=torch.full_like(d_rows, 7.0))
    assert none is None
    assert torch.equal(ones, nq.ep_pack(d_out, plan, rows=torch.full_like(d_rows, 7.0)))
    assert torch.equal(again, ones)


def inside(rows, cols, dtype, offset, fill):
    """A contiguous [rows, cols] view that starts `offset` elements into a buffer
    of canaries, and that buffer."""
    buf = torch.full((offset + rows * cols + 64,), fill, dtype=dtype, device="cuda")
    return buf[offset: offset + rows * cols].view(rows, cols), buf


@pytest.mark.parametrize("offset", [0, 1, 3, 5])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 7, 8, 9, 24, 331, 1000, 4099])
def test_rows_that_start_anywhere(H, dt, offset):
    """Buffers at every alignment of an element: the values, and nothing written
    beside the outputs."""
    dtype, g = TYPES[dt], gen(20 + offset)
    T, k, E = 21, 3, 5
    topk = route(T, k, E, g, 0.2)
    plan = nq.ep_route_plan(topk, E)
    d = dest_of(plan)
    live = d >= 0
    R = int(plan.offsets[-1])
    tok = inside(T, H, dtype, offset, 9.0)[0]
    tok.copy_(torch.randn(T, H, generator=g, device="cuda"))
    rows, buf = inside(plan.R_cap, H, dtype, (offset * 3) % 8, 7.0)
    nq.ep_pack(tok, plan, rows=rows)
    want = torch.full_like(rows, 7.0)
    want[:R] = 0
    for j in range(k):
        want[d[live[:, j], j]] = tok[live[:, j]]
    assert torch.equal(rows, want)
    first = (offset * 3) % 8
    assert (buf[:first] == 7.0).all() and (buf[first + rows.numel():] == 7.0).all()
    rows[:R] = torch.randn(R, H, generator=g, device="cuda").to(dtype)
    weights = torch.randn(T, k, generator=g, device="cuda")
    out, buf = inside(T, H, dtype, (offset * 5) % 8, 7.0)
    nq.ep_combine(rows, plan, weights, out=out)
    sums, mag = combine64(rows, d, live, weights)
    within(out, sums, ulp(dtype) * sums.abs() * (1 + B) + 2 * k * U * mag + 2.0 ** -133)
    first = (offset * 5) % 8
    assert (buf[:first] == 7.0).all() and (buf[first + out.numel():] == 7.0).all()
    d_rows, buf = inside(plan.R_cap, H, dtype, (offset * 7) % 8, 7.0)
    _, d_w = nq.ep_combine_backward(tok, plan, weights, rows=rows, d_rows=d_rows)
    first = (offset * 7) % 8
    assert (buf[:first] == 7.0).all() and (buf[first + d_rows.numel():] == 7.0).all()
    assert (d_rows[R:] == 7.0).all()
    for j in range(k):
        t = live[:, j].nonzero().reshape(-1)
        v = tok[t].double() * weights[t, j].double().unsqueeze(1)
        within(d_rows[d[t, j]], v, (ulp(dtype) + 2 * U) * v.abs() + 2.0 ** -133)
        p = tok[t].double() * rows[d[t, j]].double()
        within(d_w[t, j], p.sum(1), 2 * H * U * p.abs().sum(1))
    assert not d_w[~live].any()


def test_combine_gradient_against_differences():
    """Central differences of L = <v, combine(rows, w)> in 64 bits along random
    directions; L is bilinear, so only the gradients' own rounding is left."""
    g = gen(4)
    T, k, E, H = 37, 3, 5, 130
    topk = route(T, k, E, g, 0.2)
    plan = nq.ep_route_plan(topk, E)
    d, live = dest_of(plan), dest_of(plan) >= 0
    rows = torch.randn(plan.R_cap, H, generator=g, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    v = torch.randn(T, H, generator=g, device="cuda")
    d_rows, d_w = nq.ep_combine_backward(v, plan, weights=w, rows=rows)
    d_rows = d_rows[: int(plan.offsets[-1])].double()
    loss = lambda r, q: (combine64(r, d, live, q)[0] * v.double()).sum()   # noqa: E731
    for i in range(4):
        dr = torch.randn(rows.shape, generator=g, device="cuda").double()
        dw = torch.randn(w.shape, generator=g, device="cuda").double()
        h = 2.0 ** -10
        num = (loss(rows.double() + h * dr, w.double() + h * dw) - loss(rows.double() - h * dr, w.double() - h * dw)) / (2 * h)
        dr = dr[: d_rows.shape[0]]
        ana = (d_rows * dr).sum() + (d_w.double() * dw).sum()
        size = (d_rows * dr).abs().sum() + (d_w.double() * dw).abs().sum() * H
        assert abs(num - ana) <= 2 * H * U * size + 1e-9 * abs(num)


def test_rows_outside_the_buffer_are_reported_and_skipped():
    T, k, E, H = 4, 2, 2, 64
    topk = torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda")
    plan = nq.ep_route_plan(topk, E)
    plan.dest[3] = plan.R_cap
    plan.dest[6] = 2 ** 31 - 1
    tok = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    rows = nq.ep_pack(tok, plan)
    assert int(plan.status) == nq.EP_DEV_ERR_CAPACITY
    plan.status.zero_()
    out = nq.ep_combine(rows, plan)
    assert int(plan.status) == nq.EP_DEV_ERR_CAPACITY
    assert out[:, 0].tolist() == [2.0, 1.0, 2.0, 1.0]
    plan.status.zero_()
    _, d_w = nq.ep_combine_backward(tok, plan, rows=rows)
    assert int(plan.status) == nq.EP_DEV_ERR_CAPACITY
    assert d_w.reshape(-1).tolist() == [64.0, 64.0, 64.0, 0.0, 64.0, 64.0, 0.0, 64.0]


def test_rows_past_32_bit_offsets():
    """Rows whose element offset passes 2^32."""
    T, k, E, H = 2, 1, 1, 1 << 20
    R_cap = 4200
    topk = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    plan = nq.ep_route_plan(topk, E, R_cap=R_cap)
    plan.offsets.fill_(0)
    plan.counts.fill_(0)
    plan.dest.copy_(torch.tensor([4199, 4098], device="cuda"))
    g = gen(5)
    tok = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.empty(R_cap, H, dtype=torch.bfloat16, device="cuda")
    rows[:16] = 0
    nq.ep_pack(tok, plan, rows=rows)
    assert torch.equal(rows[4199], tok[0]) and torch.equal(rows[4098], tok[1])
    assert not rows[:16].any()
    assert torch.equal(nq.ep_combine(rows, plan), tok)
    _, d_w = nq.ep_combine_backward(tok, plan, rows=rows, d_rows=torch.empty_like(rows))
    sq = (tok.double() ** 2).sum(1, keepdim=True)
    within(d_w, sq, 2 * H * U * sq)


# ---------------------------------------------------------------- activation
def swiglu64(g, u, d):
    s = 1 / (1 + torch.exp(-g))
    return g * s * u, d * u * s * (1 + g * (1 - s)), d * g * s, s


def decode_ckpt(ckpt, R_cap, I):
    data = ckpt[: R_cap * 2 * I].view(torch.float8_e4m3fn).float().double().view(R_cap, 2 * I // 32, 32)
    scale = torch.exp2(ckpt[R_cap * 2 * I:].double() - 127).view(R_cap, 2 * I // 32, 1)
    return (data * scale).view(R_cap, 2 * I)


ACT = [  # tokens, k, E, I, extra row pitch; k = 0: no plan, all rows
    (1, 0, 1, 32, None), (3, 0, 1, 96, 8), (200, 2, 8, 512, None), (65, 3, 5, 160, 16), (700, 1, 3, 2048, None),
    (20, 8, 64, 4096, None), (0, 2, 4, 64, None), (0, 0, 1, 64, None), (9, 0, 1, 1440, 24)]


@pytest.mark.parametrize("T,k,E,I,extra", ACT)
def test_swiglu_and_its_gradient(T, k, E, I, extra):
    g = gen(6)
    if k:
        plan = nq.ep_route_plan(route(T, k, E, g), E)
        off, R_cap = plan.offsets, plan.R_cap
        R = int(off[-1])
    else:
        off, R_cap, R = None, T, T
    x = torch.randn(R_cap, 2 * I, generator=g, device="cuda") * torch.exp(torch.randn(R_cap, 1, generator=g, device="cuda"))
    x[:, ::37] *= 50
    x[:, I // 2: I // 2 + 32] = 0
    x = x.to(torch.bfloat16)
    d = torch.randn(R_cap, I, generator=g, device="cuda").to(torch.bfloat16)
    act = torch.full((R_cap, I), 7.0, dtype=torch.bfloat16, device="cuda")
    ckpt = torch.full((nq.swiglu_checkpoint_bytes(R_cap, I),), 0xAB, dtype=torch.uint8, device="cuda")
    status = nq.new_status("cuda")
    nq.ep_swiglu(strided(x, extra), off, E, act=act, ckpt=ckpt, status=status)
    X = x[:R].double()
    want, _, _, s = swiglu64(X[:, :I], X[:, I:], 0)
    within(act[:R], want, (B + 64 * U) * want.abs() + 1e-33)
    assert (act[R:] == 7.0).all()
    alone, none = nq.ep_swiglu(strided(x, extra), off, E, act=torch.full_like(act, 7.0), checkpoint=False)
    assert none is None and torch.equal(alone, act)
    # the checkpoint is the MXFP8 pack of the rows, byte for byte
    if R:
        ident = np.arange(R, dtype=np.int32)
        want8 = oracle.mxfp8_pack(x[:R].view(torch.int16).cpu().numpy().view(np.uint16), ident, 1,
                                  np.array([0, R], np.int32), np.array([R], np.int32), 1, R)
        got8 = ckpt.cpu().numpy()
        assert np.array_equal(got8[: R * 2 * I], want8[: R * 2 * I])
        assert np.array_equal(got8[R_cap * 2 * I:][: R * I // 16], want8[R * 2 * I:])
    assert (ckpt[R * 2 * I: R_cap * 2 * I] == 0xAB).all() and (ckpt[R_cap * 2 * I + R * I // 16:] == 0xAB).all()

    d_x = torch.full((R_cap, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    again = torch.full_like(act, 7.0)
    amax = torch.zeros(E, device="cuda")
    nq.ep_swiglu_backward(strided(d, extra), ckpt, off, E, d_x=d_x, act=again, expert_amax=amax, status=status)
    K = decode_ckpt(ckpt, R_cap, I)[:R]
    gg, uu, D = K[:, :I], K[:, I:], d[:R].double()
    a64, dg, du, s = swiglu64(gg, uu, D)
    within(again[:R], a64, (B + 64 * U) * a64.abs() + 1e-33)
    e_dg = (D * uu).abs() * s * (1 + gg.abs()) * 96 * U + 1e-33
    e_du = 64 * U * du.abs() + 1e-33
    within(d_x[:R, :I], dg, B * dg.abs() * (1 + B) + 2 * e_dg)
    within(d_x[:R, I:], du, B * du.abs() * (1 + B) + 2 * e_du)
    assert (d_x[R:] == 7.0).all() and (again[R:] == 7.0).all()
    bounds = off.tolist() if off is not None else [0, R]
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            assert amax[e] == 0
            continue
        top = torch.maximum(dg[a:b].abs().max(), du[a:b].abs().max())
        tol = torch.maximum(e_dg[a:b].max(), e_du[a:b].max())
        assert abs(amax[e].double() - top) <= tol, e
    # the amax is optional, and so is the activation
    d_x2, none = nq.ep_swiglu_backward(d, ckpt, off, E, d_x=torch.full_like(d_x, 7.0))
    assert none is None and torch.equal(d_x2, d_x)
    assert int(status) == 0


def test_swiglu_gradient_against_differences():
    """Central differences of act at values the checkpoint holds exactly."""
    I, n = 64, 40
    g = gen(7)
    x = (torch.randint(-28, 29, (n, 2 * I), generator=g, device="cuda").float() / 8).to(torch.bfloat16)
    x[:, ::32] = 3.5       # every block's largest element: scale 2^-7, grid step 1/8 near the top
    x = (x.float().sign() * torch.exp2(torch.round(torch.log2(x.float().abs().clamp_min(2.0 ** -4))))).to(torch.bfloat16)
    _, ckpt = nq.ep_swiglu(x)
    assert torch.equal(decode_ckpt(ckpt, n, I), x.double())
    d = torch.ones(n, I, dtype=torch.bfloat16, device="cuda")
    d_x, _ = nq.ep_swiglu_backward(d, ckpt)
    f = lambda a, b: a / (1 + torch.exp(-a)) * b   # noqa: E731
    gg, uu, h = x[:, :I].double(), x[:, I:].double(), 1e-5
    num_g = (f(gg + h, uu) - f(gg - h, uu)) / (2 * h)
    num_u = (f(gg, uu + h) - f(gg, uu - h)) / (2 * h)
    tol = 1e-8 + 256 * U * (1 + gg.abs()) * (1 + uu.abs())
    within(d_x[:, :I], num_g, B * num_g.abs() * (1 + B) + tol)
    within(d_x[:, I:], num_u, B * num_u.abs() * (1 + B) + tol)


def test_swiglu_extremes():
    """Gates far out in both directions, and infinities and NaN: they stay
    where they are and do not pass for numbers."""
    I = 64
    x = torch.ones(4, 2 * I, dtype=torch.bfloat16, device="cuda")
    x[0, :6] = torch.tensor([-1e30, -200.0, -90.0, 90.0, 1e30, 0.0])
    x[1, 3], x[1, 40], x[2, I + 5] = float("inf"), float("nan"), float("-inf")
    act, ckpt = nq.ep_swiglu(x)
    assert act[0, :6].tolist()[:2] == [0.0, 0.0] and abs(act[0, 2].item()) < 1e-35
    assert act[0, 3:6].tolist() == [90.0, torch.tensor(1e30).to(torch.bfloat16).item(), 0.0]
    kept = decode_ckpt(ckpt, 4, I)
    bad = torch.zeros_like(kept, dtype=torch.bool)
    bad[1, 3] = bad[1, 40] = bad[2, I + 5] = True
    assert torch.equal(kept.isnan(), bad)
    assert (kept[1:][~bad[1:]] == 1.0).all()
    d = torch.ones(4, I, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 1, 3, 4], dtype=torch.int32, device="cuda")
    amax = torch.zeros(3, device="cuda")
    d_x, _ = nq.ep_swiglu_backward(d, ckpt, off, 3, expert_amax=amax)
    touched = torch.zeros_like(bad)
    for r, c in ((1, 3), (1, 40), (2, 5)):
        touched[r, c] = touched[r, c + I] = True
    touched[2, I + 5] = False          # du does not depend on u
    assert torch.equal(d_x.isnan(), touched)
    assert not amax[0].isnan() and amax[1].isnan() and amax[2] > 0
    # the reduction starts from what the caller put there
    amax.fill_(1e30)
    nq.ep_swiglu_backward(d, ckpt, off, 3, expert_amax=amax)
    assert amax[2] == torch.tensor(1e30)


@pytest.mark.parametrize("I", [32, 64, 96, 256])
def test_swiglu_experts_of_any_length(I):
    """Experts that begin and end inside a warp's rows, and empty ones."""
    g = gen(30)
    off = torch.tensor([0, 3, 3, 4, 11, 11, 30, 37], dtype=torch.int32, device="cuda")
    E, R_cap = 7, 40
    x = torch.randn(R_cap, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn(R_cap, I, generator=g, device="cuda").to(torch.bfloat16)
    _, ckpt = nq.ep_swiglu(x, off, E)
    amax = torch.zeros(E, device="cuda")
    d_x, _ = nq.ep_swiglu_backward(d, ckpt, off, E, expert_amax=amax)
    o = off.tolist()
    for e in range(E):
        if o[e] == o[e + 1]:
            assert amax[e] == 0
        else:
            assert amax[e].to(torch.bfloat16) == d_x[o[e]: o[e + 1]].abs().max()


def test_swiglu_reports_rows_past_the_buffer():
    x = torch.ones(128, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    status = nq.new_status("cuda")
    act, ckpt = nq.ep_swiglu(x, off, 1, status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY and act[127, 0].item() == pytest.approx(1 / (1 + math.exp(-1)), rel=B)
    status.zero_()
    nq.ep_swiglu_backward(act, ckpt, off, 1, status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY


def test_swiglu_past_32_bit_offsets():
    I, R_cap = 4096, 530000           # 2I * R_cap > 2^32
    x = torch.zeros(R_cap, 2 * I, dtype=torch.bfloat16, device="cuda")
    x[0], x[-1] = 1.0, 2.0
    act, ckpt = nq.ep_swiglu(x)
    assert (act[0] == act[0, 0]).all() and (act[-1] == act[-1, 0]).all()
    assert act[-1, 0].item() == pytest.approx(4 / (1 + math.exp(-2)), rel=B) and not act[1].any()
    del x
    d = torch.zeros_like(act)
    d[-1] = 1.0
    del act
    d_x, _ = nq.ep_swiglu_backward(d, ckpt)
    s = 1 / (1 + math.exp(-2))
    assert d_x[-1, 0].item() == pytest.approx(2 * s * (1 + 2 * (1 - s)), rel=B)
    assert d_x[-1, I].item() == pytest.approx(2 * s, rel=B) and not d_x[0].any()


def test_amax_feeds_the_columnwise_operand():
    """The reduced amax, taken to BF16, is the largest |d_x| of the expert."""
    g = gen(8)
    E, I = 4, 128
    plan = nq.ep_route_plan(route(300, 2, E, g), E)
    x = torch.randn(plan.R_cap, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn(plan.R_cap, I, generator=g, device="cuda").to(torch.bfloat16)
    _, ckpt = nq.ep_swiglu(x, plan.offsets, E)
    amax = torch.zeros(E, device="cuda")
    d_x, _ = nq.ep_swiglu_backward(d, ckpt, plan.offsets, E, expert_amax=amax)
    off = plan.offsets.tolist()
    top = torch.stack([d_x[off[e]: off[e + 1]].float().abs().max() for e in range(E)])
    assert torch.equal(amax.to(torch.bfloat16).float(), top)
    out = nq.ep_nvfp4_colwise_rht_bf16(d_x, plan.offsets, E, amax)
    assert torch.equal(out["amax_row"], top)


# ---------------------------------------------------------------- matvec
def decode_rows(w_rows, K):
    """Packed NVFP4 rows [.., S] -> their values in 64 bits."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    c = w_rows[..., : K // 2].long()
    v = torch.stack([grid[c & 15], grid[c >> 4]], -1).reshape(*w_rows.shape[:-1], K // 16, 16)
    s = w_rows[..., K // 2: 9 * K // 16].contiguous().view(torch.float8_e4m3fn).float().double()
    S = w_rows.shape[-1]
    row = w_rows[..., S - 16: S - 12].contiguous().view(torch.float32).double()
    return (v * s.unsqueeze(-1)).reshape(*w_rows.shape[:-1], K) * row


def matvec_bound(y, mag, K, w, x):
    """One rounding, K truncating additions, and inputs scaled to a 16-bit
    format whose smallest step is 2^-39 of the largest element."""
    return B * y.abs() * (1 + B) + 2 * K * U * mag + K * 2.0 ** -36 * w.abs().max() * x.abs().max() + 2.0 ** -133


def check_matvec(x, w_rows, topk, y):
    E, N, _ = w_rows.shape
    K = x.shape[1]
    T, k = topk.shape
    W = decode_rows(w_rows, K)
    for s, e in enumerate(topk.reshape(-1).tolist()):
        xs = x[s if x.shape[0] == T * k else s // k].double()
        if 0 <= e < E:
            want, mag = W[e] @ xs, W[e].abs() @ xs.abs()
            within(y[s], want, matvec_bound(want, mag, K, W[e], xs))
        else:
            assert not y[s].any(), s


MV = [  # T, k, E, N, K, dropped share, one x row per slot, extra row pitch
    (1, 1, 1, 1, 32, 0, False, None), (1, 2, 8, 257, 1024, 0, False, None), (1, 8, 64, 1000, 4096, 0, False, None),
    (7, 3, 5, 50, 96, 0.3, True, None), (32, 8, 16, 130, 512, 0, True, 8), (3, 4, 4, 64, 7168, 0.2, False, 16),
    (70, 2, 3, 33, 160, 0.1, False, None), (130, 1, 2, 40, 2080, 0, False, None), (0, 2, 4, 16, 64, 0, False, None),
    (300, 8, 40, 17, 64, 0.5, True, None), (16, 32, 1024, 8, 32, 0, False, None), (2, 8, 8, 4099, 352, 0, False, None),
    (9, 1, 2, 20, 19968, 0.1, True, None), (12, 2, 4, 70, 8192, 0, False, None), (5, 2, 4, 33, 8224, 0, True, 8), (3, 2, 3, 21, 32768, 0.2, False, None)]


@pytest.mark.parametrize("T,k,E,N,K,drop,per_slot,extra", MV)
def test_matvec(T, k, E, N, K, drop, per_slot, extra):
    g = gen(9)
    topk = route(T, k, E, g, drop)
    w = (torch.randn(E, N, K, generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
    w[0, 0] = 0
    w_rows = nq.ep_nvfp4_pack_weights(w)
    assert w_rows.shape == (E, N, nq.row_bytes(K))
    rows = T * k if per_slot else T
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(rows, 1, generator=g, device="cuda"))
    x[:, ::13] *= 2.0 ** -20
    x = x.to(torch.bfloat16)
    if rows:
        x[0, 0] = 0
    if per_slot and drop:
        x[(topk < 0).reshape(-1)] = float("nan")     # a dropped slot's input is not used
    status = nq.new_status("cuda")
    y = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert nq.ep_nvfp4_matvec(strided(x, extra), w_rows, topk, y=y, status=status) is y
    check_matvec(x, w_rows, topk, y)
    assert int(status) == 0
    assert torch.equal(nq.ep_nvfp4_matvec(x, w_rows, topk), y)      # a second call, other buffers: the same bits


def test_matvec_dense_matches_one_expert():
    g = gen(10)
    w_rows = nq.ep_nvfp4_pack_weights(torch.randn(1, 300, 640, generator=g, device="cuda").to(torch.bfloat16))
    x = torch.randn(5, 640, generator=g, device="cuda").to(torch.bfloat16)
    y = nq.ep_nvfp4_matvec(x, w_rows)
    topk = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
    check_matvec(x, w_rows, topk, y)
    assert torch.equal(y, nq.ep_nvfp4_matvec(x, w_rows, topk))


def test_matvec_ids():
    """Repeated ids, dropped slots and ids outside [-1, E)."""
    g = gen(11)
    w_rows = nq.ep_nvfp4_pack_weights(torch.randn(3, 40, 128, generator=g, device="cuda").to(torch.bfloat16))
    x = torch.randn(4, 128, generator=g, device="cuda").to(torch.bfloat16)
    status = nq.new_status("cuda")
    topk = torch.tensor([[0, 0, 2], [-1, -1, -1], [1, -1, 1], [2, 2, 2]], dtype=torch.int32, device="cuda")
    check_matvec(x, w_rows, topk, nq.ep_nvfp4_matvec(x, w_rows, topk, status=status))
    assert int(status) == 0
    for t in range(4):       # one token alone: each of its slots is a pass of its own
        check_matvec(x[t: t + 1], w_rows, topk[t: t + 1], nq.ep_nvfp4_matvec(x[t: t + 1], w_rows, topk[t: t + 1]))
    topk[0, 1], topk[3, 2] = 3, -2
    check_matvec(x, w_rows, topk, nq.ep_nvfp4_matvec(x, w_rows, topk, status=status))
    assert int(status) == nq.EP_DEV_ERR_BAD_EXPERT


def test_matvec_every_code_and_scale():
    """All 16 codes under all finite E4M3 scales, on powers of two: exact."""
    K = 32
    S = nq.row_bytes(K)
    n = 254
    w = torch.zeros(1, n, S, dtype=torch.uint8, device="cuda")
    codes = torch.arange(16, dtype=torch.uint8, device="cuda")
    both = torch.cat([codes, codes])
    w[0, :, :16] = both[0::2] | (both[1::2] << 4)
    scale = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8, device="cuda")
    w[0, :, 16], w[0, :, 17] = scale, scale.flip(0)
    w[0, :, S - 16: S - 12] = torch.tensor([0.25], device="cuda").view(torch.uint8)
    W = decode_rows(w, K)[0]
    x = torch.eye(K, device="cuda").to(torch.bfloat16)
    y = nq.ep_nvfp4_matvec(x, w)
    assert torch.equal(y.double(), W.t())
    # and under inputs of very different sizes
    x = torch.diag(torch.exp2(torch.arange(K, device="cuda").float() * 3 - 50)).to(torch.bfloat16)
    assert torch.equal(nq.ep_nvfp4_matvec(x, w).double(), (W * x.double().diag()).t())


def test_matvec_infinities_and_nan_show():
    g = gen(12)
    w = torch.rand(1, 20, 64, generator=g, device="cuda") + 0.5
    w_rows = nq.ep_nvfp4_pack_weights(w.to(torch.bfloat16))
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 5], x[2, 6], x[3, 7] = float("inf"), float("nan"), float("-inf")
    y = nq.ep_nvfp4_matvec(x, w_rows)
    assert y[0].isfinite().all()
    assert (y[1] == float("inf")).all() and y[2].isnan().all() and (y[3] == float("-inf")).all()


def test_matvec_past_32_bit_offsets():
    K, N, E = 7168, 8192, 130          # E * N * S > 2^32
    S = nq.row_bytes(K)
    assert E * N * S > 1 << 32
    g = gen(13)
    w_rows = torch.zeros(E, N, S, dtype=torch.uint8, device="cuda")
    last = nq.ep_nvfp4_pack_weights((torch.randn(1, 64, K, generator=g, device="cuda") / 64).to(torch.bfloat16))
    w_rows[E - 1, N - 64:] = last[0]
    x = torch.randn(1, K, generator=g, device="cuda").to(torch.bfloat16)
    topk = torch.tensor([[E - 1, 0]], dtype=torch.int32, device="cuda")
    y = nq.ep_nvfp4_matvec(x, w_rows, topk)
    want = nq.ep_nvfp4_matvec(x, last)
    assert torch.equal(y[0, N - 64:], want[0]) and not y[0, : N - 64].any() and not y[1].any()


# ---------------------------------------------------------------- streams, graphs, refusals
def layer(x, topk, weights, w1, w2, stream=None):
    """One decode step of a MoE layer."""
    h = nq.ep_nvfp4_matvec(x, w1, topk, stream=stream)
    a, _ = nq.ep_swiglu(h, checkpoint=False, stream=stream)
    y = nq.ep_nvfp4_matvec(a, w2, topk, stream=stream)
    return nq.ep_combine(y, topk_idx=topk, weights=weights, stream=stream)


def test_decode_layer_on_another_stream_and_in_a_graph():
    g = gen(14)
    E, k, H, I, T = 8, 2, 256, 128, 3
    w1 = nq.ep_nvfp4_pack_weights((torch.randn(E, 2 * I, H, generator=g, device="cuda") / 16).to(torch.bfloat16))
    w2 = nq.ep_nvfp4_pack_weights((torch.randn(E, H, I, generator=g, device="cuda") / 11).to(torch.bfloat16))
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    topk = route(T, k, E, g)
    weights = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    want = layer(x, topk, weights, w1, w2)
    W1, W2 = decode_rows(w1, H), decode_rows(w2, I)
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(topk[t, j])
            h = (W1[e] @ x[t].double())
            ref[t] += weights[t, j].double() * (W2[e] @ (h[:I] / (1 + torch.exp(-h[:I])) * h[I:]))
    assert (want.double() - ref).norm() <= 4 * B * ref.norm()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer(x, topk, weights, w1, w2, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(x, topk, weights, w1, w2)
    x.mul_(-1)
    graph.replay()
    assert torch.equal(held, layer(x, topk, weights, w1, w2))


def test_binding_refuses_wrong_operands():
    dev = "cuda"
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)   # noqa: E731
    topk = torch.tensor([[0, 1], [1, 2]], dtype=torch.int32, device=dev)
    plan = nq.ep_route_plan(topk, 4)
    rows = bf(plan.R_cap, 64)
    for call in (
            lambda: nq.ep_pack(bf(3, 64), plan),                                  # tokens of another batch
            lambda: nq.ep_pack(bf(2, 64).half(), plan),                           # a type it does not take
            lambda: nq.ep_pack(bf(64, 2).t(), plan),                              # columns, not rows
            lambda: nq.ep_pack(bf(1, 64).expand(2, 64), plan),                    # one row seen twice
            lambda: nq.ep_pack(bf(2, 64), plan, rows=rows[:-1]),                  # too few rows
            lambda: nq.ep_pack(bf(2, 64), plan, rows=rows.float()),               # another type
            lambda: nq.ep_combine(rows),                                          # neither order
            lambda: nq.ep_combine(rows, plan, topk_idx=topk),                     # both
            lambda: nq.ep_combine(rows, topk_idx=topk),                           # not T*k rows
            lambda: nq.ep_combine(rows, plan, weights=torch.ones(2, 3, device=dev)),
            lambda: nq.ep_combine(rows, plan, weights=bf(2, 2)),
            lambda: nq.ep_combine(rows, plan, out=bf(2, 63)),
            lambda: nq.ep_combine_backward(bf(2, 64), plan, rows=rows[1:]),
            lambda: nq.ep_combine_backward(bf(2, 64), plan, rows=rows.float()),
            lambda: nq.ep_combine_backward(bf(2, 64), plan, d_weights=torch.zeros(2, 2, device=dev)),
            lambda: nq.ep_swiglu(bf(4, 96)),
            lambda: nq.ep_swiglu(bf(4, 64), E=2),
            lambda: nq.ep_swiglu(bf(4, 64), plan.offsets, 5),
            lambda: nq.ep_swiglu(bf(4, 64), ckpt=torch.zeros(10, dtype=torch.uint8, device=dev)),
            lambda: nq.ep_swiglu_backward(bf(4, 32), torch.zeros(10, dtype=torch.uint8, device=dev)),
            lambda: nq.ep_nvfp4_matvec(bf(2, 64), torch.zeros(4, 8, 32, dtype=torch.uint8, device=dev), topk),
            lambda: nq.ep_nvfp4_matvec(bf(3, 64), torch.zeros(4, 8, nq.row_bytes(64), dtype=torch.uint8, device=dev), topk),
            lambda: nq.ep_nvfp4_matvec(bf(2, 64), torch.zeros(4, 8, nq.row_bytes(64), dtype=torch.uint8, device=dev)),
            lambda: nq.ep_nvfp4_matvec(bf(2, 64), torch.zeros(4, 8, nq.row_bytes(64), dtype=torch.uint8, device=dev),
                                       topk.long())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nq.EpError):      # rows that are not 16-byte aligned
        nq.ep_swiglu(bf(4, 66)[:, 1:65])
