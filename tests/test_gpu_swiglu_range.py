"""The gated activation at gates, inputs and gradients of every size, against
its definition in 64 bits.

Bounds (u = 2^-24, b = 2^-8, half an FP32 and a BF16 ulp): exp by one ex2
instruction (2 ulps; its argument's rounding error is carried along), the sum,
the reciprocal (1 ulp) and at most six products behind them stay within 64 u
relative; 1 - s within 32 u absolute, which a gate multiplies; the output is
rounded once more, and BF16's own smallest step is 2^-133.
"""
import pytest
import torch

import nvfp4_quantization_gb300 as nq

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
TOP = 2.0 ** 128
GATES = [0.0, 1.0, 20.0, 50.0, 56.0, 57.0, 80.0, 85.5, 86.0, 86.5, 87.0, 87.5, 88.0, 88.5, 89.0, 90.0, 96.0, 103.0,
         104.0, 120.0, 176.0, 200.0, 255.0, 256.0, 258.0, 1000.0, 1e4, 1e30, 1e38, 2.2e38, 2.4e38, 3.2e38, 3.38e38]
UPS = [1.0, -1.5, 0.0, 2.0 ** -100, -2.0 ** 60, 2.0 ** 100, 2.0 ** 127, -3.38e38]
GRADS = [1.0, -0.75, 2.0 ** -120, 2.0 ** -40, 2.0 ** 20, -2.0 ** 64, 2.0 ** 100, 1.5 * 2.0 ** 126]


def inputs():
    """Every gate (a block of 32 of the same one) with every up value (a row
    each) and every gradient (within the block)."""
    gates = torch.tensor([s * v for v in GATES for s in (1.0, -1.0)], device="cuda")
    n, I = len(UPS), 32 * gates.numel()
    g = gates.repeat_interleave(32).expand(n, I)
    u = torch.tensor(UPS, device="cuda").unsqueeze(1).expand(n, I)
    d = torch.tensor(GRADS * 4, device="cuda").repeat(gates.numel()).expand(n, I).contiguous()
    return torch.cat([g, u], 1).to(torch.bfloat16), d.to(torch.bfloat16), I


def definition(g, u, d):
    s = 1 / (1 + torch.exp(-g))
    return g * s * u, d * u * s * (1 + g * (1 - s)), d * g * s, s


def agrees(got, want, bound, where=None):
    """Within the bound where the result lies in range, infinite with its sign
    where it does not (either where it is about to leave it)."""
    got, edge = got.double(), TOP * (1 - 2.0 ** -9)
    ok = (got - want).abs() <= bound
    over = (got.abs() == float("inf")) & (got.sign() == want.sign())
    ok = torch.where(want.abs() > edge * (1 + 2.0 ** -8), over, ok | (over & (want.abs() > edge * (1 - 2.0 ** -8))))
    if where is not None:
        ok = ok | ~where
    bad = (~ok).nonzero()
    assert not len(bad), [(tuple(i), got[tuple(i)].item(), want[tuple(i)].item()) for i in bad[:4].tolist()]


def test_forward():
    x, _, I = inputs()
    g, u = x[:, :I].double(), x[:, I:].double()
    want = definition(g, u, g)[0]
    bound = (B + 64 * U) * want.abs() + 2.0 ** -133
    for checkpoint in (True, False):
        agrees(nq.ep_swiglu(x, checkpoint=checkpoint)[0], want, bound)


def kept(ckpt, R, I):
    data = ckpt[: R * 2 * I].view(torch.float8_e4m3fn).float().double().view(R, 2 * I // 32, 32)
    scale = torch.exp2(ckpt[R * 2 * I:].double() - 127).view(R, 2 * I // 32, 1)
    v = (data * scale).view(R, 2 * I)
    return v[:, :I], v[:, I:]


@pytest.mark.parametrize("recompute", [True, False])
def test_backward(recompute):
    x, d, I = inputs()
    R = x.shape[0]
    _, ckpt = nq.ep_swiglu(x)
    g, u = kept(ckpt, R, I)
    assert g.isfinite().all() and u.isfinite().all() and g.abs().max() >= TOP and u.abs().max() >= TOP
    d_x, act = nq.ep_swiglu_backward(d, ckpt, recompute=recompute)
    D = d.double()
    a, dg, du, s = definition(g, u, D)
    agrees(d_x[:, I:], du, (B + 64 * U) * du.abs() + 2.0 ** -133)
    # d_act * u comes first: a product out of FP32's range is not brought back
    held = (D * u).abs() < TOP * (1 - B)
    e_dg = (D * u).abs() * s * (1 + g.abs() * (1 - s)) * 96 * U + (D * u).abs() * g.abs() * s * 32 * U
    agrees(d_x[:, :I], dg, B * dg.abs() * (1 + B) + 2 * e_dg + 2.0 ** -133, held)
    if recompute:
        agrees(act, a, (B + 64 * U) * a.abs() + 2.0 ** -133)


def test_amax_of_far_gates():
    """Each expert (a row) gets the amax of its finite gradients."""
    x, _, I = inputs()
    x = x[:2].contiguous()                     # up values of ordinary size
    R = x.shape[0]
    d = torch.full((R, I), 2.0 ** -8, dtype=torch.bfloat16, device="cuda")
    d[1] = -2.0 ** -30
    _, ckpt = nq.ep_swiglu(x)
    g, u = kept(ckpt, R, I)
    _, dg, du, _ = definition(g, u, d.double())
    amax = torch.zeros(R, device="cuda")
    off = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    nq.ep_swiglu_backward(d, ckpt, off, R, expert_amax=amax)
    want = torch.maximum(dg.abs(), du.abs()).amax(1)
    assert ((amax.double() - want).abs() <= 64 * U * want).all(), (amax, want)


def test_a_far_gate_leaves_its_neighbours_alone():
    """Columns beside far gates of the same thread and block: the bits that
    they have without them."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(40)
    R, I = 50, 96
    x = torch.randn(R, 2 * I, generator=gen, device="cuda").to(torch.bfloat16)
    far = torch.rand(R, I, generator=gen, device="cuda") < 0.05
    y = x.clone()
    y[:, :I][far] = -100.0
    a, b = nq.ep_swiglu(x, checkpoint=False)[0], nq.ep_swiglu(y, checkpoint=False)[0]
    assert torch.equal(a[~far], b[~far])
    assert far.any() and (b[far].float().abs() < 1e-38).all()
