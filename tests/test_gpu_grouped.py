"""The matrix products grouped by expert against their definitions in 64 bits.

Error bounds (u = 2^-24, b = 2^-8, half a step of FP32 and BF16): products of
BF16 values, and of E2M1 codes with E4M3 scales, are exact in FP32 (16 bits;
for the scaled ones 2 x (2 + 4) bits); a sum of n of them in any order, each
addition rounded or truncated, is off by at most 2 n u sum|terms|; the row
scales cost two roundings more (u each); the output one rounding (b|y| for
BF16, u|y| for FP32).
"""
import pytest
import torch

import nvfp4_quantization_gb300 as nq

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def slots(counts, spare=0, align=128):
    """Offsets, their list, capacity, and which rows hold a token."""
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // align) * align)
    R_cap = off[-1] + spare
    live = torch.zeros(R_cap, dtype=torch.bool, device="cuda")
    for e, c in enumerate(counts):
        live[off[e]: off[e] + c] = True
    return ints(off), off, R_cap, live


def within(got, want, bound):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), d[bad].max().item(),
                           bound.expand_as(d)[bad].min().item())


def strided(t, extra):
    """The same values with a row pitch `extra` elements wider."""
    if not extra:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + extra), NAN, dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def sum_bound(n, mag, want, dtype, more=0):
    half = B if dtype == torch.bfloat16 else U
    return (2 * n + more) * U * mag * (1 + half) + half * want.abs() + 1e-40


# ----------------------------------------------------------------------------
# BF16
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,K,N,extra", [
    (1, 64, 128, 0), (128, 64, 128, 0), (256, 64, 256, 0), (300, 512, 1024, 0), (1, 8, 8, 0), (7, 40, 24, 8),
    (130, 1000, 136, 0), (500, 72, 2056, 16), (1025, 4096, 520, 0), (33, 8200, 64, 0)])
def test_dense(R, K, N, extra, transpose):
    g = gen(1)
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, *((K, N) if transpose else (N, K)), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = nq.new_status("cuda")
    assert nq.ep_grouped_gemm(strided(x, extra), w, transpose=transpose, out=out, status=status) is out
    wd = w[0].double() if transpose else w[0].double().t()
    want = x.double() @ wd
    within(out, want, sum_bound(K, x.double().abs() @ wd.abs(), want, torch.bfloat16))
    assert int(status) == 0


COUNTS = [[1], [0, 5, 0], [128, 129, 1, 0, 300], [0, 0, 700, 127, 256, 257, 3], [20] * 40, [0] * 5, [1500, 2, 0, 900]]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("K,N,extra", [(64, 128, 0), (200, 264, 8), (1024, 520, 0)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_gemm(counts, K, N, extra, transpose):
    g = gen(2)
    E = len(counts)
    offsets, off, R_cap, live = slots(counts, spare=70)
    x = torch.randn(R_cap, K, generator=g, device="cuda").to(torch.bfloat16)
    x[~live] = NAN                      # rows of nobody reach no other row
    w = torch.randn(E, *((K, N) if transpose else (N, K)), generator=g, device="cuda").to(torch.bfloat16)
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = NAN                  # nor do the weights of an expert without rows
    out = torch.full((R_cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = nq.new_status("cuda")
    nq.ep_grouped_gemm(strided(x, extra), w, offsets, transpose=transpose, out=out, status=status)
    for e, c in enumerate(counts):
        if c:
            at = slice(off[e], off[e] + c)
            wd = w[e].double() if transpose else w[e].double().t()
            want = x[at].double() @ wd
            within(out[at], want, sum_bound(K, x[at].double().abs() @ wd.abs(), want, torch.bfloat16))
    assert (out[off[-1]:] == 7.0).all()
    assert int(status) == 0


@pytest.mark.parametrize("with_counts", [True, False])
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("K,N,extra", [(128, 64, 0), (264, 200, 8), (520, 1024, 0), (8, 8, 0)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_wgrad(counts, K, N, extra, dtype, accumulate, with_counts):
    g = gen(3)
    E = len(counts)
    offsets, off, R_cap, live = slots(counts, spare=70)
    x = torch.randn(R_cap, K, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(R_cap, N, generator=g, device="cuda").to(torch.bfloat16)
    x[~live] = dy[~live] = NAN if with_counts else 0.0
    x[off[-1]:] = dy[off[-1]:] = NAN
    base = torch.randn(E, N, K, generator=g, device="cuda") if accumulate else torch.full((E, N, K), NAN, device="cuda")
    d_w = base.to(dtype, copy=True)
    status = nq.new_status("cuda")
    got = nq.ep_grouped_wgrad(strided(dy, extra), strided(x, extra), offsets, E, counts=ints(counts) if with_counts else None,
                              d_w=d_w, accumulate=accumulate, status=status)
    assert got is d_w
    for e, c in enumerate(counts):
        at = slice(off[e], off[e] + c)
        a, b = dy[at].double().t(), x[at].double()
        want = a @ b
        bound = sum_bound(c, a.abs() @ b.abs(), want, dtype)
        if accumulate:
            want = want + base[e].double()
            bound = bound + U * want.abs()
        within(d_w[e], want, bound)
    assert int(status) == 0


def test_wgrad_dense():
    g = gen(4)
    for R in (0, 1, 63, 65, 300, 1000):
        x = torch.randn(R, 72, generator=g, device="cuda").to(torch.bfloat16)
        dy = torch.randn(R, 136, generator=g, device="cuda").to(torch.bfloat16)
        got = nq.ep_grouped_wgrad(dy, x)
        a, b = dy.double().t(), x.double()
        want = a @ b
        within(got[0], want, sum_bound(R, a.abs() @ b.abs(), want, torch.float32))


# ----------------------------------------------------------------------------
# NVFP4
# ----------------------------------------------------------------------------
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def code_values(codes):
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")
    c = codes.int()
    return torch.stack([grid[c & 15], grid[c >> 4]], -1).reshape(*c.shape[:-1], -1)


def e4m3(b):
    return b.contiguous().view(torch.float8_e4m3fn).double()


def untile(t, M, Kb):
    """Scale (m, b) of tiles [M/128][Kb/4][512]."""
    m = torch.arange(M, device="cuda").unsqueeze(1)
    b = torch.arange(Kb, device="cuda").unsqueeze(0)
    return t[(m // 128 * -(-Kb // 4) + b // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + b % 4]


def values(codes, scales):
    """Codes times block scales (bytes), in 64 bits."""
    v = code_values(codes)
    return (v.view(v.shape[0], -1, 16) * e4m3(scales).unsqueeze(2)).reshape(v.shape)


def decode_rows(rows, K):
    """(values, row scales) of packed rows."""
    S = rows.shape[1]
    return values(rows[:, : K // 2], rows[:, K // 2: 9 * K // 16]), \
        rows[:, S - 16: S - 12].contiguous().view(torch.float32).double().reshape(-1)


def pack_rows(x):
    """Packed rows of x [n, K], row i in its own place."""
    return nq.ep_nvfp4_pack_weights(x.to(torch.bfloat16).unsqueeze(0))[0]


def randn(g, *shape, spread=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    return x * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))


@pytest.mark.parametrize("R,K", [(1, 32), (128, 64), (130, 96), (300, 1056), (1000, 7168), (5, 4096), (129, 2080)])
def test_operand(R, K):
    g = gen(5)
    rows = pack_rows(randn(g, R, K))
    op, copied = nq.ep_nvfp4_operand(rows, K), nq.ep_nvfp4_operand(rows, K, copy_codes=True)
    assert torch.equal(copied["rw_codes"], rows[:, : K // 2]) and op["K"] == copied["K"] == K
    assert all(torch.equal(copied[name], op[name]) for name in ("rw_scales", "rw_row_scale"))
    M, kt = -(-R // 128) * 128, -(-K // 64)
    want = torch.zeros(M, kt * 4, dtype=torch.uint8, device="cuda")
    want[:R, : K // 16] = rows[:, K // 2: 9 * K // 16]
    assert op["rw_scales"].numel() == M * kt * 4 == nq.nvfp4_scale_bytes(R, K) == nq.lib().ep_nvfp4_scale_bytes(R, K)
    assert torch.equal(untile(op["rw_scales"], M, kt * 4), want)
    assert torch.equal(op["rw_row_scale"].double(), decode_rows(rows, K)[1])
    assert op["rw_codes"] is rows


def test_operand_of_slots_and_of_weights():
    g = gen(6)
    K = 160
    offsets, off, R_cap, live = slots([3, 0, 200], spare=100)
    rows = torch.full((R_cap, nq.row_bytes(K)), 0xEE, dtype=torch.uint8, device="cuda")
    rows[: off[-1]] = pack_rows(randn(g, off[-1], K))
    scales = torch.full((nq.nvfp4_scale_bytes(R_cap, K),), 0xAB, dtype=torch.uint8, device="cuda")
    row_scale = torch.full((R_cap,), 7.0, device="cuda")
    op = nq.ep_nvfp4_operand(rows, K, offsets, 3, scales=scales, row_scale=row_scale)
    want = torch.zeros(off[-1], 12, dtype=torch.uint8, device="cuda")
    want[:, :10] = rows[: off[-1], K // 2: 9 * K // 16]
    assert torch.equal(untile(op["rw_scales"], off[-1], 12), want)
    assert (scales[off[-1] * 12:] == 0xAB).all() and (row_scale[off[-1]:] == 7.0).all()
    codes = torch.full((R_cap, K // 2), 0xCD, dtype=torch.uint8, device="cuda")
    copied = nq.ep_nvfp4_operand(rows, K, offsets, 3, codes=codes)
    assert copied["rw_codes"] is codes and torch.equal(codes[: off[-1]], rows[: off[-1], : K // 2])
    assert (codes[off[-1]:] == 0xCD).all()
    w = nq.ep_nvfp4_pack_weights(randn(g, 3, 150, K).to(torch.bfloat16))
    op = nq.ep_nvfp4_operand(w, K)
    assert torch.equal(nq.ep_nvfp4_operand(w, K, copy_codes=True)["rw_codes"], w[..., : K // 2])
    for e in range(3):
        one = nq.ep_nvfp4_operand(w[e], K)
        assert torch.equal(op["rw_scales"].view(3, -1)[e], one["rw_scales"])
        assert torch.equal(op["rw_row_scale"][e], one["rw_row_scale"])


def nvfp4_reference(rows, w_rows, K):
    x, sx = decode_rows(rows, K)
    w, sw = decode_rows(w_rows, K)
    scale = sx.unsqueeze(1) * sw
    return (x @ w.t()) * scale, (x.abs() @ w.abs().t()) * scale


@pytest.mark.parametrize("R,K,N", [(128, 64, 128), (256, 256, 256), (1, 32, 8), (130, 96, 136), (300, 1056, 520),
                                   (1000, 4096, 264), (5, 7168, 64), (700, 2080, 1000)])
def test_nvfp4_dense(R, K, N):
    g = gen(7)
    rows = pack_rows(randn(g, R, K))
    w = nq.ep_nvfp4_pack_weights(randn(g, 1, N, K).to(torch.bfloat16))
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = nq.new_status("cuda")
    nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, K), nq.ep_nvfp4_operand(w, K), out=out, status=status)
    want, mag = nvfp4_reference(rows, w[0], K)
    within(out, want, sum_bound(K, mag, want, torch.bfloat16, more=2))
    assert int(status) == 0


@pytest.mark.parametrize("K,N", [(128, 128), (640, 264), (2176, 520)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_nvfp4_gemm(counts, K, N):
    g = gen(8)
    E = len(counts)
    offsets, off, R_cap, live = slots(counts, spare=70)
    rows = torch.full((R_cap, nq.row_bytes(K)), 0xFF, dtype=torch.uint8, device="cuda")    # NaN scales behind the slots
    if off[-1]:
        rows[: off[-1]] = pack_rows(randn(g, off[-1], K) * live[: off[-1]].unsqueeze(1))
    w = nq.ep_nvfp4_pack_weights(randn(g, E, N, K).to(torch.bfloat16))
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = 0xFF                 # NaN scales in the weights of an expert without rows
    wo = nq.ep_nvfp4_operand(w, K)
    outs = []
    received = nq.ep_nvfp4_direct_receive(rows, K, offsets, E, swizzled=True)
    packed, copied = (nq.ep_nvfp4_operand(rows, K, offsets, E, copy_codes=c) for c in (False, True))
    view = dict(rw_codes=rows[:, : K // 2], rw_scales=packed["rw_scales"], rw_row_scale=packed["rw_row_scale"])
    for x in (received, packed, copied, view):
        out = torch.full((R_cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
        status = nq.new_status("cuda")
        nq.ep_nvfp4_grouped_gemm(x, wo, offsets, out=out, status=status)
        assert int(status) == 0
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)
    for e, c in enumerate(counts):
        if c:
            at = slice(off[e], off[e + 1])
            want, mag = nvfp4_reference(rows[at], w[e], K)
            within(outs[0][at], want, sum_bound(K, mag, want, torch.bfloat16, more=2))
    assert (outs[0][off[-1]:] == 7.0).all()


def columnwise_values(op, H, off, e):
    a, n = off[e], off[e + 1] - off[e]
    codes = op["cw_codes"][a * H // 2: (a + n) * H // 2].view(H, n // 2)
    return values(codes, untile(op["cw_scales"][a * H // 16: (a + n) * H // 16], H, n // 16)) / op["cw_scale_enc"][e].double()


def in_large_buffers(op):
    """The operand's tensors at the start of buffers 16 times as large."""
    out = {}
    for k, v in op.items():
        big = torch.zeros(16 * v.numel() + (1 << 20), dtype=v.dtype, device="cuda")
        big[: v.numel()] = v.reshape(-1)
        out[k] = big[: v.numel()]
    return out


def columnwise(x, offsets, E, **kw):
    amax = x.float().abs().amax().repeat(E)
    return nq.ep_nvfp4_colwise_rht_bf16(x, offsets, E, amax, swizzled=True, **kw)


def test_nvfp4_wgrad_smallest():
    g = gen(9)
    offsets, off, R_cap, live = slots([128])
    dy, x = (randn(g, 128, 128).to(torch.bfloat16) for _ in range(2))
    ops = [in_large_buffers(columnwise(t, offsets, 1)) for t in (dy, x)]
    status = nq.new_status("cuda")
    got = nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], 128, 128, offsets, 1, status=status)
    a, b = (columnwise_values(op, 128, off, 0) for op in ops)
    want = a @ b.t()
    assert int(status) == 0
    within(got[0], want, sum_bound(128, a.abs() @ b.abs().t(), want, torch.float32, more=4))


@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("K,N", [(128, 128), (256, 384), (1152, 640)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_nvfp4_wgrad(counts, K, N, dtype, accumulate):
    g = gen(10)
    E = len(counts)
    offsets, off, R_cap, live = slots(counts, spare=70)
    R = off[-1]
    x = (randn(g, R_cap, K) * live.unsqueeze(1)).to(torch.bfloat16)
    dy = (randn(g, R_cap, N) * live.unsqueeze(1)).to(torch.bfloat16)
    ops = []
    for t, H in ((dy, N), (x, K)):
        op = columnwise(t, offsets, E) if H == N else None
        if op is None:                  # the other side as a direct receive makes it
            rows = torch.zeros(R_cap, nq.row_bytes(H), dtype=torch.uint8, device="cuda")
            if R:
                rows[:R] = pack_rows(t[:R])
            op = nq.ep_nvfp4_direct_receive(rows, H, offsets, E, swizzled=True)
        for k in ("cw_codes", "cw_scales"):           # what lies behind the slots enters nowhere
            op[k][R * H // (2 if k == "cw_codes" else 16):] = 0xFF
        ops.append(op)
    base = torch.randn(E, N, K, generator=g, device="cuda") if accumulate else torch.full((E, N, K), NAN, device="cuda")
    d_w = base.to(dtype, copy=True)
    status = nq.new_status("cuda")
    nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], N, K, offsets, E, d_w=d_w, accumulate=accumulate, status=status)
    for e in range(E):
        n = off[e + 1] - off[e]
        a, b = (columnwise_values(op, H, off, e) if n else torch.zeros(H, 1, dtype=torch.float64, device="cuda")
                for op, H in ((ops[0], N), (ops[1], K)))
        want = a @ b.t()
        bound = sum_bound(n, a.abs() @ b.abs().t(), want, dtype, more=4)
        if accumulate:
            want = want + base[e].double()
            bound = bound + U * want.abs()
        within(d_w[e], want, bound)
    assert int(status) == 0


def test_the_transform_cancels():
    """The sum over transformed rows is the sum over the rows: the operands'
    values, brought back through the transform's inverse, give the same d_w."""
    g = gen(11)
    offsets, off, R_cap, live = slots([300])
    K, N, n, mask = 128, 256, 384, 0x5A3C
    ops = [columnwise((randn(g, R_cap, H) * live.unsqueeze(1)).to(torch.bfloat16), offsets, 1, sign_mask=mask)
           for H in (N, K)]
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    for _ in range(4):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    sign = torch.tensor([-1.0 if mask >> i & 1 else 1.0 for i in range(16)], dtype=torch.float64, device="cuda")
    back = (h / 4) * sign                             # rows y = (h / 4) diag(sign) d, so d = y (h / 4) diag(sign)
    a, b = ((columnwise_values(op, H, off, 0).view(H, n // 16, 16) @ back).reshape(H, n) for op, H in zip(ops, (N, K)))
    want = a @ b.t()
    assert (a[:, 300:304].abs().max() < a.abs().max())
    got = nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], N, K, offsets, 1)[0]
    y = columnwise_values(ops[0], N, off, 0).abs() @ columnwise_values(ops[1], K, off, 0).abs().t()
    within(got, want, sum_bound(n, y, want, torch.float32, more=4))


def test_colwise_scales_in_tiles():
    g = gen(12)
    counts = [0, 130, 1, 512]
    offsets, off, R_cap, live = slots(counts, spare=64)
    for H in (128, 896):
        x = randn(g, R_cap, H).to(torch.bfloat16)
        amax = x.float().abs().amax().repeat(4)
        for rounding in (nq.EP_ROUND_RNE, nq.EP_ROUND_SR):
            flat = nq.ep_nvfp4_colwise_rht_bf16(x, offsets, 4, amax, rounding=rounding, seed=5)
            tiled = nq.ep_nvfp4_colwise_rht_bf16(x, offsets, 4, amax, rounding=rounding, seed=5, swizzled=True)
            R = off[-1]
            assert torch.equal(flat["cw_codes"][: R * H // 2], tiled["cw_codes"][: R * H // 2])
            assert torch.equal(flat["cw_scale_enc"], tiled["cw_scale_enc"])
            for e in range(4):
                a, n = off[e], off[e + 1] - off[e]
                if n:
                    at = slice(a * H // 16, (a + n) * H // 16)
                    assert torch.equal(untile(tiled["cw_scales"][at], H, n // 16), flat["cw_scales"][at].view(H, n // 16))
