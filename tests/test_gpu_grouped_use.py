"""The grouped products as they are used: errors that only the data shows,
streams, graphs, many tiles, large tensors, reproducibility, and the layer that
they make up.  (Bounds: see test_gpu_grouped.py.)"""
import os
import sys

import pytest
import torch

import nvfp4_quantization_gb300 as nq
import test_gpu_grouped as tg
from test_gpu_grouped import B, NAN, U, gen, ints, randn, slots, sum_bound, within

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def operands(g, R_cap, E, K, N, offsets, live):
    """Everything the four products take, for R_cap rows."""
    x = (randn(g, R_cap, K) * live.unsqueeze(1)).to(torch.bfloat16)
    dy = (randn(g, R_cap, N) * live.unsqueeze(1)).to(torch.bfloat16)
    w = randn(g, E, N, K).to(torch.bfloat16)
    return dict(x=x, dy=dy, w=w, xo=nq.ep_nvfp4_operand(tg.pack_rows(x), K),
                wo=nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(w), K),
                xc=tg.columnwise(x, offsets, E), dyc=tg.columnwise(dy, offsets, E))


def products(s, offsets, counts, E, K, N, **kw):
    return [nq.ep_grouped_gemm(s["x"], s["w"], offsets, **kw),
            nq.ep_grouped_gemm(s["dy"], s["w"], offsets, transpose=True, **kw),
            nq.ep_grouped_wgrad(s["dy"], s["x"], offsets, E, counts=counts, **kw),
            nq.ep_nvfp4_grouped_gemm(s["xo"], s["wo"], offsets, **kw),
            nq.ep_nvfp4_grouped_wgrad(s["dyc"], s["xc"], N, K, offsets, E, **kw)]


def rows_of(outs, R):
    """The rows that the calls write (the weight gradients whole)."""
    return [o[:R] if o.dim() == 2 else o for o in outs]


COUNTS = [130, 0, 300, 7, 128]
K, N = 384, 256


def test_another_stream_and_two_at_once():
    g = gen(21)
    offsets, off, R_cap, live = slots(COUNTS)
    s = operands(g, R_cap, 5, K, N, offsets, live)
    want = products(s, offsets, ints(COUNTS), 5, K, N)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
            outs.append(products(s, offsets, ints(COUNTS), 5, K, N, stream=st))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))       # and so every run gives the same bits


def test_graph_replay_with_other_values_and_offsets():
    g = gen(22)
    offsets, off, R_cap, live = slots(COUNTS)
    counts = ints(COUNTS)
    s = operands(g, R_cap, 5, K, N, offsets, live)
    products(s, offsets, counts, 5, K, N)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = products(s, offsets, counts, 5, K, N)
    for c in (COUNTS, [7, 300, 128, 130, 0]):
        o2, off2, cap2, live2 = slots(c)
        assert cap2 == R_cap
        t = operands(g, R_cap, 5, K, N, o2, live2)
        for name, v in t.items():
            for a, b in zip(*((d.values() if isinstance(d, dict) else [d]) for d in (s[name], v))):
                if isinstance(a, torch.Tensor):
                    a.copy_(b)
        offsets.copy_(o2)
        counts.copy_(ints(c))
        graph.replay()
        want = products(t, o2, ints(c), 5, K, N)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_of_other_sizes_in_turn():
    """Nothing between them, so that one starts while another ends."""
    g = gen(32)
    sets = []
    for counts, n, k in (([130, 0, 300, 7, 128], 256, 384), ([1500], 128, 128), ([5, 700, 1, 128, 0, 64, 900], 512, 256),
                         ([128] * 7, 256, 384)):
        offsets, off, R_cap, live = slots(counts)
        ops = [tg.columnwise((randn(g, R_cap, h) * live.unsqueeze(1)).to(torch.bfloat16), offsets, len(counts))
               for h in (n, k)]
        want = nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], n, k, offsets, len(counts))
        for e in range(len(counts)):
            if off[e + 1] > off[e]:
                a, b = (tg.columnwise_values(op, h, off, e) for op, h in zip(ops, (n, k)))
                within(want[e], a @ b.t(), sum_bound(off[e + 1] - off[e], a.abs() @ b.abs().t(), a @ b.t(),
                                                     torch.float32, more=4))
        sets.append((ops, n, k, offsets, len(counts), want, torch.empty_like(want), nq.new_status("cuda")))
    for _ in range(30):
        for ops, n, k, offsets, E, want, out, status in sets:
            out.fill_(NAN)
        for ops, n, k, offsets, E, want, out, status in sets:
            nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], n, k, offsets, E, d_w=out, status=status)
        assert all(torch.equal(out, want) and int(status) == 0 for *_, want, out, status in sets)


def test_slots_that_are_not_whole_tiles():
    g = gen(23)
    offsets, off, R_cap, live = slots([128, 128, 256])
    s = operands(g, R_cap, 3, K, N, offsets, live)
    want = products(s, offsets, None, 3, K, N)
    for bad in ([0, 100, 256, 512], [0, 128, 256, 512 - 64], [-128, 128, 256, 512], [0, 256, 128, 512]):
        status = nq.new_status("cuda")
        fill = torch.full((R_cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
        fill4 = fill.clone()
        nq.ep_grouped_gemm(s["x"], s["w"], ints(bad), out=fill, status=status)
        nq.ep_nvfp4_grouped_gemm(s["xo"], s["wo"], ints(bad), out=fill4, status=status)
        d_w = nq.ep_grouped_wgrad(s["dy"], s["x"], ints(bad), 3, status=status)
        d_w4 = nq.ep_nvfp4_grouped_wgrad(s["dyc"], s["xc"], N, K, ints(bad), 3, status=status)
        assert int(status) == nq.EP_DEV_ERR_BAD_EXPERT
        for e in range(3):
            a, b = bad[e], bad[e + 1]
            if a < 0 or b < a or a % 128 or b % 128:      # counts as empty
                assert (d_w[e] == 0).all() and (d_w4[e] == 0).all()
            elif [a, b] == off[e: e + 2]:
                assert torch.equal(d_w[e], want[2][e]) and torch.equal(d_w4[e], want[4][e])
                assert torch.equal(fill[a:b], want[0][a:b]) and torch.equal(fill4[a:b], want[3][a:b])
        if bad[-1] < 512:
            assert (fill[bad[-2]:] == 7.0).all() and (fill4[bad[-2]:] == 7.0).all()


def test_rows_past_the_capacity():
    g = gen(24)
    offsets, off, R_cap, live = slots([128, 256])
    s = operands(g, R_cap, 2, K, N, offsets, live)
    want = products(s, offsets, None, 2, K, N)
    cut = 256                             # of 384 rows
    status = nq.new_status("cuda")
    guard = torch.full((R_cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    nq.ep_grouped_gemm(s["x"][:cut], s["w"], offsets, out=guard[:cut], status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY
    assert torch.equal(guard[:cut], want[0][:cut]) and (guard[cut:] == 7.0).all()
    status.zero_()
    d_w = nq.ep_grouped_wgrad(s["dy"][:cut], s["x"][:cut], offsets, 2, status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY
    assert torch.equal(d_w[0], want[2][0])
    a, b = s["dy"][128:cut].double().t(), s["x"][128:cut].double()
    within(d_w[1], a @ b, sum_bound(128, a.abs() @ b.abs(), a @ b, torch.float32))
    status.zero_()
    part = lambda op, H: dict(cw_codes=op["cw_codes"][: cut * H // 2], cw_scales=op["cw_scales"][: cut * H // 16],   # noqa: E731
                              cw_scale_enc=op["cw_scale_enc"])
    d_w = nq.ep_nvfp4_grouped_wgrad(part(s["dyc"], N), part(s["xc"], K), N, K, offsets, 2, status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY
    assert torch.equal(d_w[0], want[4][0]) and (d_w[1] == 0).all()
    status.zero_()
    few = dict(s["xo"], rw_codes=s["xo"]["rw_codes"][:cut])
    guard.fill_(7.0)
    nq.ep_nvfp4_grouped_gemm(few, s["wo"], offsets, out=guard[:cut], status=status)
    assert int(status) == nq.EP_DEV_ERR_CAPACITY
    assert torch.equal(guard[:cut], want[3][:cut]) and (guard[cut:] == 7.0).all()


def test_nvfp4_capacity_below_a_slot():
    """Fewer rows than a tile hold no slot: one that is there all the same is past
    the capacity, and nothing is written."""
    g = gen(34)
    rows = tg.pack_rows(randn(g, 100, 64))
    wo = nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(randn(g, 2, 16, 64).to(torch.bfloat16)), 64)
    for offsets, want in (([0, 0, 0], 0), ([0, 128, 128], nq.EP_DEV_ERR_CAPACITY)):
        out = torch.full((100, 16), 7.0, dtype=torch.bfloat16, device="cuda")
        status = nq.new_status("cuda")
        nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, 64), wo, ints(offsets), out=out, status=status)
        assert int(status) == want and (out == 7.0).all()


def test_counts_beyond_the_slot_and_below_zero():
    g = gen(25)
    offsets, off, R_cap, live = slots([128, 256, 128])
    s = operands(g, R_cap, 3, K, N, offsets, live)
    all_rows = nq.ep_grouped_wgrad(s["dy"], s["x"], offsets, 3)
    got = nq.ep_grouped_wgrad(s["dy"], s["x"], offsets, 3, counts=ints([1 << 30, 256, -5]))
    assert torch.equal(got[:2], all_rows[:2]) and (got[2] == 0).all()


def test_infinities_and_nan_stay_in_their_rows():
    g = gen(26)
    R = 300
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, N, K, generator=g, device="cuda").to(torch.bfloat16)
    want = nq.ep_grouped_gemm(x, w)
    x[5, 3], x[17, 0], x[299, 1] = NAN, float("inf"), -float("inf")
    got = nq.ep_grouped_gemm(x, w)
    clean = torch.ones(R, dtype=torch.bool, device="cuda")
    clean[[5, 17, 299]] = False
    assert torch.equal(got[clean], want[clean])
    assert got[5].isnan().all() and got[17].isinf().all() and got[299].isinf().all()
    assert torch.equal(got[17] > 0, w[0, :, 0] > 0) and torch.equal(got[299] > 0, w[0, :, 1] < 0)


def test_a_row_does_not_depend_on_the_batch():
    """The same rows alone, among others and in another slot: the same bits, with
    one CTA a tile or two, 64 columns or 256."""
    g = gen(27)
    x = torch.randn(4096, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, 2048, K, generator=g, device="cuda").to(torch.bfloat16)
    rows, wo = tg.pack_rows(x), nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(w), K)
    whole, whole4 = nq.ep_grouped_gemm(x, w), nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, K), wo)
    for a, b in ((0, 1), (0, 64), (1000, 1200), (2048, 2560)):
        assert torch.equal(nq.ep_grouped_gemm(x[a:b], w), whole[a:b])
        assert torch.equal(nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows[a:b], K), wo), whole4[a:b])


def test_many_experts_and_many_tiles_a_cta():
    g = gen(28)
    E, n, k = 1024, 72, 40
    counts = [(7 * e) % 131 if e % 3 else 0 for e in range(E)]
    offsets, off, R_cap, live = slots(counts)
    x = torch.randn(R_cap, k, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(R_cap, n, generator=g, device="cuda").to(torch.bfloat16)
    x[~live] = dy[~live] = NAN
    w = torch.randn(E, n, k, generator=g, device="cuda").to(torch.bfloat16)
    status = nq.new_status("cuda")
    out = nq.ep_grouped_gemm(x, w, offsets, status=status)
    d_w = nq.ep_grouped_wgrad(dy, x, offsets, E, counts=ints(counts), status=status)
    of_row = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.diff(offsets.long()))
    xd, dyd, wd = (t.double() for t in (x, dy, w))
    want = torch.bmm(wd[of_row[live]], xd[live].unsqueeze(2)).squeeze(2)
    within(out[live], want, sum_bound(k, torch.bmm(wd[of_row[live]].abs(), xd[live].abs().unsqueeze(2)).squeeze(2), want,
                                      torch.bfloat16))
    for e in list(range(0, 40)) + [1021, 1022, 1023]:
        at = slice(off[e], off[e] + counts[e])
        want = dyd[at].t() @ xd[at]
        within(d_w[e], want, sum_bound(counts[e], dyd[at].t().abs() @ xd[at].abs(), want, torch.float32))
    assert int(status) == 0
    # one expert, more than 32 tiles for every CTA
    x = torch.randn(100_000, 64, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, 2056, 64, generator=g, device="cuda").to(torch.bfloat16)
    want = x.double() @ w[0].double().t()
    within(nq.ep_grouped_gemm(x, w), want, sum_bound(64, x.double().abs() @ w[0].double().abs().t(), want, torch.bfloat16))
    rows = tg.pack_rows(x)
    wr = nq.ep_nvfp4_pack_weights(w)
    want, mag = tg.nvfp4_reference(rows, wr[0], 64)
    within(nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, 64), nq.ep_nvfp4_operand(wr, 64)), want,
           sum_bound(64, mag, want, torch.bfloat16, more=2))


def test_tensors_beyond_32_bits():
    g = gen(29)
    R, n, k = 600_000, 4096, 64                       # 2.4e9 outputs
    x = torch.randn(R, k, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, n, k, generator=g, device="cuda").to(torch.bfloat16)
    out = nq.ep_grouped_gemm(x, w)
    at = torch.randint(0, R, (300,), generator=g, device="cuda")
    at[:3] = torch.tensor([0, R - 1, (1 << 31) // n], device="cuda")
    want = x[at].double() @ w[0].double().t()
    within(out[at], want, sum_bound(k, x[at].double().abs() @ w[0].double().abs().t(), want, torch.bfloat16))
    del out
    E, n, k = 40, 8192, 8192                          # 2.7e9 FP32 weights
    counts = [3] * E
    offsets, off, R_cap, live = slots(counts)
    x = torch.randn(R_cap, k, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(R_cap, n, generator=g, device="cuda").to(torch.bfloat16)
    d_w = nq.ep_grouped_wgrad(dy, x, offsets, E, counts=ints(counts))
    for e in (0, 32, E - 1):
        rows = slice(off[e], off[e] + 3)
        a, b = dy[rows].double().t(), x[rows].double()
        within(d_w[e], a @ b, sum_bound(3, a.abs() @ b.abs(), a @ b, torch.float32))


def test_long_sums_in_parts():
    """FP32 weight gradients add their parts up in FP32: the error stays that of
    the longest part, 48 additions of 16 rows in BF16 and 128 of 64 in NVFP4, each
    truncated by at most 2 u of the running sum, and one rounding for a part."""
    g = gen(30)
    for R in (767, 769, 1536, 20_000):
        x, dy = (torch.randn(R, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        a, b = dy.double().t(), x.double()
        want = a @ b
        base = torch.randn(1, 128, 128, generator=g, device="cuda")
        got = nq.ep_grouped_wgrad(dy, x, d_w=base.clone(), accumulate=True)
        # the sums of all prefixes are below sum|terms|
        parts = -(-R // 768)
        within(got[0] - base[0], want, (2 * 48 + parts + 2) * U * (a.abs() @ b.abs()) + 2 * U * base[0].double().abs())
    R = 8192 * 2 + 640
    offsets, off, R_cap, live = slots([R])
    ops = [tg.columnwise(torch.randn(R_cap, 128, generator=g, device="cuda").to(torch.bfloat16), offsets, 1) for _ in range(2)]
    a, b = (tg.columnwise_values(op, 128, off, 0) for op in ops)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    within(nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], 128, 128, offsets, 1)[0], want, (2 * 128 + 3 + 4) * U * mag)
    base = torch.randn(1, 128, 128, generator=g, device="cuda")
    got = nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], 128, 128, offsets, 1, d_w=base.clone(), accumulate=True)
    within(got[0], want + base[0].double(), (2 * 128 + 3 + 4) * U * mag + 4 * U * (base[0].double().abs() + mag))




def test_gradients_are_the_differences_of_the_product():
    """Small whole numbers: every product, sum and output is exact in BF16, so the
    differences of L = <dy, product> are the gradients exactly."""
    g = gen(31)
    counts = [3, 0, 130]
    offsets, off, R_cap, live = slots(counts)
    k, n = 16, 8
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    x, dy = whole(R_cap, k), whole(R_cap, n)
    x[~live] = dy[~live] = 0
    w = whole(3, n, k)
    loss = lambda x, w: (dy.double() * nq.ep_grouped_gemm(x, w, offsets).double())[live].sum().item()   # noqa: E731
    d_x = nq.ep_grouped_gemm(dy, w, offsets, transpose=True)
    d_w = nq.ep_grouped_wgrad(dy, x, offsets, 3, counts=ints(counts))
    at = loss(x, w)
    for e, i, j in [(0, 0, 0), (0, 7, 15), (1, 3, 3), (2, 0, 9), (2, 5, 2)]:
        w2 = w.clone()
        w2[e, i, j] += 1
        assert loss(x, w2) - at == d_w[e, i, j].item()
    for r, j in [(0, 0), (2, 15), (128, 3), (257, 8)]:
        x2 = x.clone()
        x2[r, j] += 1
        assert loss(x2, w) - at == d_x[r, j].item()


def test_empty_calls():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    assert nq.ep_grouped_gemm(z(0, 64), z(2, 8, 64), ints([0, 0, 0])).shape == (0, 8)
    assert (nq.ep_grouped_wgrad(z(0, 8), z(0, 64), ints([0, 0, 0]), 2) == 0).all()
    d_w = torch.full((2, 8, 64), 3.0, device="cuda")
    nq.ep_grouped_wgrad(z(0, 8), z(0, 64), ints([0, 0, 0]), 2, d_w=d_w, accumulate=True)
    assert (d_w == 3).all()
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")   # noqa: E731
    cw = dict(cw_codes=u8(0), cw_scales=u8(0), cw_scale_enc=torch.ones(2, device="cuda"))
    assert (nq.ep_nvfp4_grouped_wgrad(cw, cw, 128, 128, ints([0, 0, 0]), 2) == 0).all()
    op = nq.ep_nvfp4_operand(u8(0).view(0, nq.row_bytes(64)), 64)
    wo = nq.ep_nvfp4_operand(u8(8 * nq.row_bytes(64)).view(1, 8, -1), 64)
    assert nq.ep_nvfp4_grouped_gemm(op, wo).shape == (0, 8)


def test_binding_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")   # noqa: E731
    operand = lambda *s: nq.ep_nvfp4_operand(u8((*s[:-1], nq.row_bytes(s[-1]))), s[-1])   # noqa: E731
    off = ints([0, 128, 128])
    for bad in (lambda: nq.ep_grouped_gemm(z(128, 64), z(2, 8, 72), off),
                lambda: nq.ep_grouped_gemm(z(128, 64), z(2, 8, 64)),
                lambda: nq.ep_grouped_gemm(z(128, 64).t(), z(2, 8, 128), off),
                lambda: nq.ep_grouped_gemm(z(128, 64), z(2, 8, 64), off.long()),
                lambda: nq.ep_grouped_gemm(z(128, 64), z(2, 8, 64), off, out=z(128, 16)),
                lambda: nq.ep_grouped_gemm(z(128, 64).float(), z(2, 8, 64), off),
                lambda: nq.ep_grouped_wgrad(z(128, 64), z(256, 64), off, 2),
                lambda: nq.ep_grouped_wgrad(z(128, 64), z(128, 64), off, 2, accumulate=True),
                lambda: nq.ep_grouped_wgrad(z(128, 64), z(128, 64), off, 2, dtype=torch.float16),
                lambda: nq.ep_grouped_wgrad(z(128, 64), z(128, 64), off, 2, counts=ints([1])),
                lambda: nq.ep_nvfp4_operand(torch.zeros(4, 40, dtype=torch.uint8, device="cuda"), 64),
                lambda: nq.ep_nvfp4_grouped_gemm(operand(8, 64), operand(1, 8, 96)),
                lambda: nq.ep_nvfp4_grouped_gemm(dict(operand(8, 64), K=128), dict(operand(1, 8, 64), K=128)),
                lambda: nq.ep_nvfp4_grouped_gemm(operand(300, 64), dict(operand(1, 8, 64), rw_scales=u8(500))),
                lambda: nq.ep_nvfp4_grouped_gemm(dict(operand(300, 64), rw_scales=u8(1024)), operand(1, 8, 64))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nq.ep_grouped_gemm(z(128, 60), z(2, 8, 60), off),
                lambda: nq.ep_grouped_gemm(z(128, 64), z(2, 12, 64), off),
                lambda: nq.ep_grouped_gemm(z(128, 68)[:, :64], z(2, 8, 64), off),
                lambda: nq.ep_grouped_wgrad(z(128, 64), z(128, 64), off, 2, d_w=z(2, 64, 64), accumulate=True)):
        with pytest.raises(nq.EpError):
            bad()


# Relative errors in the 2-norm, with the shares of test_gpu_moe_layer.py: a
# tenth for each factor that was rounded to E2M1 to nearest, times sqrt(2) where
# it was rounded stochastically (mean squares 1/12 and 1/6 of a step), added up
# over the factors that a result has passed through; the kept activation input's
# E4M3 and the BF16 stages as there.
BF16, MX, FP4, SR = 8 * B, 3 * 2.0 ** -4, 0.1, 0.1 * 2 ** 0.5


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 128, 4, 2), (1000, 512, 384, 16, 5)])
def test_nvfp4_layer(T, H, I, E, k):
    import moe_layer
    err = moe_layer.main(T, H, I, E, k, seed=4)
    assert err["out"] <= BF16 and err["d_w1"] <= BF16 + MX and err["d_w2"] <= BF16 + MX and err["d_x"] <= BF16 + MX
    out = 4 * FP4 + BF16                              # x, w1, the activation, w2
    assert err["out_nvfp4"] <= out and err["d_weights_nvfp4"] <= out
    # d_y and w2, then g and u of x and w1 in the activation's gradient
    d_h = SR + FP4 + 2 * FP4 + MX + BF16
    assert err["d_x_nvfp4"] <= d_h + SR + FP4
    assert err["d_w1_nvfp4"] <= d_h + SR + 2 * FP4    # d_h once more, x packed and again along the tokens
    assert err["d_w2_nvfp4"] <= 2 * SR + 4 * FP4 + BF16


@pytest.mark.parametrize("n,k", [(4096, 1056), (3000, 544), (2568, 96)])
def test_large_products_of_packed_rows(n, k):
    """Enough rows and features for clusters that share the rows' side, the last
    tile of the features cut; rows of experts of 1 to 2300 tokens."""
    g = gen(33)
    counts = [2300, 1, 900, 0, 1500, 256, 700, 1024]
    offsets, off, R_cap, live = slots(counts, spare=40)
    rows = torch.zeros(R_cap, nq.row_bytes(k), dtype=torch.uint8, device="cuda")
    rows[: off[-1]] = tg.pack_rows(randn(g, off[-1], k))
    w = nq.ep_nvfp4_pack_weights(randn(g, len(counts), n, k).to(torch.bfloat16))
    status = nq.new_status("cuda")
    out = torch.full((R_cap, n), 7.0, dtype=torch.bfloat16, device="cuda")
    nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, k, offsets, len(counts)), nq.ep_nvfp4_operand(w, k), offsets,
                             out=out, status=status)
    copied = nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(rows, k, offsets, len(counts), copy_codes=True),
                                      nq.ep_nvfp4_operand(w, k, copy_codes=True), offsets, status=status)
    assert torch.equal(out[: off[-1]], copied[: off[-1]]) and (out[off[-1]:] == 7.0).all() and int(status) == 0
    for e in range(len(counts)):
        if counts[e]:
            at = slice(off[e], off[e + 1])
            want, mag = tg.nvfp4_reference(rows[at], w[e], k)
            within(out[at], want, sum_bound(k, mag, want, torch.bfloat16, more=2))


@pytest.mark.parametrize("T,H,I,E,k", [(40, 256, 128, 4, 2), (3000, 1024, 512, 16, 4)])
def test_chain_in_a_graph_without_anything_between(T, H, I, E, k):
    """Plan, pack, products, activation and combine and their gradients one after
    another in a captured graph, each launch let in while the one before ends;
    replayed with other tokens and routing, twice in a row."""
    g = gen(35)
    w1, w2 = ((torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).to(torch.bfloat16)
              for s in ((E, 2 * I, H), (E, H, I)))
    w1o, w2o = (nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(w), w.shape[2]) for w in (w1, w2))
    R_cap = nq.rows_capacity(T, k, E)
    x, d_out = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    topk, weights = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    status, ws = nq.new_status("cuda"), nq.new_route_workspace(T, k, E, "cuda")
    new = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")   # noqa: E731
    plan = nq.RoutePlan(new(E + 1, dt=torch.int32), new(E, dt=torch.int32), new(T * k, dt=torch.int32), T, k, E, 128,
                        R_cap, status)
    b = dict(rows=new(R_cap, H), h=new(R_cap, 2 * I), act=new(R_cap, I), y=new(R_cap, H), out=new(T, H),
             packed=new(R_cap, nq.row_bytes(H), dt=torch.uint8), h4=new(R_cap, 2 * I), d_y=new(R_cap, H),
             d_act=new(R_cap, I), d_w=new(E, H, I, dt=torch.float32), amax=new(E, dt=torch.float32),
             ckpt=new(nq.swiglu_checkpoint_bytes(R_cap, I), dt=torch.uint8), d_wt=new(T, k, dt=torch.float32),
             scales=new(nq.nvfp4_scale_bytes(R_cap, H), dt=torch.uint8), row_scale=new(R_cap, dt=torch.float32))
    ops = nq.alloc_grouped(R_cap, H, E, "cuda")
    d_w4 = new(E, H, H, dt=torch.float32)

    def step():
        at = plan.offsets
        nq.ep_route_plan(topk, E, plan=plan, workspace=ws)
        nq.ep_pack(x, plan, rows=b["rows"])
        nq.ep_grouped_gemm(b["rows"], w1, at, out=b["h"], status=status)
        nq.ep_swiglu(b["h"], at, E, act=b["act"], ckpt=b["ckpt"], status=status)
        nq.ep_grouped_gemm(b["act"], w2, at, out=b["y"], status=status)
        nq.ep_combine(b["y"], plan, weights, out=b["out"])
        nq.ep_combine_backward(d_out, plan, weights, rows=b["y"], d_rows=b["d_y"], d_weights=b["d_wt"])
        nq.ep_grouped_gemm(b["d_y"], w2, at, transpose=True, out=b["d_act"], status=status)
        nq.ep_grouped_wgrad(b["d_y"], b["act"], at, E, counts=plan.counts, d_w=b["d_w"], status=status)
        nq.ep_nvfp4_dispatch(x, topk, E, plan=plan, workspace=ws, rows=b["packed"], expert_amax=b["amax"])
        nq.ep_nvfp4_direct_receive(b["packed"], H, at, E, out=ops, swizzled=True, expert_amax=b["amax"], status=status)
        nq.ep_nvfp4_grouped_gemm(ops, w1o, at, out=b["h4"], status=status)
        nq.ep_nvfp4_grouped_wgrad(ops, ops, H, H, at, E, d_w=d_w4, status=status)
        op = nq.ep_nvfp4_operand(b["packed"], H, at, E, scales=b["scales"], row_scale=b["row_scale"], status=status)
        nq.ep_nvfp4_grouped_gemm(op, w1o, at, out=b["h"], status=status)

    def fill(seed):
        h = gen(seed)
        x.copy_(torch.randn(T, H, generator=h, device="cuda"))
        d_out.copy_(torch.randn(T, H, generator=h, device="cuda"))
        score, ids = torch.rand(T, E, generator=h, device="cuda").topk(k, dim=1)
        topk.copy_(ids)
        weights.copy_(score)

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kept = dict(b, d_w4=d_w4)
    for seed in (1, 2, 3):
        fill(seed)
        for t in kept.values():
            t.zero_()
        graph.replay()
        graph.replay()
        got = {n: t.clone() for n, t in kept.items()}
        for t in kept.values():
            t.zero_()
        step_alone(step)
        R = int(plan.offsets[-1])
        for n, t in kept.items():
            rows = n in ("rows", "h", "act", "y", "packed", "h4", "d_y", "d_act", "row_scale")
            assert torch.equal(got[n][:R] if rows else got[n], t[:R] if rows else t), n
    assert int(status) == 0


def step_alone(step):
    """The same calls, each alone on the GPU."""
    waiting = {n: getattr(nq, n) for n in dir(nq) if n.startswith("ep_")}
    try:
        for n, f in waiting.items():
            setattr(nq, n, lambda *a, _f=f, **kw: (_f(*a, **kw), torch.cuda.synchronize())[0])
        step()
    finally:
        for n, f in waiting.items():
            setattr(nq, n, f)
