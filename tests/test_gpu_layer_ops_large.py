"""Large batches of rows that start anywhere, and products of one token with
long rows, against the definitions in 64 bits, with the bounds of
test_gpu_layer_ops.

The batch sizes follow the device's SM count, on both sides of the number of
slots from which a slot has a warp instead of a CTA.
"""
import math

import pytest
import torch

import nvfp4_quantization_gb300 as nq
from test_gpu_layer_ops import B, TYPES, U, check_matvec, combine64, decode_rows, dest_of, gen, inside, matvec_bound
from test_gpu_layer_ops import route, ulp, within

pytestmark = pytest.mark.gpu


def tokens(k, above):
    """T with T * k well above, or just below, 16 slots an SM; no multiple of 8 slots."""
    edge = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    T = edge // k + 300 if above else edge // k - 1
    while T * k % 8 == 0:
        T += 1 if above else -1
    assert (T * k >= edge) == above
    return T


@pytest.mark.parametrize("above", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,E,offset", [(331, 16, 1), (1001, 61, 3), (2307, 300, 5), (117, 7, 1)])
def test_large_batches_of_rows_that_start_anywhere(H, E, offset, dt, above):
    dtype, g, k = TYPES[dt], gen(60 + offset), 3
    T = tokens(k, above)
    topk = route(T, k, E, g, 0.1)
    plan = nq.ep_route_plan(topk, E)
    d = dest_of(plan)
    live = d >= 0
    R = int(plan.offsets[-1])
    tok = inside(T, H, dtype, offset, float("nan"))[0]
    tok.copy_(torch.randn(T, H, generator=g, device="cuda"))

    def untouched(buf, first, n):
        assert (buf[:first] == 7.0).all() and (buf[first + n:] == 7.0).all()

    first = offset * 3 % 8
    rows, buf = inside(plan.R_cap, H, dtype, first, 7.0)
    nq.ep_pack(tok, plan, rows=rows)
    want = torch.full_like(rows, 7.0)
    want[:R] = 0
    for j in range(k):
        want[d[live[:, j], j]] = tok[live[:, j]]
    assert torch.equal(rows, want)
    untouched(buf, first, rows.numel())

    rows[:R] = torch.randn(R, H, generator=g, device="cuda").to(dtype)
    pad = torch.ones(plan.R_cap, dtype=torch.bool, device="cuda")
    pad[d[live]] = False
    rows[pad] = float("nan")             # nothing of a padding row is used
    weights = torch.randn(T, k, generator=g, device="cuda")
    weights[~live] = float("inf")
    first = offset * 5 % 8
    out, buf = inside(T, H, dtype, first, 7.0)
    nq.ep_combine(rows, plan, weights, out=out)
    sums, mag = combine64(rows, d, live, weights)
    within(out, sums, ulp(dtype) * sums.abs() * (1 + B) + 2 * k * U * mag + 2.0 ** -133)
    untouched(buf, first, out.numel())

    first = offset * 7 % 8
    d_rows, buf = inside(plan.R_cap, H, dtype, first, 7.0)
    _, d_w = nq.ep_combine_backward(tok, plan, weights, rows=rows, d_rows=d_rows)
    untouched(buf, first, d_rows.numel())
    assert (d_rows[R:] == 7.0).all() and not d_rows[:R][pad[:R]].any()
    for j in range(k):
        t = live[:, j].nonzero().reshape(-1)
        v = tok[t].double() * weights[t, j].double().unsqueeze(1)
        within(d_rows[d[t, j]], v, (ulp(dtype) + 2 * U) * v.abs() + 2.0 ** -133)
        p = tok[t].double() * rows[d[t, j]].double()
        within(d_w[t, j], p.sum(1), 2 * H * U * p.abs().sum(1))
    assert not d_w[~live].any()
    plain, _ = nq.ep_combine_backward(tok, plan, d_rows=torch.full((plan.R_cap, H), 7.0, dtype=dtype, device="cuda"))
    assert torch.equal(plain, want)      # without weights and their gradient: the pack
    assert int(plan.status) == 0


@pytest.mark.parametrize("k,E,N,K", [(8, 12, 70, 4128), (8, 16, 90, 7168), (2, 3, 33, 32768), (5, 130, 9, 32768),
                                     (1, 1, 4099, 8192), (3, 5, 16, 14336)])
def test_one_token_with_long_rows(k, E, N, K):
    g = gen(70)
    topk = route(1, k, E, g)
    topk[0, 0] = E - 1
    w = torch.randn(E, N, K, generator=g, device="cuda") / math.sqrt(K)
    w_rows = nq.ep_nvfp4_pack_weights(w.to(torch.bfloat16))
    x = torch.randn(1, K, generator=g, device="cuda")
    x[:, ::13] *= 2.0 ** -20
    x[:, K - 5:] *= 2.0 ** 6             # the last elements count
    x = x.to(torch.bfloat16)
    status = nq.new_status("cuda")
    y = torch.full((k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    nq.ep_nvfp4_matvec(x, w_rows, topk, y=y, status=status)
    check_matvec(x, w_rows, topk, y)
    xs = (torch.randn(k, K, generator=g, device="cuda")).to(torch.bfloat16)      # a row a slot
    check_matvec(xs, w_rows, topk, nq.ep_nvfp4_matvec(xs, w_rows, topk, status=status))
    assert int(status) == 0


@pytest.mark.parametrize("T", [1, 3])
def test_weights_past_32_bit_offsets(T):
    """The last expert's rows lie past 2^32 bytes."""
    K, N, E, last = 7168, 8192, 140, 64
    S = nq.row_bytes(K)
    assert (E - 1) * N * S > 1 << 32
    g = gen(71)
    w_rows = torch.zeros(E, N, S, dtype=torch.uint8, device="cuda")
    w = torch.randn(1, last, K, generator=g, device="cuda") / 64
    w_rows[E - 1, N - last:] = nq.ep_nvfp4_pack_weights(w.to(torch.bfloat16))[0]
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    topk = torch.tensor([[E - 1, 0]] * T, dtype=torch.int32, device="cuda")
    y = nq.ep_nvfp4_matvec(x, w_rows, topk).view(T, 2, N)
    assert not y[:, 0, : N - last].any() and not y[:, 1].any()
    W = decode_rows(w_rows[E - 1, N - last:], K)
    for t in range(T):
        want, mag = W @ x[t].double(), W.abs() @ x[t].double().abs()
        within(y[t, 0, N - last:], want, matvec_bound(want, mag, K, W, x[t].double()))
