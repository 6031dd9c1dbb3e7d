"""FP32 weight gradients whose sums are taken in parts, at sizes that pairs of
CTAs compute, against 64 bits.

Sizes: with 152 SMs, 8 experts of 2056 x 2056 (NVFP4: 2176 x 2176) are 17 x 9 x 8
= 1224 tiles of 128 x 256 for single CTAs, 9 rounds, and 9 x 9 x 8 = 648 of 256 x
256 for pairs, 9 rounds of 76: 9 * 12 >= 9 * 10, so pairs take them, with a last
tile of 8 (128) rows.

Bounds (u = 2^-24).  All terms are positive, so every partial sum is at most the
result S.  A part's sum is cut to 24 bits at each addition, by at most 2 u of what
it has reached: 48 additions of 16 rows in BF16, 128 of 64 in NVFP4, which makes
2 * 48 u (2 * 128 u) of S for all parts together.  Adding a part: one rounding, u
S.  BF16 then rounds once more where it adds to d_w; in NVFP4 the parts are added
to d_w one by one, so each addition rounds the base with it, and the two scales
are two factors rounded, and two products.  Lost parts would show in BF16: without
them 15001 rows lose more than twice the bound, at the 2.1e-6 of S in 2048 rows that
the matrix unit was measured to lose.
"""
import pytest
import torch

import nvfp4_quantization_gb300 as nq
from test_gpu_grouped import NAN, U, columnwise_values, gen, ints, slots, within

pytestmark = pytest.mark.gpu


def positive(g, *shape):
    return (torch.rand(*shape, generator=g, device="cuda") + 0.05).to(torch.bfloat16)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("with_counts", [True, False])
def test_bf16(with_counts, accumulate):
    g = gen(51)
    counts = [15001, 0, 1537, 768, 2000, 5, 769, 4000]
    E, N, K = len(counts), 2056, 2056
    offsets, off, R_cap, live = slots(counts, spare=40)
    dy, x = positive(g, R_cap, N), positive(g, R_cap, K)
    dy[~live] = x[~live] = NAN if with_counts else 0.0
    base = torch.rand(E, N, K, generator=g, device="cuda") if accumulate else torch.full((E, N, K), NAN, device="cuda")
    status = nq.new_status("cuda")
    d_w = nq.ep_grouped_wgrad(dy, x, offsets, E, counts=ints(counts) if with_counts else None, d_w=base.clone(),
                              accumulate=accumulate, status=status)
    for e, c in enumerate(counts):
        at = slice(off[e], off[e] + c)
        want = dy[at].double().t() @ x[at].double()
        bound = (2 * 48 + -(-c // 768) + 1) * U * want * (1 + 2.0 ** -10)
        if accumulate:
            want = want + base[e].double()
            bound = bound + U * want
        within(d_w[e], want, bound)
    assert int(status) == 0


@pytest.mark.parametrize("accumulate", [False, True])
def test_nvfp4(accumulate):
    g = gen(52)
    counts = [17024, 0, 128, 8192, 8320, 256, 100, 640]
    E, N, K = len(counts), 2176, 2176
    offsets, off, R_cap, live = slots(counts, spare=128)
    ops = []
    for H in (N, K):                    # positive codes, scales from 0.25 to 3.75
        codes = torch.randint(0, 256, (R_cap * H // 2,), generator=g, device="cuda").to(torch.uint8) & 0x77
        scales = torch.randint(0x28, 0x48, (R_cap * H // 16,), generator=g, device="cuda").to(torch.uint8)
        codes[off[-1] * H // 2:], scales[off[-1] * H // 16:] = 0xFF, 0xFF
        ops.append(dict(cw_codes=codes, cw_scales=scales,
                        cw_scale_enc=torch.rand(E, generator=g, device="cuda") * 3 + 0.5))
    base = torch.rand(E, N, K, generator=g, device="cuda") * 100 if accumulate else torch.full((E, N, K), NAN, device="cuda")
    status = nq.new_status("cuda")
    d_w = nq.ep_nvfp4_grouped_wgrad(ops[0], ops[1], N, K, offsets, E, d_w=base.clone(), accumulate=accumulate,
                                    status=status)
    for e in range(E):
        n = off[e + 1] - off[e]
        if n == 0:
            assert torch.equal(d_w[e], base[e] if accumulate else torch.zeros_like(base[e]))
            continue
        a, b = (columnwise_values(op, H, off, e) for op, H in zip(ops, (N, K)))
        want = a @ b.t()
        parts = -(-n // 8192)
        bound = (2 * 128 + parts + 4) * U * want * (1 + 2.0 ** -10)
        if accumulate:
            want = want + base[e].double()
            bound = bound + parts * U * want
        within(d_w[e], want, bound)
    assert int(status) == 0
