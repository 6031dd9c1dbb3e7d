"""What the order of a product's sum depends on: the call's shape, and not where
the other slots were routed."""
import math

import pytest
import torch

import nvfp4_quantization_gb300 as nq
from test_gpu_layer_ops import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 16, 300, 4096), (8, 4, 6, 100, 1056), (16, 2, 5, 4099, 512),
                                       (60, 3, 7, 50, 2080), (300, 2, 9, 40, 544), (40, 16, 33, 21, 7168)])
def test_a_slot_does_not_depend_on_the_others(T, k, E, N, K):
    """The same slot's row, bit for bit, wherever the other slots go (and with
    them its group, its column and the warps that compute it)."""
    g = gen(72)
    w = torch.randn(E, N, K, generator=g, device="cuda") / math.sqrt(K)
    w_rows = nq.ep_nvfp4_pack_weights(w.to(torch.bfloat16))
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    t, j, e = T // 2, k - 1, E // 2
    kept = []
    for i in range(8):
        topk = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        if i == 0:
            topk.fill_(-1)
        if i == 1:
            topk.fill_(e)
        topk[t, j] = e
        kept.append(nq.ep_nvfp4_matvec(x, w_rows, topk)[t * k + j])
    assert kept[0].any() and all(torch.equal(v, kept[0]) for v in kept[1:])
