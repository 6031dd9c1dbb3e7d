"""The MoE layer example reports what its decode calls find wrong."""
import os
import sys

import pytest
import torch

import nvfp4_quantization_gb300 as nq

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decode_shows_a_bad_expert_id():
    import moe_layer
    gen = torch.Generator(device="cuda")
    gen.manual_seed(50)
    E, H, I, T, k = 4, 128, 64, 3, 2
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")   # noqa: E731
    layer = moe_layer.Layer((rand(E, 2 * I, H) / 11).to(torch.bfloat16), (rand(E, H, I) / 8).to(torch.bfloat16))
    x, weights = rand(T, H).to(torch.bfloat16), torch.rand(T, k, generator=gen, device="cuda")
    topk = torch.tensor([[0, 3], [1, 2], [2, 0]], dtype=torch.int32, device="cuda")
    want = layer.decode(x, topk, weights)
    assert int(layer.status) == 0
    topk[1, 0] = E
    got = layer.decode(x, topk, weights)
    assert int(layer.status) == nq.EP_DEV_ERR_BAD_EXPERT
    assert torch.equal(got[[0, 2]], want[[0, 2]])
