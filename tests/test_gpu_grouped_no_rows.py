"""Buffers for no rows at all beside offsets that have some: as with any rows past
the capacity, the status says so and nothing is written."""
import pytest
import torch

import nvfp4_quantization_gb300 as nq
from test_gpu_grouped import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets,want", [([0, 0, 0], 0), ([0, 128, 256], nq.EP_DEV_ERR_CAPACITY),
                                          ([0, 0, 128], nq.EP_DEV_ERR_CAPACITY), ([0, 64, 64], nq.EP_DEV_ERR_BAD_EXPERT)])
def test_offsets_beside_no_rows(offsets, want):
    at, E, K, N = ints(offsets), 2, 128, 256
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")      # noqa: E731
    w4 = nq.ep_nvfp4_operand(u8(E, N, nq.row_bytes(K)), K)
    x4 = nq.ep_nvfp4_operand(u8(0, nq.row_bytes(K)), K)
    cw = lambda H: dict(cw_codes=u8(0), cw_scales=u8(0), cw_scale_enc=torch.ones(E, device="cuda"))   # noqa: E731
    status = nq.new_status("cuda")
    assert nq.ep_grouped_gemm(bf(0, K), bf(E, N, K), at, status=status).shape == (0, N)
    assert int(status) == want
    status.zero_()
    assert nq.ep_grouped_gemm(bf(0, N), bf(E, N, K), at, transpose=True, status=status).shape == (0, K)
    assert int(status) == want
    status.zero_()
    assert nq.ep_nvfp4_grouped_gemm(x4, w4, at, status=status).shape == (0, N)
    assert int(status) == want
    status.zero_()
    assert (nq.ep_grouped_wgrad(bf(0, N), bf(0, K), at, E, status=status) == 0).all()
    assert int(status) == want
    status.zero_()
    assert (nq.ep_nvfp4_grouped_wgrad(cw(N), cw(K), N, K, at, E, status=status) == 0).all()
    assert int(status) == want
    if want != nq.EP_DEV_ERR_BAD_EXPERT:      # (the operand only takes the end of the last slot)
        status.zero_()
        nq.ep_nvfp4_operand(u8(0, nq.row_bytes(K)), K, at, E, status=status)
        assert int(status) == want
