"""The MoE layer example: the operators together, forward, backward and decode,
against plain FP32 torch."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

# Relative errors in the 2-norm.  BF16 stages round at most 2^-8 each (four to
# the output, eight to d_x); E4M3 elements of the kept activation input are off
# by at most 2^-4 and 2^-4 / sqrt(3) in the mean square, in each of two factors;
# E2M1 weights with scales of 16 are off by a sixth of a block's largest at
# most, which for Gaussian blocks is a tenth in the mean square, in each of
# three products.
BF16, MX, FP4 = 8 * 2.0 ** -8, 3 * 2.0 ** -4, 3 * 0.1


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 128, 4, 2), (64, 512, 96, 16, 5)])
def test_moe_layer(T, H, I, E, k):
    import moe_layer
    err = moe_layer.main(T, H, I, E, k, seed=3)
    assert err["out"] <= BF16 and err["d_weights"] <= BF16
    assert err["d_x"] <= BF16 + MX and err["d_w1"] <= BF16 + MX and err["d_w2"] <= BF16 + MX
    assert err["decode"] <= BF16 + FP4
