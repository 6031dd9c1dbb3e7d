"""A MoE layer around this library: one training step and one decode step.

Training (BF16): route plan -> pack -> first product -> gated activation with
its input kept in 8 bits -> second product -> combine, then the gradients back
through combine, the activation (from its checkpoint) and pack.  The
activation's backward also leaves each expert's amax, with which d_h goes
straight into the columnwise NVFP4 operand of the weight-gradient product.

Decode (NVFP4 weights): the same layer for a few tokens, straight from the
packed rows: products, activation, products, combine, four calls in all with
the routing left as ids.

The expert products of the training step are torch.matmul per expert: the
library prepares operands for a grouped GEMM but has none of its own.

    python examples/moe_layer.py [--tokens 2048] [--hidden 1024] [--inter 512] [--experts 8] [--topk 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_quantization_gb300 as nq  # noqa: E402


def grouped_matmul(rows, w, offsets, transpose=False):
    """rows [R_cap, K] of expert e times w[e]^T ([N, K]), or times w[e]."""
    out = rows.new_zeros(rows.shape[0], w.shape[2] if transpose else w.shape[1])
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            out[a:b] = rows[a:b] @ (w[e] if transpose else w[e].t())
    return out


class Layer:
    """Weights w1 [E, 2I, H] (gate rows, then up rows) and w2 [E, H, I], BF16,
    and the same weights packed once for decoding."""

    def __init__(self, w1, w2):
        self.w1, self.w2, self.E = w1, w2, w1.shape[0]
        self.w1_rows, self.w2_rows = nq.ep_nvfp4_pack_weights(w1), nq.ep_nvfp4_pack_weights(w2)
        self.status = nq.new_status(w1.device)   # what the decode steps report: EP_DEV_ERR_* bits

    def forward(self, x, topk, weights):
        """Output [T, H] and what the backward pass keeps."""
        plan = nq.ep_route_plan(topk, self.E)
        offsets = plan.offsets.tolist()          # torch.matmul wants them on the host
        rows = nq.ep_pack(x, plan)
        h = grouped_matmul(rows, self.w1, offsets)
        act, ckpt = nq.ep_swiglu(h, plan.offsets, self.E, status=plan.status)
        y = grouped_matmul(act, self.w2, offsets)
        return nq.ep_combine(y, plan, weights), (plan, offsets, rows, ckpt, y, weights)

    def backward(self, d_out, kept):
        """Gradients of x, the routing weights, w1 and w2, and the NVFP4
        columnwise operand of d_h."""
        plan, offsets, rows, ckpt, y, weights = kept
        d_y, d_weights = nq.ep_combine_backward(d_out, plan, weights, rows=y)
        d_act = grouped_matmul(d_y, self.w2, offsets, transpose=True)
        amax = torch.zeros(self.E, device=d_out.device)
        d_h, act = nq.ep_swiglu_backward(d_act, ckpt, plan.offsets, self.E, recompute=True, expert_amax=amax,
                                         status=plan.status)
        colwise = nq.ep_nvfp4_colwise_rht_bf16(d_h, plan.offsets, self.E, amax, status=plan.status)
        d_rows = grouped_matmul(d_h, self.w1, offsets, transpose=True)
        d_x = nq.ep_combine(d_rows, plan)        # the gradient of ep_pack
        d_w1, d_w2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        for e in range(self.E):
            a, b = offsets[e], offsets[e + 1]
            d_w1[e] = d_h[a:b].t() @ rows[a:b]
            d_w2[e] = d_y[a:b].t() @ act[a:b]
        return d_x, d_weights, d_w1, d_w2, colwise

    def decode(self, x, topk, weights):
        """Output [T, H] for a few tokens, from the packed weights.  A bad id, or
        anything else that the kernels find wrong, shows in self.status, which is
        read when the host waits for the GPU anyway."""
        h = nq.ep_nvfp4_matvec(x, self.w1_rows, topk, status=self.status)
        act, _ = nq.ep_swiglu(h, checkpoint=False, status=self.status)
        y = nq.ep_nvfp4_matvec(act, self.w2_rows, topk, status=self.status)
        return nq.ep_combine(y, topk_idx=topk, weights=weights, status=self.status)


def plain_layer(x, topk, weights, w1, w2):
    """The layer in plain torch, FP32."""
    out = torch.zeros(x.shape, device=x.device)
    for e in range(w1.shape[0]):
        t, j = (topk == e).nonzero(as_tuple=True)
        g, u = (x[t] @ w1[e].t()).chunk(2, dim=1)
        y = (torch.nn.functional.silu(g) * u) @ w2[e].t()
        out = out.index_add(0, t, weights[t, j].unsqueeze(1) * y)
    return out


def relative(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def main(T=2048, H=1024, I=512, E=8, k=2, seed=0):
    """Both steps, against plain torch; returns the relative errors."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    layer = Layer((rand(E, 2 * I, H) / H ** 0.5).to(torch.bfloat16), (rand(E, H, I) / I ** 0.5).to(torch.bfloat16))
    x, d_out = rand(T, H).to(torch.bfloat16), rand(T, H).to(torch.bfloat16)
    score, topk = rand(T, E).topk(k, dim=1)
    weights, topk = torch.softmax(score, 1), topk.to(torch.int32)
    topk[0, 0] = -1                              # a slot over capacity

    leaves = [t.float().requires_grad_() for t in (x, weights, layer.w1, layer.w2)]
    want = plain_layer(leaves[0], topk, leaves[1], leaves[2], leaves[3])
    want.backward(d_out.float())
    out, kept = layer.forward(x, topk, weights)
    grads = layer.backward(d_out, kept)
    err = {"out": relative(out, want)}
    for name, got, leaf in zip(("d_x", "d_weights", "d_w1", "d_w2"), grads, leaves):
        err[name] = relative(got, leaf.grad)

    few = slice(0, 4)                            # decoding: the weights' 4 bits are what is left of an error
    err["decode"] = relative(layer.decode(x[few], topk[few].contiguous(), weights[few].contiguous()), want[few])
    assert int(kept[0].status) == 0 and int(layer.status) == 0
    return err


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 2048), ("hidden", 1024), ("inter", 512), ("experts", 8), ("topk", 2)):
        p.add_argument(f"--{name}", type=int, default=default)
    a = p.parse_args()
    for name, e in main(a.tokens, a.hidden, a.inter, a.experts, a.topk).items():
        print(f"{name:10s} relative error against plain FP32 torch: {e:.2e}")
