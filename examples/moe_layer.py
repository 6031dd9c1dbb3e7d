"""A MoE layer around this library: training steps and a decode step.

Training (BF16): route plan -> pack -> first product -> gated activation with
its input kept in 8 bits -> second product -> combine, then the gradients back
through combine, the activation (from its checkpoint) and pack, and those of
the weights.  The activation's backward also leaves each expert's amax, with
which d_h goes straight into the columnwise NVFP4 operand of a weight gradient.
Nothing is copied to the host: the expert offsets stay where the plan put them.

Training (NVFP4): the same step with every product in NVFP4.  Tokens are
dispatched as packed rows; the direct receive makes the rowwise operand of the
product and the columnwise one of the weight gradient; gradients are rounded
stochastically.

Decode (NVFP4 weights): the same layer for a few tokens, straight from the
packed rows: products, activation, products, combine, four calls in all with
the routing left as ids.

    python examples/moe_layer.py [--tokens 2048] [--hidden 1024] [--inter 512] [--experts 8] [--topk 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_quantization_gb300 as nq  # noqa: E402


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
        rows = nq.ep_pack(x, plan)
        h = nq.ep_grouped_gemm(rows, self.w1, plan.offsets, status=plan.status)
        act, ckpt = nq.ep_swiglu(h, plan.offsets, self.E, status=plan.status)
        y = nq.ep_grouped_gemm(act, self.w2, plan.offsets, status=plan.status)
        return nq.ep_combine(y, plan, weights), (plan, rows, ckpt, y, weights)

    def backward(self, d_out, kept):
        """Gradients of x, the routing weights, w1 and w2, and the NVFP4
        columnwise operand of d_h."""
        plan, rows, ckpt, y, weights = kept
        offsets, st = plan.offsets, plan.status
        d_y, d_weights = nq.ep_combine_backward(d_out, plan, weights, rows=y)
        d_act = nq.ep_grouped_gemm(d_y, self.w2, offsets, transpose=True, status=st)
        amax = torch.zeros(self.E, device=d_out.device)
        d_h, act = nq.ep_swiglu_backward(d_act, ckpt, offsets, self.E, recompute=True, expert_amax=amax, status=st)
        colwise = nq.ep_nvfp4_colwise_rht_bf16(d_h, offsets, self.E, amax, status=st)
        d_rows = nq.ep_grouped_gemm(d_h, self.w1, offsets, transpose=True, status=st)
        d_x = nq.ep_combine(d_rows, plan)        # the gradient of ep_pack
        d_w1 = nq.ep_grouped_wgrad(d_h, rows, offsets, self.E, counts=plan.counts, status=st)
        d_w2 = nq.ep_grouped_wgrad(d_y, act, offsets, self.E, counts=plan.counts, status=st)
        return d_x, d_weights, d_w1, d_w2, colwise

    def decode(self, x, topk, weights):
        """Output [T, H] for a few tokens, from the packed weights.  A bad id, or
        anything else that the kernels find wrong, shows in self.status, which is
        read when the host waits for the GPU anyway."""
        h = nq.ep_nvfp4_matvec(x, self.w1_rows, topk, status=self.status)
        act, _ = nq.ep_swiglu(h, checkpoint=False, status=self.status)
        y = nq.ep_nvfp4_matvec(act, self.w2_rows, topk, status=self.status)
        return nq.ep_combine(y, topk_idx=topk, weights=weights, status=self.status)


class Nvfp4Layer:
    """The same layer with every product in NVFP4 (H and I multiples of 128).
    The weights are packed as they are and transposed, for the two directions."""

    def __init__(self, w1, w2):
        self.E, self.I = w2.shape[0], w2.shape[2]
        operand = lambda w: nq.ep_nvfp4_operand(nq.ep_nvfp4_pack_weights(w), w.shape[2], copy_codes=True)   # noqa: E731
        self.w1, self.w2 = operand(w1), operand(w2)
        self.w1_t, self.w2_t = (operand(w.transpose(1, 2).contiguous()) for w in (w1, w2))

    def receive(self, rows, plan, rounding=nq.EP_ROUND_RNE, seed=0):
        """Both operands of BF16 rows that are in expert order already."""
        packed = nq.ep_nvfp4_pack_weights(rows.unsqueeze(0), rounding=rounding, seed=seed)[0]
        return nq.ep_nvfp4_direct_receive(packed, rows.shape[1], plan.offsets, self.E, rounding=rounding, seed=seed,
                                          swizzled=True, status=plan.status)

    def forward(self, x, topk, weights):
        amax = torch.empty(self.E, device=x.device)
        plan, packed = nq.ep_nvfp4_dispatch(x, topk, self.E, expert_amax=amax)
        at, st = plan.offsets, plan.status
        rows = nq.ep_nvfp4_direct_receive(packed, x.shape[1], at, self.E, expert_amax=amax, swizzled=True, status=st)
        h = nq.ep_nvfp4_grouped_gemm(rows, self.w1, at, status=st)
        act = torch.zeros(plan.R_cap, self.I, dtype=torch.bfloat16, device=x.device)   # finite behind the slots too
        _, ckpt = nq.ep_swiglu(h, at, self.E, act=act, status=st)
        act = self.receive(act, plan)
        y = nq.ep_nvfp4_grouped_gemm(act, self.w2, at, status=st)
        return nq.ep_combine(y, plan, weights), (plan, rows, ckpt, act, y, weights)

    def backward(self, d_out, kept, seed=0):
        plan, rows, ckpt, act, y, weights = kept
        at, st, H, I = plan.offsets, plan.status, d_out.shape[1], self.I
        zeros = lambda n: torch.zeros(plan.R_cap, n, dtype=torch.bfloat16, device=d_out.device)   # noqa: E731
        d_y, d_weights = nq.ep_combine_backward(d_out, plan, weights, rows=y, d_rows=zeros(H))
        d_y = self.receive(d_y, plan, nq.EP_ROUND_SR, seed)
        d_act = nq.ep_nvfp4_grouped_gemm(d_y, self.w2_t, at, status=st)
        amax = torch.zeros(self.E, device=d_out.device)
        d_h, _ = nq.ep_swiglu_backward(d_act, ckpt, at, self.E, d_x=zeros(2 * I), expert_amax=amax, status=st)
        columns = nq.ep_nvfp4_colwise_rht_bf16(d_h, at, self.E, amax, rounding=nq.EP_ROUND_SR, seed=seed, swizzled=True,
                                               status=st)
        packed = nq.ep_nvfp4_pack_weights(d_h.unsqueeze(0), rounding=nq.EP_ROUND_SR, seed=seed + 1)[0]
        d_rows = nq.ep_nvfp4_grouped_gemm(nq.ep_nvfp4_operand(packed, 2 * I, at, self.E, status=st), self.w1_t, at,
                                          status=st)
        d_x = nq.ep_combine(d_rows, plan)
        d_w1 = nq.ep_nvfp4_grouped_wgrad(columns, rows, 2 * I, H, at, self.E, status=st)
        d_w2 = nq.ep_nvfp4_grouped_wgrad(d_y, act, H, I, at, self.E, status=st)
        return d_x, d_weights, d_w1, d_w2


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
    """The steps, against plain torch; returns the relative errors."""
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

    if H % 128 == 0 and I % 128 == 0:
        layer = Nvfp4Layer(layer.w1, layer.w2)
        out, kept = layer.forward(x, topk, weights)
        grads = layer.backward(d_out, kept, seed)
        err["out_nvfp4"] = relative(out, want)
        for name, got, leaf in zip(("d_x", "d_weights", "d_w1", "d_w2"), grads, leaves):
            err[name + "_nvfp4"] = relative(got, leaf.grad)
        assert int(kept[0].status) == 0
    return err


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 2048), ("hidden", 1024), ("inter", 512), ("experts", 8), ("topk", 2)):
        p.add_argument(f"--{name}", type=int, default=default)
    a = p.parse_args()
    for name, e in main(a.tokens, a.hidden, a.inter, a.experts, a.topk).items():
        print(f"{name:15s} relative error against plain FP32 torch: {e:.2e}")
