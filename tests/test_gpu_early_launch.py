"""Calls that start while the ones before them still run: what they read has to
be what those wrote, not what lay there when they started."""
import pytest
import torch

import nvfp4_quantization_gb300 as nq

pytestmark = pytest.mark.gpu


def test_receive_with_a_given_amax_two_calls_behind_the_plan():
    """The plan is made by the call before last, and the call between lets the
    receive start as soon as it has started itself: the offsets in the shared
    plan are then still those of the routing before."""
    T, H, E, k = 4000, 512, 16, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    R_cap = nq.rows_capacity(T, k, E)
    status, ws = nq.new_status("cuda"), nq.new_route_workspace(T, k, E, "cuda")
    routings = []
    for skew in (0.0, 3.0, -3.0):
        load = torch.linspace(-1, 1, E, device="cuda") * skew
        topk = (torch.randn(T, E, generator=g, device="cuda") + load).topk(k, dim=1)[1].to(torch.int32).contiguous()
        amax = torch.empty(E, device="cuda")
        plan, rows = nq.ep_nvfp4_dispatch(x, topk, E, expert_amax=amax)
        torch.cuda.synchronize()
        want = nq.ep_nvfp4_direct_receive(rows, H, plan.offsets, E, swizzled=True)
        torch.cuda.synchronize()
        routings.append((topk, rows, amax, want, int(plan.offsets[-1]), nq.alloc_grouped(R_cap, H, E, "cuda")))
    assert len({r[4] for r in routings}) > 1 or len({tuple(r[2].tolist()) for r in routings}) == 3
    plan = nq.ep_route_plan(routings[0][0], E, status=status, workspace=ws)
    between = torch.empty(R_cap, H, dtype=torch.bfloat16, device="cuda")
    for turn in range(10):
        for topk, rows, amax, want, R, out in routings:
            out["cw_codes"].zero_()
            out["rw_scales"].zero_()
            nq.ep_route_plan(topk, E, plan=plan, workspace=ws)
            nq.ep_pack(x, plan, rows=between)
            nq.ep_nvfp4_direct_receive(rows, H, plan.offsets, E, out=out, swizzled=True, expert_amax=amax,
                                       status=status)
        for topk, rows, amax, want, R, out in routings:
            for name, n in (("cw_codes", R * H // 2), ("cw_scales", R * H // 16), ("amax_col", E), ("cw_scale_enc", E)):
                assert torch.equal(out[name][:n], want[name][:n]), (turn, name)
            for name in ("rw_codes", "rw_scales", "rw_row_scale"):
                assert torch.equal(out[name][:R], want[name][:R]), (turn, name)
    assert int(status) == 0
