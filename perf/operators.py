"""Cases of the operators around the expert products of a MoE layer.

Each case names one operator, its direction and its sizes.  ``prepare`` makes
what a program holds before the call (tokens, a routing plan, packed weights,
output buffers), ``run`` makes the call -- in plain torch where ``own`` is
false, through ``nvfp4_quantization_gb300`` where it is true -- and ``exact``
computes the same outputs in 64 bits from the operator's definition.

  pack              tokens [T, H] -> expert rows, padding rows zero
  combine           expert rows -> tokens, weighted by the router
  combine_backward  token gradients -> row gradients and weight gradients
  swiglu            gated activation with its input kept in 8 bits, and its
                    backward pass from those 8 bits
  matvec            products of a few tokens with NVFP4 expert weights
"""
import math

import torch

own = False

ALIGN = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a prefill batch of a 16-expert top-2 layer entering its experts in BF16
        {"name": "pack_prefill", "op": "pack", "dtype": "bf16", "T": 4096, "H": 4096, "E": 16, "k": 2, "drop": 0.0},
        # a training batch of a 64-expert top-6 layer
        {"name": "pack_train", "op": "pack", "dtype": "bf16", "T": 16384, "H": 7168, "E": 64, "k": 6, "drop": 0.0},
        # one generated token: its eight expert outputs, still in slot order, become one row (the smallest call)
        {"name": "combine_token", "op": "combine", "dtype": "bf16", "T": 1, "H": 7168, "E": 256, "k": 8, "drop": 0.0,
         "slots": True, "weighted": True},
        # the way back of a training batch of 256 experts top-8
        {"name": "combine_train", "op": "combine", "dtype": "bf16", "T": 16384, "H": 7168, "E": 256, "k": 8,
         "drop": 0.0, "slots": False, "weighted": True},
        # a small ragged batch with capacity drops, gradients kept in FP32
        {"name": "combine_back_odd", "op": "combine_backward", "dtype": "f32", "T": 1021, "H": 1001, "E": 61, "k": 5,
         "drop": 0.1},
        # the gradient of the 256-expert batch: row gradients and the router's weight gradients (the largest)
        {"name": "combine_back_train", "op": "combine_backward", "dtype": "bf16", "T": 16384, "H": 7168, "E": 256,
         "k": 8, "drop": 0.0},
        # a short sequence through eight experts
        {"name": "swiglu_short", "op": "swiglu", "T": 200, "I": 512, "E": 8, "k": 2, "recompute": False},
        # a training batch of eight wide experts
        {"name": "swiglu_wide", "op": "swiglu", "T": 8192, "I": 4096, "E": 8, "k": 2, "recompute": False},
        # many narrow experts; the second product's weight gradient wants the activation again
        {"name": "swiglu_train", "op": "swiglu", "T": 16384, "I": 2048, "E": 64, "k": 6, "recompute": True},
        # one token through two of eight small experts: latency
        {"name": "matvec_small", "op": "matvec", "T": 1, "K": 1024, "N": 1024, "E": 8, "k": 2, "slots": False,
         "drop": 0.0},
        # one generated token through eight of 64 experts
        {"name": "matvec_token", "op": "matvec", "T": 1, "K": 4096, "N": 4096, "E": 64, "k": 8, "slots": False,
         "drop": 0.0},
        # a decode batch in which every expert has tokens, second product (one input row per slot)
        {"name": "matvec_batch", "op": "matvec", "T": 32, "K": 4096, "N": 4096, "E": 64, "k": 8, "slots": True,
         "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack", "combine", "combine_backward", "swiglu", "matvec"])
    E = _log(rng, 1, 256)
    k = rng.randint(1, min(8, E))
    if op in ("pack", "combine", "combine_backward"):
        H = _log(rng, 33, 7168)
        if rng.random() < 0.5:
            H = max(32, H // 32 * 32)
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "T": _log(rng, 1, 16384), "H": H, "E": E, "k": k,
             "drop": rng.choice([0.0, 0.0, 0.05, 0.3])}
        if c["dtype"] == "f32":
            c["T"] = min(c["T"], 4096)
        if op == "combine":
            c["slots"] = rng.random() < 0.3
            c["weighted"] = rng.random() < 0.7
        return c
    if op == "swiglu":
        return {"op": op, "T": _log(rng, 1, 8192), "I": 32 * _log(rng, 1, 128), "E": min(E, 64), "k": min(k, 6),
                "recompute": rng.random() < 0.5}
    E = _log(rng, 1, 64)
    return {"op": op, "T": _log(rng, 1, 32), "K": 32 * _log(rng, 2, 128), "N": _log(rng, 50, 4096), "E": E,
            "k": rng.randint(1, min(8, E)), "slots": rng.random() < 0.5, "drop": rng.choice([0.0, 0.0, 0.2])}


def _row_bytes(K):
    return (9 * K // 16 + 16 + 15) // 16 * 16


def work(case):
    """Least bytes and operations of one pass; padding rows are not counted."""
    op, T, k = case["op"], case["T"], case["k"]
    if op == "matvec":
        # with T tokens choosing uniformly, this many experts are in use
        used = case["E"] * (1.0 - (1.0 - k * (1.0 - case["drop"]) / case["E"]) ** T)
        xrows = T * k if case["slots"] else T
        nbytes = used * case["N"] * _row_bytes(case["K"]) + xrows * case["K"] * 2 + T * k * case["N"] * 2 + T * k * 4
        return {"bytes": nbytes, "flops": 2.0 * T * k * (1.0 - case["drop"]) * case["N"] * case["K"]}
    if op == "swiglu":
        n = T * k * case["I"]
        forward = 4 * n + 2 * n + 2 * n * 33 / 32
        backward = 2 * n + 2 * n * 33 / 32 + 4 * n + (2 * n if case["recompute"] else 0)
        return {"bytes": forward + backward, "flops": 20.0 * n}
    size = 2 if case["dtype"] == "bf16" else 4
    live = T * k * (1.0 - case["drop"])
    H = case["H"]
    if op == "pack":
        return {"bytes": (T + live) * H * size + T * k * 4, "flops": 0.0}
    if op == "combine":
        return {"bytes": (T + live) * H * size + T * k * (8 if case["weighted"] else 4), "flops": 2.0 * live * H}
    return {"bytes": (T + 2 * live) * H * size + T * k * 12, "flops": 3.0 * live * H}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _routing(T, E, k, drop, g):
    """Expert ids [T, k] (-1 = dropped) drawn with uneven loads, and router weights."""
    load = torch.randn(E, generator=g, device="cuda") * 0.5
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)))
    score, topk = (gumbel + load).topk(k, dim=1)
    weights = torch.softmax(score, dim=1).contiguous()
    if drop:
        gone = torch.rand(T, k, generator=g, device="cuda") < drop
        gone[T // 2] = True          # a token that lost every slot
        topk = torch.where(gone, -1, topk)
    return topk.to(torch.int32).contiguous(), weights


def _plan(topk, E):
    """Expert-contiguous rows, each expert's slot a multiple of ALIGN rows."""
    T, k = topk.shape
    flat = topk.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.argsort(key, stable=True)
    first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device="cuda")
    dest = torch.where(flat < 0, -1, offsets[key.clamp(max=E - 1)] + rank - first[key.clamp(max=E - 1)])
    to32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return {"offsets": to32(offsets), "counts": to32(counts), "dest": to32(dest), "T": T, "k": k, "E": E, "A": ALIGN,
            "R_cap": T * k + E * (ALIGN - 1), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _tokens(rows, cols, dtype, g, spread=0.5):
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(rows, 1, generator=g, device="cuda"))
    return x.to(dtype)


def _weights(E, N, K, g):
    """Gaussian weights as packed NVFP4 rows [E, N, S]: E2M1 codes, E4M3 scales
    of 16, and a trailer with the row's power-of-two scale."""
    S = _row_bytes(K)
    out = torch.zeros(E, N, S, dtype=torch.uint8, device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
        top = w.abs().amax(1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(top / 2688)))
        block = (w.view(N, K // 16, 16).abs().amax(2) / (6 * scale)).to(torch.float8_e4m3fn)
        unit = (block.float() * scale).clamp_min(1e-30).unsqueeze(2)
        v = (w.view(N, K // 16, 16) / unit).reshape(N, K)
        code = torch.bucketize(v.abs(), mid).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        out[e, :, : K // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
        out[e, :, K // 2: 9 * K // 16] = block.view(torch.uint8)
        trailer = torch.cat([scale, top], 1).contiguous().view(torch.uint8)
        out[e, :, S - 16: S - 8] = trailer
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    topk, weights = _routing(T, E, k, case.get("drop", 0.0), g)
    s = {"case": case, "topk": topk, "weights": weights, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "matvec":
        K, N = case["K"], case["N"]
        s["x"] = _tokens(T * k if case["slots"] else T, K, torch.bfloat16, g)
        s["w"] = _weights(E, N, K, g)
        s["y"] = torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda")
        return s
    p = s["plan"] = _plan(topk, E)
    R_cap = p["R_cap"]
    if op == "swiglu":
        I = case["I"]
        live = torch.zeros(R_cap, 1, device="cuda")
        live[p["dest"].long()] = 1.0
        s["x"] = (_tokens(R_cap, 2 * I, torch.float32, g) * live).to(torch.bfloat16)
        s["d_act"] = (1e-3 * _tokens(R_cap, I, torch.float32, g) * live).to(torch.bfloat16)
        s["act"] = torch.zeros(R_cap, I, dtype=torch.bfloat16, device="cuda")
        s["again"] = torch.zeros_like(s["act"]) if case["recompute"] else None
        s["d_x"] = torch.zeros(R_cap, 2 * I, dtype=torch.bfloat16, device="cuda")
        s["ckpt"] = torch.zeros(R_cap * 2 * I + R_cap * (2 * I // 32), dtype=torch.uint8, device="cuda")
        s["amax"] = torch.zeros(E, device="cuda")
        return s
    H, dtype = case["H"], DTYPES[case["dtype"]]
    if op == "pack":
        s["tokens"] = _tokens(T, H, dtype, g)
        s["rows"] = torch.zeros(R_cap, H, dtype=dtype, device="cuda")
    elif op == "combine":
        s["rows"] = _tokens(T * k if case["slots"] else R_cap, H, dtype, g)
        s["out"] = torch.zeros(T, H, dtype=dtype, device="cuda")
    else:
        s["rows"] = _tokens(R_cap, H, dtype, g)
        s["d_out"] = _tokens(T, H, dtype, g, spread=1.0) * 1e-3
        s["d_rows"] = torch.zeros(R_cap, H, dtype=dtype, device="cuda")
        s["d_weights"] = torch.zeros(T, k, device="cuda")
    return s


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------
def _plain_pack(s):
    p, x = s["plan"], s["tokens"]
    dest = p["dest"].long()
    rows = x.new_zeros(p["R_cap"] + 1, x.shape[1])          # the last row takes the dropped slots
    rows[torch.where(dest < 0, p["R_cap"], dest)] = x.repeat_interleave(p["k"], 0)
    return rows[: p["R_cap"]]


def _slot_rows(s):
    """Row of every slot [T, k], and whether the slot is live."""
    T, k = s["topk"].shape
    if s["case"].get("slots"):
        return torch.arange(T * k, device="cuda").view(T, k), s["topk"] >= 0
    dest = s["plan"]["dest"].view(T, k).long()
    return dest.clamp_min(0), dest >= 0


def _plain_combine(s):
    at, live = _slot_rows(s)
    v = s["rows"][at].float()
    if s["case"]["weighted"]:
        v = v * s["weights"].unsqueeze(2)
    return torch.where(live.unsqueeze(2), v, 0.0).sum(1).to(s["rows"].dtype)


def _plain_combine_backward(s):
    p, d_out = s["plan"], s["d_out"].float()
    at, live = _slot_rows(s)
    d_weights = torch.where(live, (s["rows"][at].float() * d_out.unsqueeze(1)).sum(2), 0.0)
    d_rows = s["rows"].new_zeros(p["R_cap"] + 1, d_out.shape[1])
    to = torch.where(live, at, p["R_cap"])
    d_rows[to] = (s["weights"].unsqueeze(2) * d_out.unsqueeze(1)).to(s["rows"].dtype)
    return d_rows[: p["R_cap"]], d_weights


def _plain_mx(x):
    """The values that MXFP8 blocks of 32 hold in place of x."""
    b = x.view(x.shape[0], -1, 32)
    frac, power = torch.frexp(b.abs().amax(2, keepdim=True))
    e = (power - 9 + (frac > 0.875)).clamp(-127, 127)          # max|b| <= 448 * 2^e
    v = torch.ldexp(b, -e)
    step = torch.frexp(v)[1].clamp_min(-5) - 4                 # four significant bits, least normal 2^-6
    v = torch.ldexp(torch.round(torch.ldexp(v, -step)), step)
    return torch.ldexp(v, e).view_as(x)


def _plain_swiglu(s):
    I, E, p = s["case"]["I"], s["case"]["E"], s["plan"]
    x, d = s["x"].float(), s["d_act"].float()
    row = torch.arange(x.shape[0], device="cuda")
    used = (row < p["offsets"][E]).unsqueeze(1)
    act = torch.where(used, x[:, :I] * torch.sigmoid(x[:, :I]) * x[:, I:], 0.0)
    kept = _plain_mx(x)
    g, u = kept[:, :I], kept[:, I:]
    sg = torch.sigmoid(g)
    d_x = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], 1)
    d_x = torch.where(used, d_x, 0.0)
    expert = torch.searchsorted(p["offsets"][1:].long(), row, right=True).clamp_max(E - 1)
    amax = torch.zeros(E, device="cuda").scatter_reduce(0, expert, d_x.abs().amax(1), "amax")
    out = {"act": act.to(torch.bfloat16), "d_x": d_x.to(torch.bfloat16), "amax": amax}
    if s["case"]["recompute"]:
        out["again"] = torch.where(used, g * sg * u, 0.0).to(torch.bfloat16)
    return out


def _decode(w, K):
    S = w.shape[-1]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    grid = torch.cat([grid, -grid])
    codes = w[..., : K // 2].int()
    v = torch.stack([grid[codes & 15], grid[codes >> 4]], -1).reshape(*w.shape[:-1], K // 16, 16)
    block = w[..., K // 2: 9 * K // 16].contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    row = w[..., S - 16: S - 12].contiguous().view(torch.float32)
    return (v * block).reshape(*w.shape[:-1], K) * row


def _plain_matvec(s):
    c = s["case"]
    T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
    slot_e = s["topk"].reshape(-1, 1).long()
    e = slot_e.squeeze(1).clamp_min(0)
    x = s["x"].float()
    if T * k <= E:                                             # few slots: only the experts they name
        xs = x if c["slots"] else x.repeat_interleave(k, 0)
        y = torch.bmm(_decode(s["w"][e], K), xs.unsqueeze(2)).squeeze(2)
        return torch.where(slot_e < 0, 0.0, y).to(torch.bfloat16)
    y = (x @ _decode(s["w"], K).view(E * N, K).t()).view(-1, E, N)
    slot = torch.arange(T * k, device="cuda")
    return torch.where(slot_e < 0, 0.0, y[slot if c["slots"] else slot // k, e]).to(torch.bfloat16)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"pack": _plain_pack, "combine": _plain_combine, "combine_backward": _plain_combine_backward,
                "swiglu": _plain_swiglu, "matvec": _plain_matvec}[op](s)
    import nvfp4_quantization_gb300 as nq
    if op == "matvec":
        return nq.ep_nvfp4_matvec(s["x"], s["w"], s["topk"], y=s["y"], status=s["status"])
    if op == "combine" and s["case"]["slots"]:
        return nq.ep_combine(s["rows"], topk_idx=s["topk"], weights=s["weights"] if s["case"]["weighted"] else None,
                             out=s["out"], status=s["status"])
    plan = nq.RoutePlan(**s["plan"])
    if op == "pack":
        return nq.ep_pack(s["tokens"], plan, rows=s["rows"])
    if op == "combine":
        return nq.ep_combine(s["rows"], plan, weights=s["weights"] if s["case"]["weighted"] else None, out=s["out"])
    if op == "combine_backward":
        return nq.ep_combine_backward(s["d_out"], plan, weights=s["weights"], rows=s["rows"], d_rows=s["d_rows"],
                                      d_weights=s["d_weights"])
    E = s["case"]["E"]
    nq.ep_swiglu(s["x"], plan.offsets, E, act=s["act"], ckpt=s["ckpt"], status=s["status"])
    s["amax"].zero_()
    nq.ep_swiglu_backward(s["d_act"], s["ckpt"], plan.offsets, E, d_x=s["d_x"], act=s["again"], expert_amax=s["amax"],
                          status=s["status"])
    out = {"act": s["act"], "d_x": s["d_x"], "amax": s["amax"]}
    if s["case"]["recompute"]:
        out["again"] = s["again"]
    return out


# ----------------------------------------------------------------------------
# 64 bits, from the definitions
# ----------------------------------------------------------------------------
def _e2m1_64(code):
    """Sign, two exponent bits (bias 1), one mantissa bit."""
    c = code.to(torch.int32)
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((exp - 1).double()))
    return torch.where(c >= 8, -mag, mag)


def _exact_matvec(s):
    c = s["case"]
    K, k, S = c["K"], c["k"], s["w"].shape[2]
    y = torch.zeros(c["T"] * k, c["N"], dtype=torch.float64, device="cuda")
    for e in sorted(set(s["topk"].reshape(-1).tolist()) - {-1}):
        w = s["w"][e]
        mat = torch.empty(c["N"], K, dtype=torch.float64, device="cuda")
        mat[:, 0::2] = _e2m1_64(w[:, : K // 2] & 15)
        mat[:, 1::2] = _e2m1_64(w[:, : K // 2] >> 4)
        for i in range(16):
            mat[:, i::16] *= w[:, K // 2: 9 * K // 16].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
        mat *= w[:, S - 16: S - 12].contiguous().view(torch.float32).double()
        for i in (s["topk"].reshape(-1) == e).nonzero().reshape(-1).tolist():
            y[i] = mat @ s["x"][i if c["slots"] else i // k].double()
    return y


def _exact_swiglu(s):
    I, E = s["case"]["I"], s["case"]["E"]
    off = s["plan"]["offsets"].tolist()
    R = off[E]
    out = {n: torch.zeros_like(s[n], dtype=torch.float64) for n in ("act", "d_x")}
    if s["case"]["recompute"]:
        out["again"] = torch.zeros_like(out["act"])
    amax = torch.zeros(E, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = off[e], min(off[e + 1], R)
        if a == b:
            continue
        x = s["x"][a:b].double()
        out["act"][a:b] = x[:, :I] / (1 + torch.exp(-x[:, :I])) * x[:, I:]
        blocks = x.reshape(-1, 32)
        top = blocks.abs().amax(1, keepdim=True).clamp_min(1e-300)
        unit = torch.exp2(torch.ceil(torch.log2(top / 448) - 1e-12).clamp(-127, 127))
        kept = ((blocks / unit).float().to(torch.float8_e4m3fn).float().double() * unit).reshape(x.shape)
        g, u = kept[:, :I], kept[:, I:]
        sig = 1 / (1 + torch.exp(-g))
        d = s["d_act"][a:b].double()
        out["d_x"][a:b, :I] = d * u * (sig + g * sig * (1 - sig))
        out["d_x"][a:b, I:] = d * g * sig
        amax[e] = out["d_x"][a:b].abs().max()
        if s["case"]["recompute"]:
            out["again"][a:b] = g * sig * u
    out["amax"] = amax
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, T, k = case["op"], case["T"], case["k"]
    if op == "matvec":
        return _exact_matvec(s)
    if op == "swiglu":
        return _exact_swiglu(s)
    index = s["topk"] if case.get("slots") else s["plan"]["dest"].view(T, k)
    out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
    wide = torch.zeros(s["plan"]["R_cap"], case["H"], dtype=torch.float64, device="cuda") if op != "combine" else None
    d_weights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):                                         # slot by slot
        t = (index[:, j] >= 0).nonzero().reshape(-1)
        r = t * k + j if case.get("slots") else index[t, j].long()
        if op == "pack":
            wide[r] = s["tokens"][t].double()
        elif op == "combine":
            w = s["weights"][t, j].double().unsqueeze(1) if case["weighted"] else 1.0
            out[t] += w * s["rows"][r].double()
        else:
            d = s["d_out"][t].double()
            wide[r] = s["weights"][t, j].double().unsqueeze(1) * d
            d_weights[t, j] = (s["rows"][r].double() * d).sum(1)
    return wide if op == "pack" else out if op == "combine" else (wide, d_weights)
