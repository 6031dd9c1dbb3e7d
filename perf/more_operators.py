"""Cases of the expert products of a MoE layer: matrix products grouped by
expert, in BF16 and in NVFP4, with their gradients.

Each case names one operator, its direction and its sizes.  ``prepare`` makes
what a program holds before the call (expert rows, weights, quantised
operands, output buffers), ``run`` makes the call -- in plain torch where
``own`` is false, through ``nvfp4_quantization_gb300`` where it is true -- and
``exact`` computes the same outputs in 64 bits from the operator's definition.

  gemm          rows of expert e times W_e^T (BF16), or times W_e with
                ``transpose`` (the gradient of the rows)
  wgrad         d_w[e] = sum over e's rows of dy[r] x[r]^T (BF16 in)
  operand       packed NVFP4 rows -> the scales of a block-scaled product:
                block scales in 128 x 4 tiles, one FP32 scale a row
  nvfp4_gemm    the product of NVFP4 rows with NVFP4 weights
  nvfp4_wgrad   the weight gradient from the columnwise NVFP4 operands

Rows lie in expert order, each expert's slot a multiple of 128 rows and zero
behind its tokens; rows behind the last slot belong to nobody.
"""
import math

import torch

own = False

ALIGN = 128


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one token through two of eight small experts: latency (the smallest call)
        {"name": "gemm_token", "op": "gemm", "T": 1, "E": 8, "k": 2, "K": 1024, "N": 1024, "transpose": False,
         "drop": 0.0},
        # first product of a training batch, 64 experts top-6
        {"name": "gemm_train", "op": "gemm", "T": 16384, "E": 64, "k": 6, "K": 4096, "N": 4096, "transpose": False,
         "drop": 0.0},
        # the rows' gradient of a ragged batch with capacity drops, odd widths
        {"name": "gemm_back_odd", "op": "gemm", "T": 1021, "E": 61, "k": 5, "K": 1000, "N": 2056, "transpose": True,
         "drop": 0.1},
        # weight gradient of the same batch, handed to a BF16 reduction
        {"name": "wgrad_odd", "op": "wgrad", "T": 1021, "E": 61, "k": 5, "K": 2056, "N": 1000, "dtype": "bf16",
         "drop": 0.1},
        # weight gradient of a training batch of 16 experts top-2, kept in FP32
        {"name": "wgrad_train", "op": "wgrad", "T": 16384, "E": 16, "k": 2, "K": 4096, "N": 4096, "dtype": "f32",
         "drop": 0.0},
        # rows of one decoded token as a product's operand
        {"name": "operand_token", "op": "operand", "T": 1, "E": 64, "k": 8, "K": 4096, "drop": 0.0},
        # rows of a training batch of 64 experts top-6
        {"name": "operand_train", "op": "operand", "T": 16384, "E": 64, "k": 6, "K": 7168, "drop": 0.0},
        # a decode batch of 128 sequences, 8 of 64 experts: the weights are read once
        {"name": "nvfp4_gemm_decode", "op": "nvfp4_gemm", "T": 128, "E": 64, "k": 8, "K": 4096, "N": 4096, "drop": 0.0},
        # a short prompt, odd widths, capacity drops
        {"name": "nvfp4_gemm_odd", "op": "nvfp4_gemm", "T": 1021, "E": 61, "k": 5, "K": 1056, "N": 2056, "drop": 0.1},
        # a training batch of 64 experts top-6 (with gemm_train the largest)
        {"name": "nvfp4_gemm_train", "op": "nvfp4_gemm", "T": 16384, "E": 64, "k": 6, "K": 4096, "N": 4096,
         "drop": 0.0},
        # weight gradient of a short batch with drops
        {"name": "nvfp4_wgrad_short", "op": "nvfp4_wgrad", "T": 1021, "E": 16, "k": 4, "K": 1024, "N": 1152,
         "dtype": "bf16", "drop": 0.1},
        # weight gradient of the 64-expert training batch
        {"name": "nvfp4_wgrad_train", "op": "nvfp4_wgrad", "T": 16384, "E": 64, "k": 6, "K": 4096, "N": 2048,
         "dtype": "f32", "drop": 0.0},
    ]


_MOST_FLOPS = 3.2e12      # of the largest listed case
_MOST_WEIGHTS = 2 ** 30


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "wgrad", "operand", "nvfp4_gemm", "nvfp4_wgrad"])
    E = _log(rng, 1, 256)
    c = {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
         "drop": rng.choice([0.0, 0.0, 0.05, 0.3])}
    unit = {"gemm": 8, "wgrad": 8, "operand": 32, "nvfp4_gemm": 32, "nvfp4_wgrad": 128}[op]
    c["K"] = unit * _log(rng, max(1, 64 // unit), 7168 // unit)
    if op == "operand":
        return c
    unit = 8 if op == "nvfp4_gemm" else unit
    c["N"] = unit * _log(rng, max(1, 64 // unit), 7168 // unit)
    while E * c["K"] * c["N"] > _MOST_WEIGHTS:
        c["N"] = max(unit, c["N"] // 2 // unit * unit)
    while 2.0 * c["T"] * c["k"] * c["K"] * c["N"] > _MOST_FLOPS:
        c["T"] //= 2
    if op == "gemm":
        c["transpose"] = rng.random() < 0.5
    if op in ("wgrad", "nvfp4_wgrad"):
        c["dtype"] = rng.choice(["bf16", "f32"])
    return c


def _row_bytes(K):
    return (9 * K // 16 + 16 + 15) // 16 * 16


def work(case):
    """Least bytes and operations of one pass; padding rows are not counted."""
    op, E, K = case["op"], case["E"], case["K"]
    live = case["T"] * case["k"] * (1.0 - case["drop"])
    if op == "operand":
        return {"bytes": live * (2 * (K / 16) + 8), "flops": 0.0}
    N = case["N"]
    flops = 2.0 * live * N * K
    # with T tokens choosing uniformly, this many experts are in use
    used = E * (1.0 - (1.0 - case["k"] * (1.0 - case["drop"]) / E) ** case["T"])
    if op == "gemm":
        return {"bytes": 2 * (live * (K + N) + used * N * K), "flops": flops}
    if op == "nvfp4_gemm":
        return {"bytes": (live + used * N) * (9 * K / 16 + 4) + 2 * live * N, "flops": flops}
    rows = live * (N + K) * (2 if op == "wgrad" else 9 / 16)
    return {"bytes": rows + E * N * K * (2 if case["dtype"] == "bf16" else 4), "flops": flops}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _routing(case, g):
    """Expert ids [T, k] (-1 = dropped) drawn with uneven loads."""
    T, E, k = case["T"], case["E"], case["k"]
    load = torch.randn(E, generator=g, device="cuda") * 0.5
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)))
    topk = (gumbel + load).topk(k, dim=1)[1]
    if case["drop"]:
        topk = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, topk)
    return topk


def _slots(case, g):
    """Counts, offsets (device and host), capacity, and which rows hold a token."""
    T, E, k = case["T"], case["E"], case["k"]
    flat = _routing(case, g).reshape(-1)
    counts = torch.bincount(torch.where(flat < 0, E, flat), minlength=E + 1)[:E]
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    R_cap = T * k + E * (ALIGN - 1)
    row = torch.arange(R_cap, device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row, right=True).clamp_max(E - 1)
    live = row - offsets[expert] < counts[expert]
    return {"offsets": offsets.to(torch.int32), "counts": counts.to(torch.int32), "R_cap": R_cap, "live": live,
            "bounds": offsets.tolist()}


def _rows(live, width, g, spread=0.5):
    """BF16 rows, zero where nobody is."""
    x = torch.randn(live.shape[0], width, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(live.shape[0], 1, generator=g, device="cuda"))
    return (x * live.unsqueeze(1)).to(torch.bfloat16)


def _codes(v):
    """E2M1 codes of values in units of their scale, two to a byte, the even one low."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(v.abs(), mid).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _quantise(x):
    """x [n, K] -> packed NVFP4 rows [n, S]: codes, E4M3 scales of 16, a trailer
    that starts with the row's power-of-two scale and its largest magnitude."""
    n, K = x.shape
    S = _row_bytes(K)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-30) / 2688)))
    block = (x.view(n, K // 16, 16).abs().amax(2) / (6 * scale)).to(torch.float8_e4m3fn)
    unit = (block.float() * scale).clamp_min(1e-35).unsqueeze(2)
    out = torch.zeros(n, S, dtype=torch.uint8, device="cuda")
    out[:, : K // 2] = _codes((x.view(n, K // 16, 16) / unit).view(n, K))
    out[:, K // 2: 9 * K // 16] = block.view(torch.uint8)
    out[:, S - 16: S - 8] = torch.cat([scale, top], 1).contiguous().view(torch.uint8)
    return out


def _tiles(s):
    """Scales [M, Kb] (bytes) in tiles of 128 rows x 4, zero where a tile overhangs."""
    M, Kb = s.shape
    mt, kt = -(-M // 128), -(-Kb // 4)
    full = torch.zeros(mt * 128, kt * 4, dtype=torch.uint8, device="cuda")
    full[:M, :Kb] = s
    return full.view(mt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _row_scale(rows):
    S = rows.shape[-1]
    return rows[..., S - 16: S - 12].contiguous().view(torch.float32).squeeze(-1)


def _as_operand(rows, K):
    """Packed rows [M, S] or [E, N, S] as a product's operand: the codes where
    they are, the scales in tiles."""
    s = rows[..., K // 2: 9 * K // 16]
    tiles = _tiles(s) if rows.dim() == 2 else torch.cat([_tiles(e) for e in s])
    return {"rw_codes": rows[..., : K // 2], "rw_scales": tiles, "rw_row_scale": _row_scale(rows)}


def _columnwise(slots, H, g, spread):
    """The columnwise NVFP4 operand of transformed rows: per expert H columns of
    n_e codes, blocks of 16 along them, and one FP32 scale (values are
    code * block / scale)."""
    bounds, E = slots["bounds"], len(slots["bounds"]) - 1
    codes = torch.zeros(slots["R_cap"] * H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(slots["R_cap"] * H // 16, dtype=torch.uint8, device="cuda")
    enc = torch.ones(E, device="cuda")
    counts = slots["counts"].tolist()
    for e in range(E):
        a, n = bounds[e], bounds[e + 1] - bounds[e]
        if n == 0:
            continue
        y = torch.randn(H, n, generator=g, device="cuda")
        y *= torch.exp(spread * torch.randn(H, 1, generator=g, device="cuda"))
        y[:, (counts[e] + 15) // 16 * 16:] = 0
        enc[e] = 2688 / (2 * y.abs().amax())
        block = (y.view(H, n // 16, 16).abs().amax(2) * (enc[e] / 6)).to(torch.float8_e4m3fn)
        v = y.view(H, n // 16, 16) * enc[e] / block.float().clamp_min(1e-30).unsqueeze(2)
        codes[a * H // 2: (a + n) * H // 2] = _codes(v.view(H, n)).reshape(-1)
        scales[a * H // 16: (a + n) * H // 16] = _tiles(block.view(torch.uint8))
    return {"cw_codes": codes, "cw_scales": scales, "cw_scale_enc": enc}


def _weights(E, rows, cols, g):
    w = torch.empty(E, rows, cols, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(cols)
    return w


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, E, K, N = case["op"], case["E"], case["K"], case.get("N")
    s = _slots(case, g)
    s.update(case=case, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    R_cap = s["R_cap"]
    if op == "gemm":
        s["x"] = _rows(s["live"], K, g)
        s["w"] = _weights(E, K, N, g) if case["transpose"] else _weights(E, N, K, g)
        s["out"] = torch.zeros(R_cap, N, dtype=torch.bfloat16, device="cuda")
    elif op == "wgrad":
        s["x"] = _rows(s["live"], K, g)
        s["dy"] = 1e-3 * _rows(s["live"], N, g, spread=1.0)
    elif op == "operand":
        s["rows"] = _quantise(_rows(s["live"], K, g).float())
        s["scales"] = torch.zeros(-(-R_cap // 128) * -(-K // 64) * 512, dtype=torch.uint8, device="cuda")
        s["row_scale"] = torch.zeros(R_cap, device="cuda")
    elif op == "nvfp4_gemm":
        s["a"] = _as_operand(_quantise(_rows(s["live"], K, g).float()), K)
        w = torch.stack([_quantise(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)) for _ in range(E)])
        s["w"] = _as_operand(w, K)
        s["out"] = torch.zeros(R_cap, N, dtype=torch.bfloat16, device="cuda")
    else:
        s["x"], s["dy"] = _columnwise(s, K, g, 0.3), _columnwise(s, N, g, 0.3)
    if op in ("wgrad", "nvfp4_wgrad"):
        s["d_w"] = torch.zeros(E, N, K, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32,
                               device="cuda")
    return s


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------
def _slot_list(s):
    """The experts that have rows, and where."""
    b = s["bounds"]
    return [(e, slice(b[e], b[e + 1])) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _plain_gemm(s, x, weight):
    out = torch.zeros_like(s["out"])
    for e, at in _slot_list(s):
        out[at] = x(at) @ weight(e)
    return out


def _plain_wgrad(s, dy, x):
    d_w = torch.zeros_like(s["d_w"])
    for e, at in _slot_list(s):
        d_w[e] = dy(e, at) @ x(e, at)
    return d_w


def _untile(t, M, Kb):
    mt, kt = -(-M // 128), -(-Kb // 4)
    return t.view(mt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(mt * 128, kt * 4)[:M, :Kb].contiguous()


def _values(codes, scales):
    """Codes [n, K/2] and block scales [n, K/16] (bytes) as FP32 values."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    grid = torch.cat([grid, -grid])
    c = codes.int()
    v = torch.stack([grid[c & 15], grid[c >> 4]], -1).reshape(c.shape[0], -1, 16)
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(2)).reshape(c.shape[0], -1)


def _plain_nvfp4_gemm(s):
    K, N, R = s["case"]["K"], s["case"]["N"], s["bounds"][-1]
    a, w = s["a"], s["w"]
    x = _values(a["rw_codes"][:R], _untile(a["rw_scales"], s["R_cap"], K // 16)[:R]) * a["rw_row_scale"][:R].unsqueeze(1)
    tiles = w["rw_scales"].view(s["case"]["E"], -1)
    return _plain_gemm(s, lambda at: x[at],
                       lambda e: (_values(w["rw_codes"][e], _untile(tiles[e], N, K // 16))
                                  * w["rw_row_scale"][e].unsqueeze(1)).t())


def _plain_nvfp4_wgrad(s):
    def side(op, H):
        def of(e, at):
            n = at.stop - at.start
            c = op["cw_codes"][at.start * H // 2: at.stop * H // 2].view(H, n // 2)
            sc = _untile(op["cw_scales"][at.start * H // 16: at.stop * H // 16], H, n // 16)
            return _values(c, sc) / op["cw_scale_enc"][e]
        return of
    x = side(s["x"], s["case"]["K"])
    return _plain_wgrad(s, side(s["dy"], s["case"]["N"]), lambda e, at: x(e, at).t())


def _plain_operand(s):
    K, R = s["case"]["K"], s["bounds"][-1]
    scales, row_scale = torch.zeros_like(s["scales"]), torch.zeros_like(s["row_scale"])
    tiles = _tiles(s["rows"][:R, K // 2: 9 * K // 16])
    scales[: tiles.numel()] = tiles
    row_scale[:R] = _row_scale(s["rows"][:R])
    return scales.view(torch.float8_e4m3fn), row_scale


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "gemm":
            return _plain_gemm(s, lambda at: s["x"][at].float(),
                               (lambda e: s["w"][e].float()) if c["transpose"] else (lambda e: s["w"][e].float().t()))
        if op == "wgrad":
            return _plain_wgrad(s, lambda e, at: s["dy"][at].float().t(), lambda e, at: s["x"][at].float())
        return {"operand": _plain_operand, "nvfp4_gemm": _plain_nvfp4_gemm, "nvfp4_wgrad": _plain_nvfp4_wgrad}[op](s)
    import nvfp4_quantization_gb300 as nq
    E, offsets, status = c["E"], s["offsets"], s["status"]
    if op == "gemm":
        return nq.ep_grouped_gemm(s["x"], s["w"], offsets, transpose=c["transpose"], out=s["out"], status=status)
    if op == "wgrad":
        return nq.ep_grouped_wgrad(s["dy"], s["x"], offsets, E, counts=s["counts"], d_w=s["d_w"], status=status)
    if op == "operand":
        a = nq.ep_nvfp4_operand(s["rows"], c["K"], offsets, E, scales=s["scales"], row_scale=s["row_scale"],
                                status=status)
        return a["rw_scales"].view(torch.float8_e4m3fn), a["rw_row_scale"]
    if op == "nvfp4_gemm":
        return nq.ep_nvfp4_grouped_gemm(s["a"], s["w"], offsets, out=s["out"], status=status)
    return nq.ep_nvfp4_grouped_wgrad(s["dy"], s["x"], c["N"], c["K"], offsets, E, d_w=s["d_w"], status=status)


# ----------------------------------------------------------------------------
# 64 bits, from the definitions
# ----------------------------------------------------------------------------
def _e2m1_64(code):
    """Sign, two exponent bits (bias 1), one mantissa bit."""
    c = code.to(torch.int32)
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((exp - 1).double()))
    return torch.where(c >= 8, -mag, mag)


def _decode_64(codes, tiles, M, K):
    """[M, K] in units of the outer scale, from the tiled layout's formula."""
    v = torch.empty(M, K, dtype=torch.float64, device="cuda")
    v[:, 0::2] = _e2m1_64(codes & 15)
    v[:, 1::2] = _e2m1_64(codes >> 4)
    m = torch.arange(M, device="cuda").unsqueeze(1)
    b = torch.arange(K // 16, device="cuda").unsqueeze(0)
    at = (m // 128 * -(-K // 64) + b // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + b % 4
    scale = tiles[at].view(torch.float8_e4m3fn).to(torch.float32).double()
    for i in range(16):
        v[:, i::16] *= scale
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op, E, K, N = case["op"], case["E"], case["K"], case.get("N")
    b = s["bounds"]
    if op == "operand":
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        row_scale = torch.zeros(s["R_cap"], dtype=torch.float64, device="cuda")
        m = torch.arange(b[E], device="cuda")
        for j in range(K // 16):                               # one scale column after another
            at = (m // 128 * -(-K // 64) + j // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + j % 4
            scales[at] = s["rows"][: b[E], K // 2 + j].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
        S = s["rows"].shape[1]
        row_scale[: b[E]] = s["rows"][: b[E], S - 16: S - 12].contiguous().view(torch.float32).double().reshape(-1)
        return scales, row_scale
    if op in ("gemm", "nvfp4_gemm"):
        out = torch.zeros(s["R_cap"], N, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    if op == "nvfp4_gemm":
        a, wt = s["a"], s["w"]["rw_scales"].view(E, -1)
    for e in range(E):
        lo, hi = b[e], b[e + 1]
        if lo == hi:
            continue
        if op == "gemm":
            w = s["w"][e].double()
            out[lo:hi] = s["x"][lo:hi].double().matmul(w if case["transpose"] else w.t())
        elif op == "wgrad":
            out[e] = s["dy"][lo:hi].double().t().matmul(s["x"][lo:hi].double())
        elif op == "nvfp4_gemm":
            per = K // 64 if K % 64 == 0 else K // 64 + 1      # tiles of a block of 128 rows
            x = _decode_64(a["rw_codes"][lo:hi], a["rw_scales"][lo // 128 * per * 512:], hi - lo, K)
            w = _decode_64(s["w"]["rw_codes"][e], wt[e], N, K)
            y = x.matmul(w.t()) * s["w"]["rw_row_scale"][e].double()
            out[lo:hi] = y * a["rw_row_scale"][lo:hi].double().unsqueeze(1)
        else:
            n = hi - lo
            v = [_decode_64(s[o]["cw_codes"][lo * H // 2: hi * H // 2].view(H, n // 2),
                            s[o]["cw_scales"][lo * H // 16:], H, n) for o, H in (("dy", N), ("x", K))]
            out[e] = v[0].matmul(v[1].t()) / (s["dy"]["cw_scale_enc"][e].double() * s["x"]["cw_scale_enc"][e].double())
    return out
