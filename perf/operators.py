"""Timed cases of the MXFP4 and expert-routing operators.

Each case is one pass through one operator: ``prepare`` makes what a program
holds before the call, ``run`` makes the call (in plain torch operations, or
through the package where ``own`` is set), ``exact`` computes the same outputs
in 64 bits from the definitions.
"""
import math

import torch

own = False

BLOCK = 32                                      # values per E8M0 scale
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the activation of a verify step, made 4-bit and read back
        {"name": "quantize verify activation bf16 8x5120", "op": "quantize", "rows": 8, "K": 5120, "dtype": "bf16"},
        # encoding one weight matrix of a dense layer from its fp32 master copy
        {"name": "quantize weights fp32 17408x5120", "op": "quantize", "rows": 17408, "K": 5120, "dtype": "fp32"},
        # one projection of a batch-1 decode step
        {"name": "gemv M1 5120->5120", "op": "gemv", "M": 1, "K": 5120, "N": 5120, "silu": False},
        # the MLP's first product for eight verified tokens
        {"name": "gemv M8 5120->2x17408 silu", "op": "gemv", "M": 8, "K": 5120, "N": 34816, "silu": True},
        # a short prompt of odd length through one projection
        {"name": "gemm 333 tokens 5120->5120", "op": "gemm", "M": 333, "K": 5120, "N": 5120, "silu": False},
        # a long prompt through the MLP's first product
        {"name": "gemm 8192 tokens 5120->2x17408 silu", "op": "gemm", "M": 8192, "K": 5120, "N": 34816, "silu": True},
        # experts' first product for a small batch: few rows per expert, some experts without any, padded tokens
        {"name": "grouped E64 61 tokens 4096->2x1024 silu", "op": "grouped", "M": 61, "top_k": 8, "E": 64, "K": 4096,
         "N": 2048, "silu": True, "gather": True, "empty": 0.05},
        # experts' second product of a long prompt
        {"name": "grouped E64 4096 tokens 2048->4096", "op": "grouped", "M": 4096, "top_k": 8, "E": 64, "K": 2048,
         "N": 4096, "silu": False, "gather": False, "empty": 0.0},
        # a verify step's tokens put in expert order
        {"name": "dispatch 8 tokens top8 of 256 H6144", "op": "dispatch", "M": 8, "top_k": 8, "E": 256, "H": 6144,
         "dtype": "bf16", "train": False, "empty": 0.0},
        # a training step's tokens put in expert order, and the gradient back
        {"name": "dispatch 4099 tokens top8 of 256 H6144 train", "op": "dispatch", "M": 4099, "top_k": 8, "E": 256,
         "H": 6144, "dtype": "bf16", "train": True, "empty": 0.0},
        # the experts' rows of a verify step added up
        {"name": "combine 8 tokens top8 of 256 H6144", "op": "combine", "M": 8, "top_k": 8, "E": 256, "H": 6144,
         "dtype": "bf16", "train": False, "empty": 0.0},
        # the same for a training step, with padded tokens, and both gradients
        {"name": "combine 4099 tokens top8 of 256 H6144 train", "op": "combine", "M": 4099, "top_k": 8, "E": 256,
         "H": 6144, "dtype": "bf16", "train": True, "empty": 0.1},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemv", "gemm", "grouped", "dispatch", "combine"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 12000), "K": 32 * _log_int(rng, 1, 200),
                "dtype": rng.choice(["bf16", "fp32"])}
    if op == "gemv":
        M = rng.randint(1, 16)
        K = 32 * _log_int(rng, 4, 69632 // M // 32)
        silu = rng.random() < 0.5
        N = _log_int(rng, 16, min(30000, 170_000_000 // K))
        return {"op": op, "M": M, "K": K, "N": N + N % 2, "silu": silu}
    if op == "gemm":
        K = 128 * rng.randint(1, 40)
        N = _log_int(rng, 64, 16000)
        return {"op": op, "M": _log_int(rng, 1, 6000), "K": K, "N": N + N % 2, "silu": rng.random() < 0.5}
    E = rng.choice([8, 16, 60, 64, 128, 256])
    top_k = rng.randint(1, 8)
    empty = rng.choice([0.0, 0.0, 0.1, 0.5])
    if op == "grouped":
        K = 128 * rng.randint(1, 24)
        N = _log_int(rng, 64, min(4096, 400_000_000 // (E * K)))
        return {"op": op, "M": _log_int(rng, 1, 3000), "top_k": top_k, "E": E, "K": K, "N": N + N % 2,
                "silu": rng.random() < 0.5, "gather": rng.random() < 0.5, "empty": empty}
    return {"op": op, "M": _log_int(rng, 1, 4000), "top_k": top_k, "E": E, "H": 8 * rng.randint(16, 700),
            "dtype": rng.choice(["bf16", "bf16", "fp32"]), "train": rng.random() < 0.6, "empty": empty}


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        # read the input, write codes and scales, write the values back
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["rows"] * c["K"]
        return {"bytes": n * e * 2 + n // 2 + n // 32, "flops": 0}
    if op in ("gemv", "gemm"):
        out = c["N"] // 2 if c["silu"] else c["N"]
        return {"bytes": c["N"] * (c["K"] // 2 + c["K"] // 32) + 2 * c["M"] * (c["K"] + out),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    P = c["M"] * c["top_k"]
    rows = int(P * (1.0 - c["empty"]))              # pairs that have an expert
    if op == "grouped":
        out = c["N"] // 2 if c["silu"] else c["N"]
        # experts that get a row when the rows fall evenly
        used = c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** rows)
        src = min(rows, c["M"]) if c["gather"] else rows
        return {"bytes": int(used * c["N"] * (c["K"] // 2 + c["K"] // 32)) + 2 * src * c["K"] + 2 * rows * out + 4 * P,
                "flops": 2 * rows * c["N"] * c["K"]}
    e = 2 if c["dtype"] == "bf16" else 4
    row = c["H"] * e
    tok = c["M"] * row
    if op == "dispatch":
        b = 4 * P + 8 * P + 4 * c["E"] + tok + P * row
        return {"bytes": b + (rows * row + tok if c["train"] else 0), "flops": 0}
    b = rows * row + tok + 8 * P
    # backward: the rows are read once for both directions, dy read, dys and dw written
    return {"bytes": b + (tok + P * row + 4 * P if c["train"] else 0), "flops": (4 if c["train"] else 2) * rows * c["H"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _activation(rows, K, g, dtype=torch.bfloat16):
    """N(0,1) with a few outlier channels, as activations of trained models have."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    ch = torch.randint(0, K, (2,), generator=g, device="cuda")
    x[:, ch] *= 20.0
    return x.to(dtype)


def _weights(shape, g):
    """0.02 N(0,1), quantised: packed codes [..., K/2] and scale bytes [..., K/32]."""
    n, K = math.prod(shape[:-1]), shape[-1]
    codes = torch.empty((n, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, K // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for i in range(0, n, step):
        w = 0.02 * torch.randn((min(step, n - i), K), generator=g, device="cuda")
        codes[i:i + step], scales[i:i + step] = _quantize(w)
    return codes.view(*shape[:-1], K // 2), scales.view(*shape[:-1], K // BLOCK)


def _topk_ids(c, g):
    """top_k distinct experts per token from noisy popularity; `empty` of the tokens are padding (-1)."""
    E, k = c["E"], c["top_k"]
    pop = 0.5 * torch.randn((1, E), generator=g, device="cuda")
    ids = torch.topk(pop + torch.randn((c["M"], E), generator=g, device="cuda"), k, dim=1).indices.to(torch.int32)
    pad = torch.rand((c["M"], 1), generator=g, device="cuda") < c["empty"]
    return torch.where(pad, torch.full_like(ids, -1), ids).contiguous()


def prepare(case, seed):
    c, op, g = case, case["op"], _gen(seed)
    s = dict(c)
    dt = torch.float32 if c.get("dtype") == "fp32" else torch.bfloat16
    if op == "quantize":
        s["x"] = _activation(c["rows"], c["K"], g, dt)
    elif op in ("gemv", "gemm"):
        s["x"] = _activation(c["M"], c["K"], g)
        s["w"], s["ws"] = _weights((c["N"], c["K"]), g)
    else:
        P = c["M"] * c["top_k"]
        s["ids"] = _topk_ids(c, g)
        if op != "dispatch":                        # later steps are given the order that the sort made
            s["order"], s["inverse"], s["offsets"] = _sort(s["ids"], c["E"])
        if op == "grouped":
            s["x"] = _activation(c["M"] if c["gather"] else P, c["K"], g)
            s["w"], s["ws"] = _weights((c["E"], c["N"], c["K"]), g)
            # the longest run of rows of one expert, for the plain form's padded layout
            s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        else:
            s["x"] = torch.randn((c["M"] if op == "dispatch" else P, c["H"]), generator=g, device="cuda").to(dt)
            if op == "combine":
                s["topk_w"] = torch.softmax(torch.randn((c["M"], c["top_k"]), generator=g, device="cuda"), 1)
            if c["train"]:
                s["dy"] = torch.randn((P if op == "dispatch" else c["M"], c["H"]), generator=g, device="cuda").to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantize(x):
    """Packed E2M1 codes and E8M0 scale bytes of blocks of 32 values."""
    v = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp_min(0)      # floor(log2 amax) - 2, biased by 127
    byte = torch.where(amax == 0, 127, byte)
    a = v.abs() * ((254 - byte) << 23).view(torch.float32)        # times 2^(127 - byte): exact
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), byte.squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """The fp32 values of packed codes [..., K/2] and scale bytes [..., K/32]."""
    level = torch.tensor(LEVELS, device=codes.device)
    table = torch.cat([level, -level])
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, BLOCK)
    b = scales.to(torch.int32)
    s = torch.where(b == 0, 1 << 22, b << 23).view(torch.float32)
    return (table[nib.to(torch.int32)] * s.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _epilogue(y, silu):
    if silu:
        gate, up = y.chunk(2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y


def _sort(ids, E):
    """order [P], inverse [P], offsets [E+1] of the (token, slot) pairs by expert; -1 marks no expert."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    count = (key.unsqueeze(0) == torch.arange(E, device=ids.device).unsqueeze(1)).sum(1)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    row = torch.arange(flat.numel(), device=ids.device)
    inverse = torch.empty_like(row)
    inverse[order] = row
    inverse = torch.where(flat < 0, -1, inverse)
    order = torch.where(row < offsets[-1], order, -1)
    return order.to(torch.int32), inverse.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def _gather(x, order, top_k):
    """Rows x[order / top_k], zero where order is -1."""
    rows = x[order.clamp_min(0).long() // top_k]
    return torch.where((order < 0).unsqueeze(1), torch.zeros((), dtype=x.dtype, device=x.device), rows)


def _sum_back(rows, inverse, w):
    """sum_s w[m,s] rows[inverse[m,s]] in fp32, rounded to the rows' type."""
    picked = rows[inverse.clamp_min(0).long()].float()
    w = torch.where(inverse < 0, 0.0, w)
    return (picked * w.unsqueeze(-1)).sum(1).to(rows.dtype)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _values(*_quantize(s["x"])).to(s["x"].dtype)
    if op == "gemv":
        return _epilogue(s["x"].float() @ _values(s["w"], s["ws"]).t(), s["silu"]).to(torch.bfloat16)
    if op == "gemm":
        return _epilogue(_values(*_quantize(s["x"])) @ _values(s["w"], s["ws"]).t(), s["silu"]).to(torch.bfloat16)
    if op == "grouped":
        xv = _values(*_quantize(s["x"]))
        order, offsets = s["order"], s["offsets"]
        if s["gather"]:
            xv = _gather(xv, order, s["top_k"])
        # every expert's rows side by side, padded to the longest run
        row = offsets[:-1].long().unsqueeze(1) + torch.arange(s["longest"], device=xv.device)
        has = row < offsets[1:].unsqueeze(1)
        wt = _values(s["w"], s["ws"]).transpose(1, 2)
        y = _epilogue(torch.bmm(xv[row.clamp_max(xv.shape[0] - 1)], wt), s["silu"]).to(torch.bfloat16)
        out = y.new_zeros((order.shape[0], y.shape[2]))
        out[row[has]] = y[has]
        return out
    if op == "dispatch":
        order, inverse, offsets = _sort(s["ids"], s["E"])
        got = {"xs": _gather(s["x"], order, s["top_k"]), "order": order, "inverse": inverse, "offsets": offsets}
        if s["train"]:
            got["dx"] = _sum_back(s["dy"], inverse, torch.ones((), device=inverse.device))
        return got
    inverse, order, w = s["inverse"], s["order"], s["topk_w"]
    got = {"y": _sum_back(s["x"], inverse, w)}
    if s["train"]:
        dy = s["dy"].float()
        wr = torch.where(order < 0, 0.0, w.reshape(-1)[order.clamp_min(0).long()])
        got["dys"] = (_gather(dy, order, s["top_k"]) * wr.unsqueeze(1)).to(s["dy"].dtype)
        dot = (s["x"][inverse.clamp_min(0).long()].float() * dy.unsqueeze(1)).sum(-1)
        got["dw"] = torch.where(inverse < 0, 0.0, dot)
    return got


def _package(s):
    import quantized_moe_weight_amd as pq
    op = s["op"]
    if op == "quantize":
        return pq.dequantize_mxfp4(*pq.quantize_mxfp4(s["x"]), dtype=s["x"].dtype)
    epi = pq.EPI_SILU_MUL if s.get("silu") else pq.EPI_NONE
    if op == "gemv":
        return pq.gemv_mxfp4(s["x"], s["w"], s["ws"], epi)
    if op == "gemm":
        return pq.gemm_mxfp4(s["x"], s["w"], s["ws"], epi)
    if op == "dispatch":
        plan = pq.moe_sort(s["ids"], s["E"])
        got = {"xs": pq.moe_dispatch(s["x"], plan), "order": plan.order, "inverse": plan.inverse,
               "offsets": plan.offsets}
        if s["train"]:
            got["dx"] = pq.moe_dispatch_grad(s["dy"], plan)
        return got
    plan = pq.MoePlan(s["order"], s["inverse"], s["offsets"])
    if op == "grouped":
        return pq.gemm_mxfp4_grouped(s["x"], s["w"], s["ws"], plan, epi, gather=s["gather"])
    got = {"y": pq.moe_combine(s["x"], plan, s["topk_w"])}
    if s["train"]:
        got["dys"], got["dw"] = pq.moe_combine_grad(s["dy"], s["x"], plan, s["topk_w"])
    return got


def run(state):
    return _package(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# 64-bit results from the definitions
# ---------------------------------------------------------------------------
def _fake_quant64(x):
    """The values that x takes in blocks of 32 under a power-of-two scale: the nearest of the sixteen levels,
    the one with the even code where two are equally near."""
    v = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)                         # top = m 2^e with 0.5 <= m < 1
    scale = torch.ldexp(torch.ones_like(top), (e - 3).clamp(-127, 127))
    a = v.abs() / scale
    lv = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    # the largest level below a, and the next one
    lo = (torch.bucketize(a, lv, right=True) - 1).clamp(0, 6)
    dlo, dhi = a - lv[lo], lv[lo + 1] - a
    up = (dhi < dlo) | ((dhi == dlo) & (lo % 2 == 1))
    q = lv[lo + up] * scale
    return torch.where(v < 0, -q, q).reshape(x.shape)


def _decode64(codes, scales):
    n = codes.shape[0]
    out = torch.empty((n, codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    for half, nib in enumerate((codes % 16, codes // 16)):
        nib = nib.double()
        mag = nib % 8
        expo, man = torch.floor(mag / 2), mag % 2
        val = torch.where(expo == 0, man * 0.5, torch.exp2(expo - 1) * (1 + man * 0.5))
        out[:, half::2] = torch.where(nib >= 8, -val, val)
    return out * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def _act64(y, silu):
    if silu:
        n = y.shape[-1] // 2
        y = y[..., :n] * torch.sigmoid(y[..., :n]) * y[..., n:]
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return _fake_quant64(s["x"])
    if op in ("gemv", "gemm"):
        x = s["x"].double() if op == "gemv" else _fake_quant64(s["x"])
        return _act64(x @ _decode64(s["w"], s["ws"]).T, s["silu"])
    ids, k, E = s["ids"].reshape(-1).tolist(), case["top_k"], case["E"]
    rows = [[] for _ in range(E)]
    for p, e in enumerate(ids):
        if e >= 0:
            rows[e].append(p)
    pairs = [p for r in rows for p in r]
    n, P = len(pairs), len(ids)
    dev = s["x"].device
    pair = torch.tensor(pairs, dtype=torch.int64, device=dev)
    if op == "grouped":
        x = _fake_quant64(s["x"])
        out = torch.zeros((P, case["N"] // 2 if s["silu"] else case["N"]), dtype=torch.float64, device=dev)
        at = 0
        for e in range(E):
            if rows[e]:
                xe = x[pair[at:at + len(rows[e])] // k] if s["gather"] else x[at:at + len(rows[e])]
                out[at:at + len(rows[e])] = _act64(xe @ _decode64(s["w"][e], s["ws"][e]).T, s["silu"])
            at += len(rows[e])
        return out
    if op == "dispatch":
        inverse, offsets, at = [-1] * P, [0], 0
        for r, p in enumerate(pairs):
            inverse[p] = r
        for r in rows:
            at += len(r)
            offsets.append(at)
        xs = torch.zeros((P, case["H"]), dtype=torch.float64, device=dev)
        xs[:n] = s["x"].double()[pair // k]
        got = {"xs": xs, "order": torch.tensor(pairs + [-1] * (P - n), dtype=torch.int32),
               "inverse": torch.tensor(inverse, dtype=torch.int32).view(case["M"], k),
               "offsets": torch.tensor(offsets, dtype=torch.int32)}
        if s["train"]:
            dx = torch.zeros((case["M"], case["H"]), dtype=torch.float64, device=dev)
            got["dx"] = dx.index_add_(0, pair // k, s["dy"][:n].double())
        return got
    w = s["topk_w"].double().reshape(-1)[pair]
    ys = s["x"][:n].double()
    y = torch.zeros((case["M"], case["H"]), dtype=torch.float64, device=dev)
    got = {"y": y.index_add_(0, pair // k, ys * w[:, None])}
    if s["train"]:
        dy = s["dy"].double()[pair // k]
        dys = torch.zeros((P, case["H"]), dtype=torch.float64, device=dev)
        dys[:n] = dy * w[:, None]
        dw = torch.zeros(P, dtype=torch.float64, device=dev)
        dw[pair] = (dy * ys).sum(1)
        got["dys"], got["dw"] = dys, dw.view(case["M"], k)
    return got
