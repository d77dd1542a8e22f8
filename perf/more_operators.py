"""Cases and plain forms of the operators that train the expert layer, and of the 16-bit dense product.

Six operators, named by the case's "op":

  ragged   matrix product grouped by expert; group e is rows offsets[e] .. offsets[e + 1], of any size
               "out":    out[r, n] = sum_k a[r, k] w_e[n, k]
               "input":  out[r, k] = sum_n a[r, n] w_e[n, k]     (the gradient of its input)
  wgrad    the gradient of its weight:  dw_e[n, k] = (base_e[n, k]) + sum_{r in e} dy[r, n] x[r, k]
  dense    z = a w^T + bias,  out = f(z) + residual, and z itself where the gradient needs it
  dgrad    its gradient:  dz = d_out f'(z);  d_a = dz w,  d_w = dz^T a,  d_bias = sum_m dz
  glu      SwiGLU of stacked [rows, 2 I] gate/up products
               "out":   h = g s(g) u,  s(g) = 1 / (1 + exp(-g))
               "grad":  d_g = d_h u s(g) (1 + g (1 - s(g))),  d_u = d_h g s(g),  and h again
  routing  rows to the experts and the gradients of what brings them back: xs[row of (t, j)] = x[t],
           d_y[row] = w_tj d_out[t],  d_w_tj = d_out[t] . y[row],  and from d_w the gradient of the logits
"""

import math

import torch

own = False

DEV = "cuda"
ACT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # eight sequences decoding through the gate/up product of 128 narrow experts: most of them have a row or two
        {"name": "ragged_few", "op": "ragged", "dir": "out", "act": "bf16", "rows": 64, "E": 128, "N": 1536, "K": 2048,
         "skew": 0.0},
        # a short training batch, back through the down product of 64 experts of uneven load
        {"name": "ragged_input", "op": "ragged", "dir": "input", "act": "f16", "rows": 3066, "E": 64, "N": 2048,
         "K": 1408, "skew": 0.5},
        # 4096 tokens through the gate/up product of 8 wide experts: tensor-bound
        {"name": "ragged_prompt", "op": "ragged", "dir": "out", "act": "bf16", "rows": 8192, "E": 8, "N": 28672,
         "K": 4096, "skew": 0.0},
        # a micro-batch added to the f32 gradients of 64 experts: bound by the gradients' bytes
        {"name": "wgrad_add", "op": "wgrad", "act": "f16", "rows": 12288, "E": 64, "N": 2048, "K": 1408, "skew": 0.5,
         "f32": True, "base": True},
        # 4096 tokens, the gradient of 8 wide down products
        {"name": "wgrad_wide", "op": "wgrad", "act": "bf16", "rows": 8192, "E": 8, "N": 4096, "K": 14336, "skew": 0.0,
         "f32": False, "base": False},
        # three sequences through a shared expert's down product, added to the routed experts' output: latency
        {"name": "dense_few", "op": "dense", "act": "f16", "M": 3, "N": 2048, "K": 1408, "f": "none", "bias": True,
         "residual": True, "pre": False},
        # a training batch through the first product of a dense block: tensor-bound, z kept for the gradient
        {"name": "dense_prompt", "op": "dense", "act": "bf16", "M": 4096, "N": 14336, "K": 4096, "f": "gelu_tanh",
         "bias": True, "residual": False, "pre": True},
        # and the gradient of a shared expert's first product
        {"name": "dense_grad", "op": "dgrad", "act": "bf16", "M": 1333, "N": 2816, "K": 2048, "f": "gelu",
         "bias": True},
        # a few tokens' rows of the narrow experts
        {"name": "glu_few", "op": "glu", "dir": "out", "act": "f16", "rows": 64, "I": 768},
        # 4096 tokens back through the wide experts' activation, which is computed again
        {"name": "glu_grad", "op": "glu", "dir": "grad", "act": "bf16", "rows": 8192, "I": 14336},
        # a small batch of the fine-grained layer, all experts in the softmax
        {"name": "routing_few", "op": "routing", "act": "f16", "T": 61, "H": 2048, "E": 128, "k": 8, "renorm": False},
        # 4096 tokens of the layer of 8 wide experts
        {"name": "routing_prompt", "op": "routing", "act": "bf16", "T": 4096, "H": 4096, "E": 8, "k": 2,
         "renorm": True},
    ]


def _log_size(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    while True:
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step
        if lo <= v <= hi:
            return v


def _largest_share(e, skew):
    """What the fullest group has, in shares of the mean."""
    return e / sum((i + 1) ** -skew for i in range(e))


MOST = 8192 * 28672 * 4096


def draw(rng):
    op = rng.choice(["ragged", "ragged", "wgrad", "wgrad", "dense", "dense", "dgrad", "glu", "routing"])
    act = rng.choice(["bf16", "f16"])
    if op in ("ragged", "wgrad"):
        while True:
            c = {"op": op, "act": act, "rows": _log_size(rng, 1, 32768), "E": _log_size(rng, 1, 256),
                 "N": _log_size(rng, 64, 28672, 8), "K": _log_size(rng, 64, 14336, 8),
                 "skew": rng.choice([0.0, 0.5])}
            each = c["N"] * c["K"]
            padded = c["rows"] * _largest_share(c["E"], c["skew"]) + 4 * c["E"] * math.sqrt(c["rows"] / c["E"] + 1)
            if c["E"] * each <= 8 * 28672 * 4096 // 2 and padded * each <= MOST // 2:
                break
        if op == "ragged":
            return {**c, "dir": rng.choice(["out", "input"])}
        f32 = rng.random() < 0.6
        return {**c, "f32": f32, "base": f32 and rng.random() < 0.6}
    if op in ("dense", "dgrad"):
        while True:
            c = {"op": op, "act": act, "M": _log_size(rng, 1, 4096), "N": _log_size(rng, 64, 28672, 8),
                 "K": _log_size(rng, 64, 14336, 8), "f": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 "bias": rng.random() < 0.6}
            if c["M"] * c["N"] * c["K"] <= MOST // 4 and c["N"] * c["K"] <= 28672 * 4096:
                break
        if op == "dgrad":
            return c
        return {**c, "residual": rng.random() < 0.5, "pre": rng.random() < 0.4}
    if op == "glu":
        return {"op": op, "act": act, "rows": _log_size(rng, 1, 8192), "I": _log_size(rng, 64, 14336, 8),
                "dir": rng.choice(["out", "grad"])}
    e = _log_size(rng, 2, 256)
    return {"op": op, "act": act, "T": _log_size(rng, 1, 4096), "H": _log_size(rng, 64, 8192, 8), "E": e,
            "k": rng.randint(1, min(e, 8)), "renorm": rng.random() < 0.6}


def work(case):
    op = case["op"]
    if op in ("ragged", "wgrad"):
        r, e, n, k = case["rows"], case["E"], case["N"], case["K"]
        if op == "ragged":
            touched = e * (1.0 - (1.0 - 1.0 / e) ** r)  # the expected number of groups with rows
            return {"bytes": 2 * (r * (n + k) + touched * n * k) + 4 * (e + 1), "flops": 2 * r * n * k}
        out = (4 if case["f32"] else 2) + (4 if case["base"] else 0)
        return {"bytes": 2 * r * (n + k) + out * e * n * k + 4 * (e + 1), "flops": 2 * r * n * k}
    if op in ("dense", "dgrad"):
        m, n, k = case["M"], case["N"], case["K"]
        if op == "dense":
            rows = 1 + (1 if case["residual"] else 0) + (1 if case["pre"] else 0)
            return {"bytes": 2 * (m * k + n * k + m * n * rows + (n if case["bias"] else 0)), "flops": 2 * m * n * k}
        ins = 1 + (1 if case["f"] != "none" else 0)
        return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * ins) + (4 * n if case["bias"] else 0),
                "flops": 4 * m * n * k}
    if op == "glu":
        each = 6 if case["dir"] == "out" else 12
        return {"bytes": each * case["rows"] * case["I"], "flops": 10 * case["rows"] * case["I"]}
    t, h, e, k = case["T"], case["H"], case["E"], case["k"]
    return {"bytes": 2 * t * h * (2 + 3 * k) + 4 * t * (2 * e + 5 * k), "flops": 4 * t * k * h}


# ---- inputs ------------------------------------------------------------------------

def _groups(case, seed):
    """Offsets of the groups (device) and the fullest group's size: rows dealt at random, low experts more often."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    share = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -case["skew"]
    to = torch.multinomial(share, case["rows"], replacement=True, generator=gen)
    counts = torch.bincount(to, minlength=case["E"])
    offsets = torch.zeros(case["E"] + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    return offsets.to(DEV), int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, act = case["op"], ACT[case["act"]]
    s = dict(case)

    def randn(*shape, std=1.0, dtype=act):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)

    def empty(*shape, dtype=act):
        return torch.empty(shape, dtype=dtype, device=DEV)

    s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op in ("ragged", "wgrad"):
        r, e, n, k = case["rows"], case["E"], case["N"], case["K"]
        s["offsets"], s["cap"] = _groups(case, seed)
        if op == "ragged":
            back = case["dir"] == "input"
            s["a"], s["w"] = randn(r, n if back else k, std=0.1 if back else 1.0), randn(e, n, k, std=0.02)
            s["out"] = empty(r, k if back else n)
        else:
            dt = torch.float32 if case["f32"] else act
            s["dy"], s["x"] = randn(r, n, std=0.1), randn(r, k)
            s["base"] = randn(e, n, k, dtype=dt) if case["base"] else None
            s["dw"] = empty(e, n, k, dtype=dt)
    elif op == "dense":
        m, n, k = case["M"], case["N"], case["K"]
        s["a"], s["w"] = randn(m, k), randn(n, k, std=0.02)
        s["bias"] = randn(n, std=0.2) if case["bias"] else None
        s["residual"] = randn(m, n) if case["residual"] else None
        s["pre"] = empty(m, n) if case["pre"] else None
        s["out"] = empty(m, n)
    elif op == "dgrad":
        m, n, k = case["M"], case["N"], case["K"]
        s["d_out"], s["a"], s["w"] = randn(m, n, std=0.1), randn(m, k), randn(n, k, std=0.02)
        s["pre"] = randn(m, n, std=1.5) if case["f"] != "none" else None
        s["dz"] = empty(m, n) if case["f"] != "none" else None
        s["d_a"], s["d_w"] = empty(m, k), empty(n, k)
        s["d_bias"] = empty(n, dtype=torch.float32) if case["bias"] else None
    elif op == "glu":
        r, i = case["rows"], case["I"]
        s["gu"], s["h"] = randn(r, 2 * i), empty(r, i)
        if case["dir"] == "grad":
            s["dh"], s["dgu"] = randn(r, i, std=0.1), empty(r, 2 * i)
    else:
        t, h, e, k = case["T"], case["H"], case["E"], case["k"]
        s["x"], s["y"], s["d_out"] = randn(t, h), randn(t * k, h), randn(t, h, std=0.1)
        s["logits"] = randn(t, e, dtype=torch.float32)
        top, ids = torch.topk(s["logits"], k, dim=1)
        s["ids"] = ids.int()
        s["weights"] = (torch.softmax(top, 1) if case["renorm"]
                        else torch.softmax(s["logits"], 1).gather(1, ids)).contiguous()
        order = torch.sort(ids.flatten(), stable=True).indices  # pairs in the experts' order
        s["row"] = torch.empty(t * k, dtype=torch.int32, device=DEV)
        s["row"][order] = torch.arange(t * k, device=DEV, dtype=torch.int32)
        s["xs"], s["dy"] = empty(t * k, h), empty(t * k, h)
        s["dw"], s["dl"] = empty(t, k, dtype=torch.float32), empty(t, e, dtype=torch.float32)
    return s


# ---- one pass -----------------------------------------------------------------------

def _run_own(s):
    from mixture_experts_grouped_gb300 import moe as M

    op, act = s["op"], M.ACT_CODES[s["act"]]
    if op == "ragged":
        M.moe_ragged_gemm(s["a"], act, s["w"], s["dir"] == "input", s["offsets"], s["rows"], s["N"], s["K"], s["E"],
                          s["out"], s["err"])
        return s["out"]
    if op == "wgrad":
        M.moe_ragged_wgrad(s["dy"], s["x"], act, s["offsets"], s["rows"], s["N"], s["K"], s["E"], s["base"], s["dw"],
                           s["f32"], s["err"])
        return s["dw"]
    if op == "dense":
        M.moe_dense_gemm(s["a"], act, s["w"], s["bias"], M.FN_CODES[s["f"]], s["residual"], s["pre"], s["out"], s["M"],
                         s["N"], s["K"], s["err"])
        return {"out": s["out"], "pre": s["pre"]} if s["pre"] is not None else s["out"]
    if op == "dgrad":
        m, n, k, dz = s["M"], s["N"], s["K"], s["d_out"]
        if s["f"] != "none" or s["bias"]:
            M.moe_bias_act_backward(dz, s["pre"], act, M.FN_CODES[s["f"]], m, n, s["dz"], s["d_bias"])
        if s["f"] != "none":
            dz = s["dz"]
        M.moe_ragged_gemm(dz, act, s["w"], True, None, m, n, k, 1, s["d_a"], s["err"])
        M.moe_ragged_wgrad(dz, s["a"], act, None, m, n, k, 1, None, s["d_w"], False, s["err"])
        out = {"a": s["d_a"], "w": s["d_w"]}
        return {**out, "bias": s["d_bias"]} if s["bias"] else out
    if op == "glu":
        if s["dir"] == "out":
            M.moe_swiglu(s["gu"], act, s["rows"], s["I"], s["h"])
            return s["h"]
        M.moe_swiglu_backward(s["gu"], s["dh"], act, s["rows"], s["I"], s["dgu"], s["h"])
        return {"gate_up": s["dgu"], "h": s["h"]}
    t, h, k = s["T"], s["H"], s["k"]
    M.moe_dispatch(s["x"], act, s["row"], s["xs"], t, h, k, t * k, s["err"])
    M.moe_combine_backward(s["d_out"], s["y"], act, s["row"], s["weights"], s["dy"], s["dw"], t, h, k, t * k, s["err"])
    M.moe_route_backward(s["logits"], s["ids"], s["weights"], s["dw"], s["dl"], t, s["E"], k, s["renorm"], s["err"])
    return {"xs": s["xs"], "dy": s["dy"], "dw": s["dw"], "dl": s["dl"]}


def _by_group(rows, offsets, cap):
    """f32 rows in the groups' order as [E, cap, columns], filled up with zeros; and where each row went."""
    at = torch.arange(rows.shape[0], device=DEV)
    e = torch.searchsorted(offsets[1:].long(), at, right=True)
    slot = e * cap + at - offsets.long()[e]
    out = torch.zeros((offsets.shape[0] - 1) * cap, rows.shape[1], device=DEV)
    out[slot] = rows.float()
    return out.unflatten(0, (-1, cap)), slot


def _f(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z * (z > 0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


def _df(name, z):
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    c = (2.0 / math.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _run_plain(s):
    op, act = s["op"], ACT[s["act"]]
    if op == "ragged":
        a, slot = _by_group(s["a"], s["offsets"], s["cap"])
        w = s["w"].float()
        return torch.bmm(a, w if s["dir"] == "input" else w.mT).flatten(0, 1)[slot].to(act)
    if op == "wgrad":
        dy, _ = _by_group(s["dy"], s["offsets"], s["cap"])
        x, _ = _by_group(s["x"], s["offsets"], s["cap"])
        dw = torch.bmm(dy.mT, x)
        return (dw + s["base"] if s["base"] is not None else dw).to(s["dw"].dtype)
    if op == "dense":
        z = s["a"].float() @ s["w"].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _f(s["f"], z)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return {"out": out.to(act), "pre": z.to(act)} if s["pre"] is not None else out.to(act)
    if op == "dgrad":
        dz = s["d_out"].float()
        if s["pre"] is not None:
            dz = dz * _df(s["f"], s["pre"].float())
        out = {"a": (dz @ s["w"].float()).to(act), "w": (dz.T @ s["a"].float()).to(act)}
        return {**out, "bias": dz.sum(0)} if s["bias"] else out
    if op == "glu":
        g, u = s["gu"].float().chunk(2, -1)
        sg = 1.0 / (1.0 + torch.exp(-g))
        h = (g * sg * u).to(act)
        if s["dir"] == "out":
            return h
        dh = s["dh"].float()
        return {"gate_up": torch.cat((dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg), -1).to(act), "h": h}
    t, k = s["T"], s["k"]
    w, ids, row = s["weights"], s["ids"].long(), s["row"].long()
    xs = torch.empty_like(s["xs"])
    xs[row] = s["x"].repeat_interleave(k, 0)
    d_out = s["d_out"].float()
    dw = (d_out[:, None] * s["y"][row].float().unflatten(0, (t, k))).sum(-1)
    dy = torch.empty_like(s["y"])
    dy[row] = (w[..., None] * d_out[:, None]).flatten(0, 1).to(act)
    mean = (dw * w).sum(1, keepdim=True)
    if s["renorm"]:
        dl = torch.zeros_like(s["logits"]).scatter(1, ids, w * (dw - mean))
    else:
        p = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dl = p * (torch.zeros_like(p).scatter(1, ids, dw) - mean)
    return {"xs": xs, "dy": dy, "dw": dw, "dl": dl}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_f(name, z):
    """f(z) and f'(z)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), torch.where(z > 0, 1.0, 0.0).double()
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    # 1/2 (1 + tanh v) = expit(2 v)
    v2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.special.expit(v2)
    return z * p, p + z * p * torch.special.expit(-v2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ragged", "wgrad"):
        at = s["offsets"].tolist()
        if op == "ragged":
            out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
            for e in range(case["E"]):
                lo, hi = at[e], at[e + 1]
                if hi > lo:
                    w = s["w"][e].double()
                    out[lo:hi] = s["a"][lo:hi].double() @ (w if case["dir"] == "input" else w.T)
            return out
        dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            lo, hi = at[e], at[e + 1]
            if s["base"] is not None:
                dw[e] += s["base"][e]
            if hi > lo:
                dw[e] += s["dy"][lo:hi].double().T @ s["x"][lo:hi].double()
        return dw
    if op == "dense":
        z = torch.nn.functional.linear(s["a"].double(), s["w"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        out = _exact_f(case["f"], z)[0]
        if s["residual"] is not None:
            out = out + s["residual"]
        return {"out": out, "pre": z} if case["pre"] else out
    if op == "dgrad":
        dz = s["d_out"].double()
        if s["pre"] is not None:
            dz = dz * _exact_f(case["f"], s["pre"].double())[1]
        out = {"a": torch.einsum("mn,nk->mk", dz, s["w"].double()),
               "w": torch.einsum("mn,mk->nk", dz, s["a"].double())}
        if case["bias"]:
            out["bias"] = torch.einsum("mn->n", dz)
        return out
    if op == "glu":
        i = case["I"]
        g, u = s["gu"][:, :i].double(), s["gu"][:, i:].double()
        f, df = _exact_f("silu", g)
        if case["dir"] == "out":
            return f * u
        dh = s["dh"].double()
        return {"gate_up": torch.cat((dh * u * df, dh * f), 1), "h": f * u}
    t, k = case["T"], case["k"]
    w, ids = s["weights"].double(), s["ids"].long()
    dw = torch.zeros((t, k), dtype=torch.float64, device=DEV)
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    row = s["row"].long().view(t, k)
    for j in range(k):
        dw[:, j] = torch.einsum("th,th->t", s["d_out"].double(), s["y"][row[:, j]].double())
        dy.index_copy_(0, row[:, j], w[:, j, None] * s["d_out"].double())
    xs = torch.empty(s["xs"].shape, dtype=torch.float64, device=DEV)
    for j in range(k):
        xs.index_copy_(0, row[:, j], s["x"].double())
    logits = s["logits"].double()
    if case["renorm"]:
        chosen = torch.zeros_like(logits).scatter_(1, ids, 1.0)
        logits = torch.where(chosen > 0, logits, -math.inf)
    p = torch.softmax(logits, 1)
    g = torch.zeros_like(logits).scatter_(1, ids, dw)
    return {"xs": xs, "dy": dy, "dw": dw, "dl": p * (g - (p * g).sum(1, keepdim=True))}
