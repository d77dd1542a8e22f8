"""Cases and plain forms of the serving operators around the expert layer.

Four operators, named by the case's "op":

  norm   residual addition, root-mean-square norm, and the normed row in E4M3
         with one f32 scale per 128 columns
             r = x + residual,  y = r / sqrt(mean(r^2) + eps) * weight
             s = max(amax |y| over the group / 448, 2^-126),  q = e4m3(y / s)
  silu   SiLU-mul of a stacked [T, 2 I] gate/up product, quantised the same way
  gemm   E4M3 matrix product with scales: one per row and 128 columns of the
         activations, one per 128 x 128 block of the weight
             out[m, n] = sum_kb sa[m, kb] sb[n / 128, kb] sum_{k in kb} a[m, k] w[n, k]  (+ addend[m, n])
  few    a whole mixture-of-experts layer for at most 32 tokens: routing from
         logits, gate/up with SiLU-mul, down, weighted sum over the experts

Codes in 8 bits come back as float8_e4m3fn tensors, the values they stand for.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GROUP = 128
FP8_MAX = 448.0
TINY_SCALE = 2.0 ** -126
ACT = {"bf16": torch.bfloat16, "f16": torch.float16}
MAX_FEW_TOKENS = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
WEIGHT_BITS = {"bf16": 16.0, "fp8": 8.0, "nvfp4": 4.5, "gptq": 4.0 + 20.0 / 128}


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # one token of a serving step on the 2048-wide layers: latency only
        {"name": "norm_token", "op": "norm", "act": "bf16", "T": 1, "H": 2048, "residual": True},
        # a ragged prompt batch on the 4096-wide layer
        {"name": "norm_prompt", "op": "norm", "act": "f16", "T": 4001, "H": 4096, "residual": True},
        # three sequences decoding through a shared expert of 1408 columns
        {"name": "silu_decode", "op": "silu", "act": "f16", "T": 3, "I": 1408},
        # a 4096-token prompt through a dense feed-forward of 14336 columns
        {"name": "silu_prompt", "op": "silu", "act": "bf16", "T": 4096, "I": 14336},
        # one token through the gate/up product of a shared expert: weights read once, latency
        {"name": "gemm_token", "op": "gemm", "act": "bf16", "M": 1, "N": 2816, "K": 2048, "addend": False},
        # an odd decode batch through a wide down product, added to the routed experts' output
        {"name": "gemm_decode", "op": "gemm", "act": "f16", "M": 17, "N": 4096, "K": 14336, "addend": True},
        # a short ragged prompt: rows and columns that end inside a tile
        {"name": "gemm_ragged", "op": "gemm", "act": "bf16", "M": 333, "N": 2816, "K": 2048, "addend": False},
        # a 4096-token prompt through the gate/up product of a dense feed-forward: tensor-bound
        {"name": "gemm_prompt", "op": "gemm", "act": "bf16", "M": 4096, "N": 28672, "K": 4096, "addend": False},
        # one sequence decoding on the fine-grained layer: 8 of 128 experts
        {"name": "few_one", "op": "few", "act": "bf16", "fmt": "bf16", "T": 1, "H": 2048, "I": 768, "E": 128, "k": 8,
         "renorm": True},
        # sixteen sequences on the 4-bit integer layer
        {"name": "few_gptq", "op": "few", "act": "f16", "fmt": "gptq", "T": 16, "H": 2048, "I": 1408, "E": 64, "k": 6,
         "renorm": True},
        # the most tokens of the range, on the 4-bit floating-point layer: every expert touched
        {"name": "few_nvfp4", "op": "few", "act": "bf16", "fmt": "nvfp4", "T": 32, "H": 2048, "I": 768, "E": 128,
         "k": 8, "renorm": True},
        # an odd batch on the layer of 8 wide experts: 2.8 GB of weights
        {"name": "few_wide", "op": "few", "act": "bf16", "fmt": "bf16", "T": 7, "H": 4096, "I": 14336, "E": 8, "k": 2,
         "renorm": True},
    ]


def _log_size(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    while True:
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step
        if lo <= v <= hi and v not in (3072, 1536):
            return v


def draw(rng):
    op = rng.choice(["norm", "silu", "gemm", "gemm", "few", "few"])
    act = rng.choice(["bf16", "f16"])
    if op == "norm":
        return {"op": op, "act": act, "T": _log_size(rng, 1, 4096), "H": _log_size(rng, 64, 8192, 8),
                "residual": rng.random() < 0.7}
    if op == "silu":
        return {"op": op, "act": act, "T": _log_size(rng, 1, 4096), "I": _log_size(rng, 64, 14336, 8)}
    if op == "gemm":
        while True:
            c = {"op": op, "act": act, "M": _log_size(rng, 1, 4096), "N": _log_size(rng, 64, 28672, 8),
                 "K": _log_size(rng, 128, 14336, 16), "addend": rng.random() < 0.4}
            if c["M"] * c["N"] * c["K"] <= 4096 * 28672 * 4096 and c["N"] * c["K"] <= 28672 * 4096:
                return c
    fmt = rng.choice(["bf16", "fp8", "nvfp4", "gptq"])
    step = {"bf16": 8, "fp8": 16, "nvfp4": 32, "gptq": 128}[fmt]
    while True:
        e = _log_size(rng, 2, 256)
        c = {"op": op, "act": "bf16" if fmt == "bf16" else act, "fmt": fmt, "T": _log_size(rng, 1, MAX_FEW_TOKENS),
             "H": _log_size(rng, 128, 4096, step), "I": _log_size(rng, 128, 14336, step), "E": e,
             "k": rng.randint(1, min(e, 8)), "renorm": rng.random() < 0.8}
        one = 3 * c["H"] * c["I"]
        if e * one <= 8 * 3 * 4096 * 14336 // 2 and c["T"] * c["k"] * one <= 14 * 3 * 4096 * 14336:
            return c


def work(case):
    op = case["op"]
    if op == "norm":
        t, h = case["T"], case["H"]
        acts = 3 + (1 if case["residual"] else 0)
        return {"bytes": t * h * (2 * acts + 1) + 4 * t * -(-h // GROUP) + 2 * h, "flops": 6 * t * h}
    if op == "silu":
        t, i = case["T"], case["I"]
        return {"bytes": t * i * 5 + 4 * t * -(-i // GROUP), "flops": 8 * t * i}
    if op == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        kb = -(-k // GROUP)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // GROUP)) + 2 * m * n * (2 if case["addend"] else 1),
                "flops": 2 * m * n * k}
    t, h, i, e, k = (case[x] for x in ("T", "H", "I", "E", "k"))
    touched = e * (1.0 - (1.0 - k / e) ** t)  # the expected number of distinct experts
    return {"bytes": touched * 3 * h * i * WEIGHT_BITS[case["fmt"]] / 8 + t * (4 * h + 4 * e + 8 * k),
            "flops": 6 * t * k * h * i}


# ---- inputs ------------------------------------------------------------------------

def _groups(v, width=GROUP):
    """[..., n] as [..., groups, width], the last group filled up with zeros."""
    pad = -v.shape[-1] % width
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    return v.unflatten(-1, (-1, width))


def _quantise(y):
    """E4M3 codes and f32 scales of f32 rows, one scale per 128 columns."""
    g = _groups(y)
    s = (g.abs().amax(-1) / FP8_MAX).clamp_min(TINY_SCALE)
    q = (g / s[..., None]).clamp(-FP8_MAX, FP8_MAX).flatten(-2)[..., : y.shape[-1]]
    return q.to(torch.float8_e4m3fn), s


def _weight(gen, fmt, e, n, k, groups2):
    """A stacked expert weight [e, n, k], of about N(0, 0.02), in the library's layouts."""
    if fmt == "bf16":
        w = torch.empty((e, n, k), dtype=torch.bfloat16, device=DEV)
        return {"w": w.normal_(0.0, 0.02, generator=gen)}
    if fmt == "fp8":
        v = torch.randn((e, n, k), generator=gen, device=DEV)
        s = v.abs().amax(-1) / FP8_MAX
        return {"w": (v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), "scales": s * 0.02}
    if fmt == "nvfp4":
        w = torch.randint(0, 256, (e, n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s = torch.rand((e, k // 16, n), generator=gen, device=DEV) * 1.5 + 0.25
        s2 = torch.rand((groups2, e), generator=gen, device=DEV) * 0.004 + 0.004
        return {"w": w, "scales": s.to(torch.float8_e4m3fn).view(torch.uint8), "scale2": s2}
    low, high = -2 ** 31, 2 ** 31
    w = torch.randint(low, high, (e, k // 8, n), generator=gen, device=DEV, dtype=torch.int32)
    s = (torch.rand((e, k // GROUP, n), generator=gen, device=DEV) * 0.004 + 0.002).half()
    z = torch.full((e, k // GROUP, n // 8), -2004318072, dtype=torch.int32, device=DEV)  # every zero point 8
    return {"w": w, "scales": s, "zeros": z}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, act = case["op"], ACT[case["act"]]
    s = dict(case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if op == "norm":
        t, h = case["T"], case["H"]
        loud = 1.0 + 9.0 * (torch.rand(h, generator=gen, device=DEV) < 0.01)  # a few loud channels
        s["x"] = randn(t, h).to(act)
        s["res"] = (randn(t, h) * 2.0 * loud).to(act) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * randn(h)).to(act)
        s["res_out"], s["y"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["q"] = torch.empty((t, h), dtype=torch.float8_e4m3fn, device=DEV)
        s["s"] = torch.empty((t, -(-h // GROUP)), device=DEV)
    elif op == "silu":
        t, i = case["T"], case["I"]
        s["gu"] = randn(t, 2 * i).to(act)
        s["q"] = torch.empty((t, i), dtype=torch.float8_e4m3fn, device=DEV)
        s["s"] = torch.empty((t, -(-i // GROUP)), device=DEV)
    elif op == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        q, s["sa"] = _quantise(randn(m, k))
        s["a"] = q.view(torch.uint8)
        w = torch.nn.functional.pad(randn(n, k) * 0.02, (0, -k % GROUP, 0, -n % GROUP))
        blocks = w.unflatten(1, (-1, GROUP)).unflatten(0, (-1, GROUP))  # [nb, 128, kb, 128]
        s["sb"] = (blocks.abs().amax((1, 3)) / FP8_MAX).contiguous()
        w = (blocks / s["sb"][:, None, :, None]).flatten(2, 3).flatten(0, 1)[:n, :k]
        s["w"] = w.to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
        s["addend"] = randn(m, n).to(act) if case["addend"] else None
        s["out"] = torch.empty((m, n), dtype=act, device=DEV)
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    else:
        t, h, i, e = case["T"], case["H"], case["I"], case["E"]
        s["x"] = randn(t, h).to(act)
        s["logits"] = randn(t, e)
        s["gu"] = _weight(gen, case["fmt"], e, 2 * i, h, 2)
        s["down"] = _weight(gen, case["fmt"], e, h, i, 1)
        if own:  # the buffers and weight descriptors of the layer, kept between calls; no work on the data
            s["plan"] = _few_plan(s)
    return s


# ---- one pass -----------------------------------------------------------------------

def _few_plan(s):
    from mixture_experts_grouped_gb300 import ffn, layer
    from mixture_experts_grouped_gb300 import moe as M

    code = M.WFMT_CODES[s["fmt"]]

    def weight(w):
        def at(name):
            return w[name].data_ptr() if name in w else None
        desc = M.MoeWeight(code, GROUP if s["fmt"] == "gptq" else 0, at("w"), at("scales"), at("zeros"), at("scale2"))
        return layer.DeviceWeight(desc, list(w.values()))

    return ffn.FewTokensLayer(s["T"], s["H"], s["I"], s["E"], s["k"], s["act"], weight(s["gu"]), weight(s["down"]),
                              DEV, renormalize=s["renorm"])


def _run_own(s):
    from mixture_experts_grouped_gb300 import moe as M

    op, act = s["op"], M.ACT_CODES[s["act"]]
    if op == "norm":
        M.moe_add_rmsnorm_quant(s["x"], s["res"], act, s["weight"], EPS, s["T"], s["H"], s["res_out"], s["y"], s["q"],
                                s["s"])
        return {"residual": s["res_out"], "y": s["y"], "q": s["q"], "scales": s["s"]}
    if op == "silu":
        M.moe_silu_mul_quant(s["gu"], act, s["T"], s["I"], s["q"], s["s"])
        return {"q": s["q"], "scales": s["s"]}
    if op == "gemm":
        M.moe_block_fp8_gemm(s["a"], s["sa"], s["w"], s["sb"], s["addend"], s["out"], act, s["M"], s["N"], s["K"],
                             s["err"])
        return s["out"]
    plan = s["plan"]
    return {"out": plan.forward(s["x"], s["logits"]), "ids": plan.topk_ids, "weights": plan.topk_weights}


def _expand_blocks(s, n, k):
    return s.repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]


def _dequant(w, fmt, ids):
    """The f32 weights [p, n, k] of the experts in ids."""
    if fmt == "bf16":
        return w["w"][ids].float()
    if fmt == "fp8":
        return w["w"].view(torch.float8_e4m3fn)[ids].float() * w["scales"][ids][..., None]
    if fmt == "nvfp4":
        lut = torch.tensor(E2M1, device=DEV)
        b = w["w"][ids]
        v = lut[torch.stack((b & 15, b >> 4), -1).flatten(-2).int()]
        sc = w["scales"].view(torch.float8_e4m3fn)[ids].float().transpose(1, 2)  # [p, n, k / 16]
        s2 = w["scale2"][:, ids].T.repeat_interleave(v.shape[1] // w["scale2"].shape[0], 1)  # [p, n]
        return (v.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2) * s2[..., None]
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    q = (w["w"][ids][:, :, None, :] >> shifts[:, None]) & 15          # [p, k / 8, 8, n]
    z = (w["zeros"][ids][..., None] >> shifts) & 15                    # [p, k / G, n / 8, 8]
    q = q.flatten(1, 2).unflatten(1, (-1, GROUP)) - z.flatten(-2)[:, :, None, :]
    return (q * w["scales"][ids].float()[:, :, None, :]).flatten(1, 2).transpose(1, 2)


def _run_plain(s):
    op, act = s["op"], ACT[s["act"]]
    if op == "norm":
        r = s["x"].float()
        if s["res"] is not None:
            r = r + s["res"].float()
        y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, sc = _quantise(y)
        return {"residual": r.to(act), "y": y.to(act), "q": q, "scales": sc}
    if op == "silu":
        g, u = s["gu"].float().chunk(2, -1)
        q, sc = _quantise(g / (1.0 + torch.exp(-g)) * u)
        return {"q": q, "scales": sc}
    if op == "gemm":
        m, n, k = s["M"], s["N"], s["K"]
        a = s["a"].view(torch.float8_e4m3fn).float() * s["sa"].repeat_interleave(GROUP, 1)[:, :k]
        w = s["w"].view(torch.float8_e4m3fn).float() * _expand_blocks(s["sb"], n, k)
        out = a @ w.T
        if s["addend"] is not None:
            out = out + s["addend"].float()
        return out.to(act)
    t, k, i = s["T"], s["k"], s["I"]
    top, ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True)  # equal logits: the lowest expert first
    top, ids = top[:, :k], ids[:, :k]
    e = torch.exp(top - top[:, :1])
    total = e if s["renorm"] else torch.exp(s["logits"] - top[:, :1])
    wt = e / total.sum(-1, keepdim=True)
    pairs = ids.reshape(-1)
    x = s["x"].float().repeat_interleave(k, 0)[..., None]              # [p, h, 1]
    gu = torch.bmm(_dequant(s["gu"], s["fmt"], pairs), x)[..., 0]
    g, u = gu[:, :i], gu[:, i:]
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(_dequant(s["down"], s["fmt"], pairs), h[..., None])[..., 0]
    out = (y.unflatten(0, (t, k)) * wt[..., None]).sum(1)
    return {"out": out.to(act), "ids": ids.int(), "weights": wt}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_quant(y):
    """Scales, and the quotients before their rounding to 8 bits: what the codes stand for."""
    t, h = y.shape
    scales = torch.empty((t, -(-h // GROUP)), dtype=torch.float64, device=DEV)
    quot = torch.empty_like(y)
    for j in range(scales.shape[1]):
        part = y[:, j * GROUP:(j + 1) * GROUP]
        top = torch.maximum(part.max(1).values, -part.min(1).values)
        scales[:, j] = torch.clamp(top / FP8_MAX, min=TINY_SCALE)
        quot[:, j * GROUP:(j + 1) * GROUP] = part / scales[:, j:j + 1]
    return quot, scales


def _exact_weight(w, fmt, e):
    """The f64 weight [n, k] of expert e."""
    if fmt == "bf16":
        return w["w"][e].double()
    if fmt == "fp8":
        return w["scales"][e].double().unsqueeze(1) * w["w"][e].view(torch.float8_e4m3fn).double()
    if fmt == "nvfp4":
        packed = w["w"][e].long()
        n, half = packed.shape
        mag = torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)
        out = torch.empty((n, 2 * half), dtype=torch.float64, device=DEV)
        for odd in (0, 1):
            code = (packed // 16) if odd else (packed % 16)
            out[:, odd::2] = mag[code % 8] * torch.where(code >= 8, -1.0, 1.0).double()
        sc = w["scales"][e].view(torch.float8_e4m3fn).double()
        for j in range(sc.shape[0]):
            out[:, 16 * j:16 * j + 16] *= sc[j].unsqueeze(1)
        part = n // w["scale2"].shape[0]
        for g in range(w["scale2"].shape[0]):
            out[g * part:(g + 1) * part] *= float(w["scale2"][g, e])
        return out
    words = w["w"][e].long() % (1 << 32)
    zeros = w["zeros"][e].long() % (1 << 32)
    kk, n = words.shape[0] * 8, words.shape[1]
    out = torch.empty((n, kk), dtype=torch.float64, device=DEV)
    zp = torch.empty((zeros.shape[0], n), dtype=torch.float64, device=DEV)
    for j in range(8):
        out[:, j::8] = ((words // 16 ** j) % 16).double().T
        zp[:, j::8] = ((zeros // 16 ** j) % 16).double()
    sc = w["scales"][e].double()
    for g in range(sc.shape[0]):
        at = slice(g * GROUP, (g + 1) * GROUP)
        out[:, at] = (out[:, at] - zp[g].unsqueeze(1)) * sc[g].unsqueeze(1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        r = s["x"].double()
        if s["res"] is not None:
            r += s["res"].double()
        rms = (torch.linalg.vector_norm(r, dim=1) ** 2 / case["H"] + EPS).sqrt()
        y = r / rms.unsqueeze(1) * s["weight"].double()
        q, sc = _exact_quant(y)
        return {"residual": r, "y": y, "q": q, "scales": sc}
    if op == "silu":
        gu = s["gu"].double()
        g, u = gu[:, :case["I"]], gu[:, case["I"]:]
        q, sc = _exact_quant(g * torch.sigmoid(g) * u)
        return {"q": q, "scales": sc}
    if op == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        out = torch.zeros((m, n), dtype=torch.float64, device=DEV)
        if s["addend"] is not None:
            out += s["addend"].double()
        a, w = (s[x].view(torch.float8_e4m3fn) for x in ("a", "w"))
        for j in range(-(-k // GROUP)):
            at = slice(j * GROUP, min(k, (j + 1) * GROUP))
            rows = s["sb"][:, j].double().repeat_interleave(GROUP)[:n]
            out += (a[:, at].double() * s["sa"][:, j:j + 1].double()) @ (w[:, at].double() * rows.unsqueeze(1)).T
        return out
    t, k = case["T"], case["k"]
    logits = s["logits"].double()
    order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    probs = torch.softmax(logits, dim=1).gather(1, order)
    if case["renorm"]:
        probs = probs / probs.sum(1, keepdim=True)
    out = torch.zeros((t, case["H"]), dtype=torch.float64, device=DEV)
    x = s["x"].double()
    for e in torch.unique(order).tolist():
        tok, slot = torch.nonzero(order == e, as_tuple=True)
        gu = x[tok] @ _exact_weight(s["gu"], case["fmt"], e).T
        g, u = gu[:, :case["I"]], gu[:, case["I"]:]
        y = (g * torch.sigmoid(g) * u) @ _exact_weight(s["down"], case["fmt"], e).T
        out.index_add_(0, tok, y * probs[tok, slot].unsqueeze(1))
    return {"out": out, "ids": None, "weights": probs}
