"""Plain 64-bit forms of the serving operators, and the error bounds that go with them.

Everything here is elementary torch arithmetic on f64 CPU tensors. The bounds
follow from the operators' stated roundings: `u(act)` is half a unit in the
last place of the output type, F32 = 2^-24 the same for f32, and a sum of n
products in f32, in any order, is off by at most about n F32 times the sum of
the products' magnitudes.
"""
import torch

F32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {a: torch.finfo(t).eps / 2 for a, t in DT.items()}                        # 2^-8, 2^-11
TINY = {a: torch.finfo(t).tiny * torch.finfo(t).eps / 2 for a, t in DT.items()}  # half the smallest subnormal
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def e4m3(codes):
    """uint8 codes to the f64 values they stand for."""
    return codes.cpu().view(torch.float8_e4m3fn).float().double()


def groups(v, width=128):
    pad = -v.shape[-1] % width
    return torch.nn.functional.pad(v, (0, pad)).unflatten(-1, (-1, width))


def quant_scales(v):
    return (groups(v).abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)


def check_quant(v, q, s, rel):
    """Codes q and scales s of f64 values v that the kernel knows to a relative error `rel` of its group's
    largest value: the scale is off by that and an f32 division, a code by half a step and the same."""
    q, s = q.cpu(), s.cpu().double()
    ref_s = quant_scales(v)
    assert torch.all((s - ref_s).abs() <= ref_s * (rel + 2 * F32)), ((s - ref_s).abs() / ref_s).max()
    quot = v / ref_s.repeat_interleave(128, -1)[..., : v.shape[-1]]
    step = torch.maximum(quot.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    err = (e4m3(q) - quot).abs()
    assert torch.all(err <= step * (1 + 2.0 ** -10) + 448.0 * 2 * (rel + 4 * F32)), (err / step).max()


def close(got, ref, act, slack):
    """|got - ref| <= the rounding to `act` of anything within `slack` of ref."""
    err = (got.cpu().double() - ref).abs()
    bound = slack + (ref.abs() + slack) * U[act] + TINY[act]
    assert torch.isfinite(got.float()).all()
    assert torch.all(err <= bound), f"worst error / bound {(err / bound).max():.3f}"


def silu_mul(g, u):
    return g * torch.sigmoid(g) * u


def dequant(w, fmt, e):
    """The f64 weight [N, K] of expert e from a dict of CPU tensors in the library's layouts."""
    if fmt == "bf16":
        return w["w"][e].double()
    if fmt == "fp8":
        return e4m3(w["w"][e]) * w["scales"][e].double()[:, None]
    if fmt == "nvfp4":
        b = w["w"][e].long()
        v = E2M1[torch.stack((b & 15, b >> 4), -1).flatten(1)]
        v = (v.unflatten(1, (-1, 16)) * e4m3(w["scales"][e]).T[..., None]).flatten(1)
        s2 = w["scale2"][:, e].double()
        return v * s2.repeat_interleave(v.shape[0] // len(s2))[:, None]
    words, zeros = w["w"][e].long() & 0xFFFFFFFF, w["zeros"][e].long() & 0xFFFFFFFF
    k8, n = words.shape
    q = torch.stack([(words >> 4 * j) & 15 for j in range(8)], 1).reshape(8 * k8, n)
    z = torch.stack([(zeros >> 4 * j) & 15 for j in range(8)], -1).reshape(zeros.shape[0], n)
    per = 8 * k8 // zeros.shape[0]
    z, s = z.repeat_interleave(per, 0), w["scales"][e].double().repeat_interleave(per, 0)
    return ((q - z).double() * s).T


def route(logits, k, renorm):
    l = logits.double()
    order = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
    p = torch.softmax(l, 1).gather(1, order)
    return order, (p / p.sum(1, keepdim=True) if renorm else p)


def few_tokens(x, ids, weights, gu, down, fmt, act, I, E):
    """The layer in f64, and how far the kernels may be off before the last rounding."""
    x, T, H = x.double(), x.shape[0], x.shape[1]
    out, slack = torch.zeros((T, H), dtype=torch.float64), torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(tok) == 0:
            continue
        wg, wd, xe, w = dequant(gu, fmt, e), dequant(down, fmt, e), x[tok], weights[tok, slot].double()[:, None]
        y1, mag = xe @ wg.T, xe.abs() @ wg.abs().T
        g, u = y1[:, :I], y1[:, I:]
        dg, du = mag[:, :I] * H * F32, mag[:, I:] * H * F32
        h = silu_mul(g, u)
        # silu' is within 1.1; exp and the division are good to a few ulp beside |g|'s rounding
        dh = 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du
        dh = dh + h.abs() * (16 + g.abs()) * F32 * 2
        dh = dh + (h.abs() + dh) * U[act] + TINY[act]
        out.index_add_(0, tok, w * (h @ wd.T))
        slack.index_add_(0, tok, w * (dh @ wd.abs().T + (h.abs() @ wd.abs().T) * (I + 64) * F32))
    return out, slack
