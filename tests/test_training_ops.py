"""Ragged products, the 16-bit dense product and the row operators of a training step against plain
64-bit forms, their gradients against differences, and their refusals."""
import math
import os
import pathlib
import subprocess
import sys

import pytest
import torch

import plain

F32 = plain.F32
FNS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_gb300 import build as b
    b.build()
    from mixture_experts_grouped_gb300 import moe as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, act="bf16", std=1.0):
    return (torch.randn(shape, generator=g) * std).to(plain.DT[act])


def offsets_of(counts, first=0):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    return off + first


def f64(name, z):
    """f(z) and f'(z)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi) if name == "gelu_tanh" else 1.0
    v = k * (z + 0.044715 * z ** 3) if name == "gelu_tanh" else z
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    dv = k * (1 + 0.134145 * z * z) if name == "gelu_tanh" else 1.0
    return z * p, p + z * p * q * dv


def sum_slack(mag, n):
    """How far an f32 sum of n products may be off: mag is the sum of their magnitudes. A tensor core adds 16
    products at a time and may cut instead of rounding (twice the half step), which n + 64 half steps cover."""
    return mag * (n + 64) * F32


# ---- products grouped by expert ------------------------------------------------------------

# counts of rows per group: none, one, tile edges, long, one group alone
COUNTS = [
    [1], [0, 1, 0], [5], [16, 17, 15, 0, 1, 33], [0, 0, 255, 256, 257, 3, 0], [700], [64] * 5, [31, 300, 0, 2],
    [3] * 40, [0] * 30 + [9] + [0] * 9, [1000, 24], [0, 0, 0], [130, 140, 127, 129, 128],
]
NK = [(8, 8), (72, 136), (256, 64), (264, 200), (520, 1032), (1000, 72), (128, 2056)]


def ragged_case(moe, dev, counts, N, K, act, transposed, seed, lead=0, tail=0):
    g = gen(seed)
    rows, E = lead + sum(counts) + tail, len(counts)
    a = randn(g, rows, N if transposed else K, act=act)
    w = randn(g, E, N, K, act=act, std=0.1)
    off = offsets_of(counts, lead)
    J = K if transposed else N
    out = torch.full((rows, J), 7.0, dtype=plain.DT[act], device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_ragged_gemm(a.to(dev), moe.ACT_CODES[act], w.to(dev), transposed, off.to(dev), rows, N, K, E, out, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    ref, mag = torch.full((rows, J), 7.0, dtype=torch.float64), torch.zeros((rows, J), dtype=torch.float64)
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        we = w[e].double() if transposed else w[e].double().T
        ref[at], mag[at] = a[at].double() @ we, a[at].double().abs() @ we.abs()
    plain.close(out, ref, act, sum_slack(mag, N if transposed else K))
    out = out.cpu()
    assert torch.all(out[:lead] == 7) and torch.all(out[lead + sum(counts):] == 7)


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("i", range(len(COUNTS)))
def test_ragged_product_matches_the_formula(moe, dev, i, transposed):
    for j in range(3):
        N, K = NK[(2 * i + j) % len(NK)]
        ragged_case(moe, dev, COUNTS[i], N, K, ["bf16", "f16"][(i + j) % 2], transposed, 100 * i + j)


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
def test_ragged_rows_outside_the_groups_are_left_alone(moe, dev, transposed):
    ragged_case(moe, dev, [3, 0, 40], 264, 136, "bf16", transposed, 1, lead=5, tail=9)
    ragged_case(moe, dev, [300, 1], 72, 520, "f16", transposed, 2, lead=1, tail=300)


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,E,N,K", [(64, 128, 1536, 2048), (3000, 64, 2048, 1408), (2500, 3, 4096, 1032)])
def test_ragged_product_of_layers(moe, dev, rows, E, N, K, transposed):
    counts = torch.bincount(torch.multinomial(torch.arange(1, E + 1.0) ** -0.5, rows, True, generator=gen(E)),
                            minlength=E).tolist()
    g = torch.Generator(device=dev).manual_seed(rows)
    a = torch.randn((rows, N if transposed else K), generator=g, device=dev).bfloat16()
    w = (torch.randn((E, N, K), generator=g, device=dev) * 0.05).bfloat16()
    off = offsets_of(counts)
    out = torch.empty((rows, K if transposed else N), dtype=torch.bfloat16, device=dev)
    again = torch.empty_like(out)
    for o in (out, again):
        moe.moe_ragged_gemm(a, 0, w, transposed, off.to(dev), rows, N, K, E, o)
    assert torch.equal(out, again)
    ref, mag = torch.empty(out.shape, dtype=torch.float64, device=dev), torch.empty(out.shape, dtype=torch.float64,
                                                                                      device=dev)
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        we = w[e].double() if transposed else w[e].double().T
        ref[at], mag[at] = a[at].double() @ we, a[at].double().abs() @ we.abs()
    plain.close(out, ref.cpu(), "bf16", sum_slack(mag, N if transposed else K).cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
def test_ragged_product_keeps_non_finite_values_apart(moe, dev, transposed):
    """A row's NaN stays in its row, an expert's in its rows, and rows outside the groups are not read."""
    counts, N, K = [20, 0, 37, 5, 16], 136, 72
    rows = sum(counts) + 6
    off = offsets_of(counts, 2)
    g = gen(3)
    a, w = randn(g, rows, N if transposed else K), randn(g, 5, N, K)
    clean = a.clone()
    a[:2], a[rows - 4:] = float("nan"), float("inf")
    a[30, 4] = float("nan")
    w[1] = float("inf")  # no row's
    w[3, 5] = float("nan")
    outs = []
    for x in (a, clean):
        out = torch.zeros((rows, K if transposed else N), dtype=torch.bfloat16, device=dev)
        moe.moe_ragged_gemm(x.to(dev), 0, w.to(dev), transposed, off.to(dev), rows, N, K, 5, out)
        outs.append(out.cpu())
    bad = torch.isnan(outs[0])
    assert bad[30].all()
    expert = slice(2 + 57, 2 + 62)
    if transposed:
        assert bad[expert].all()
    else:
        assert bad[expert, 5].all() and not bad[expert][:, torch.arange(N) != 5].any()
    ok = torch.ones(rows, dtype=torch.bool)
    ok[30], ok[expert] = False, False
    assert torch.equal(outs[0][ok], outs[1][ok]) and torch.isfinite(outs[0][ok].float()).all()


def wgrad_case(moe, dev, counts, N, K, act, f32, addend, seed, lead=0, tail=0):
    g = gen(seed)
    rows, E = lead + sum(counts) + tail, len(counts)
    dy, x = randn(g, rows, N, act=act), randn(g, rows, K, act=act)
    dy[:lead], x[lead + sum(counts):] = float("nan"), float("inf")  # outside the groups: not read
    off = offsets_of(counts, lead)
    add = torch.randn((E, N, K), generator=g) if addend else None
    dw = torch.full((E, N, K), 5.0, dtype=torch.float32 if f32 else plain.DT[act], device=dev)
    if addend == "in place":
        dw = add.to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_ragged_wgrad(dy.to(dev), x.to(dev), moe.ACT_CODES[act], off.to(dev), rows, N, K, E,
                         dw if addend == "in place" else add.to(dev) if addend else None, dw, f32, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        d, xe = dy[at].double(), x[at].double()
        ref, mag = d.T @ xe, d.abs().T @ xe.abs()
        n = counts[e]
        if addend:
            ref, mag, n = ref + add[e].double(), mag + add[e].double().abs(), n + 1
        if f32:
            got = dw[e].cpu().double()
            assert torch.all((got - ref).abs() <= sum_slack(mag, n)), (e, counts[e])
            if counts[e] == 0:
                assert torch.equal(got, ref)
        else:
            plain.close(dw[e], ref, act, sum_slack(mag, n))


@pytest.mark.gpu
@pytest.mark.parametrize("f32,addend", [(True, None), (True, "apart"), (True, "in place"), (False, None)])
@pytest.mark.parametrize("i", range(len(COUNTS)))
def test_weight_gradient_matches_the_formula(moe, dev, i, f32, addend):
    for j in range(2):
        N, K = NK[(2 * i + 3 * j + 1) % len(NK)]
        if len(COUNTS[i]) * N * K <= 1 << 21:
            wgrad_case(moe, dev, COUNTS[i], N, K, ["bf16", "f16"][(i + j) % 2], f32, addend, 100 * i + j)


@pytest.mark.gpu
def test_weight_gradient_reads_its_groups_alone(moe, dev):
    """Neighbouring groups, and rows outside all, hold NaN and infinities."""
    wgrad_case(moe, dev, [3, 0, 40], 264, 136, "bf16", True, None, 1, lead=5, tail=9)
    wgrad_case(moe, dev, [65, 1], 72, 520, "f16", False, None, 2, lead=70, tail=3)
    for bad in range(3):
        counts, N, K = [17, 30, 50], 136, 264
        g = gen(bad)
        dy, x = randn(g, 97, N), randn(g, 97, K)
        off = offsets_of(counts)
        hot = slice(int(off[bad]), int(off[bad + 1]))
        outs = []
        for v in (1.0, float("nan"), float("inf")):
            dy[hot], x[hot] = v, v
            dw = torch.empty((3, N, K), device=dev)
            moe.moe_ragged_wgrad(dy.to(dev), x.to(dev), 0, off.to(dev), 97, N, K, 3, None, dw, True)
            outs.append(dw.cpu())
        for e in range(3):
            if e != bad:
                assert torch.equal(outs[0][e], outs[1][e]) and torch.equal(outs[0][e], outs[2][e])
        assert torch.isnan(outs[1][bad]).all() and torch.isinf(outs[2][bad]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,E,N,K,f32", [(4096, 1, 2816, 2048, True), (12288, 64, 2048, 1408, True),
                                            (4100, 8, 1408, 4096, False), (30000, 1, 264, 520, True)])
def test_weight_gradient_of_layers(moe, dev, rows, E, N, K, f32):
    counts = torch.bincount(torch.multinomial(torch.arange(1, E + 1.0) ** -0.5, rows, True, generator=gen(E)),
                            minlength=E).tolist()
    g = torch.Generator(device=dev).manual_seed(rows)
    dy = (torch.randn((rows, N), generator=g, device=dev) * 0.1 + 0.05).bfloat16()
    x = (torch.randn((rows, K), generator=g, device=dev) + 0.5).bfloat16()
    off = offsets_of(counts)
    dw = torch.empty((E, N, K), dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    again = torch.empty_like(dw)
    for o in (dw, again):
        moe.moe_ragged_wgrad(dy, x, 0, off.to(dev), rows, N, K, E, None, o, f32)
    assert torch.equal(dw, again)
    num, den = 0.0, 0.0
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        d, xe = dy[at].double(), x[at].double()
        ref, mag = d.T @ xe, d.abs().T @ xe.abs()
        if f32:
            assert torch.all((dw[e].double() - ref).abs() <= sum_slack(mag, counts[e]))
            num, den = num + float(((dw[e].double() - ref) ** 2).sum()), den + float((ref ** 2).sum())
        else:
            plain.close(dw[e], ref.cpu(), "bf16", sum_slack(mag, counts[e]).cpu())
    if f32:
        # the sums here grow steadily (means are not 0), so each of the rows / 16 steps may lose half a step (2^-24) on
        # average of a sum half as large; the chunks of 4096 rows are added one by one
        assert math.sqrt(num / den) <= (4096 / 16 / 2 + 16) * F32


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N,K", [(1, 8, 8), (70, 72, 136), (300, 264, 520), (600, 520, 264), (1000, 1032, 1000),
                                      (2414, 920, 256), (4097, 512, 520), (9000, 264, 136), (30000, 264, 520),
                                      (1333, 2816, 2048)])
def test_weight_gradient_of_one_group_in_every_form(moe, dev, rows, N, K):
    """Without offsets: pairs, or one to eight CTAs that share a tile's rows; and with, where only pairs do."""
    g = torch.Generator(device=dev).manual_seed(rows)
    for act, i in (("bf16", 0), ("f16", 1)):
        dy, x = (torch.randn((rows, n), generator=g, device=dev).to(plain.DT[act]) for n in (N, K))
        add = torch.randn((N, K), generator=g, device=dev)
        ref, mag = dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs()
        for off in (None, torch.tensor([0, rows], dtype=torch.int32, device=dev)):
            for f32, addend in ((False, None), (True, None), (True, add), (True, "in place")):
                outs = []
                for _ in range(2):
                    dw = torch.full((N, K), 3.0, dtype=torch.float32 if f32 else plain.DT[act], device=dev)
                    if addend == "in place":
                        dw = add.clone()
                    moe.moe_ragged_wgrad(dy, x, i, off, rows, N, K, 1, dw if addend == "in place" else addend, dw, f32)
                    outs.append(dw)
                assert torch.equal(*outs)
                if f32:
                    want, m = (ref + add.double(), mag + add.double().abs()) if addend is not None else (ref, mag)
                    assert torch.all((dw.double() - want).abs() <= sum_slack(m, rows + 1))
                    assert float((dw.double() - want).norm()) <= (4096 / 16 / 2 + 16) * F32 * float(want.norm())
                else:
                    plain.close(dw, ref.cpu(), act, sum_slack(mag, rows).cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,N,K", [([0, 9, 25, 0], 840, 1320), ([2, 1, 0], 72, 4104), ([60, 3, 65], 520, 200),
                                        ([128], 136, 2056), ([7] * 16, 512, 520), ([1] * 128, 136, 72), ([0] * 4, 72, 72)])
def test_few_rows_of_groups(moe, dev, counts, N, K, transposed):
    for j, act in enumerate(("bf16", "f16")):
        ragged_case(moe, dev, counts, N, K, act, transposed, 7 + j)
        if sum(counts) <= 100:
            ragged_case(moe, dev, counts, N, K, act, transposed, 9 + j, lead=5, tail=20)


@pytest.mark.gpu
@pytest.mark.parametrize("f32,addend", [(True, None), (True, "in place"), (False, None)])
@pytest.mark.parametrize("counts,N,K", [([30, 0, 65, 2, 17], 2056, 1416), ([5, 21] * 20, 520, 296), ([100, 1], 4104, 1000),
                                        ([19] * 64, 776, 328), ([140, 9, 70], 136, 8200)])
def test_weight_gradient_of_uneven_tiles_over_many_waves(moe, dev, counts, N, K, f32, addend):
    wgrad_case(moe, dev, counts, N, K, "bf16" if N % 16 else "f16", f32, addend, N, lead=3, tail=4)


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[0, 5, 4, 9], [-1, 3, 5, 9], [0, 3, 5, 11], [2 ** 31 - 1, 0, 5, 9], [5, 3, 2, 1]])
def test_bad_offsets_are_reported_and_compute_nothing(moe, dev, off):
    off = torch.tensor(off, dtype=torch.int32, device=dev)
    x, w = torch.ones((10, 64), device=dev).bfloat16(), torch.ones((3, 64, 64), device=dev).bfloat16()
    for call in range(3):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.full((10, 64) if call < 2 else (3, 64, 64), 5.0, device=dev)
        if call < 2:
            out = out.bfloat16()
            moe.moe_ragged_gemm(x, 0, w, call, off, 10, 64, 64, 3, out, err)
        else:
            moe.moe_ragged_wgrad(x, x, 0, off, 10, 64, 64, 3, None, out, True, err)
        torch.cuda.synchronize()
        assert err.item() == moe.MOE_DEV_ERR_OFFSETS and torch.all(out == 5)


# ---- dense product ------------------------------------------------------------------------------

def fn_error(name, z, dz):
    """How far f of a z that is off by dz may be: its slope is within 1.2, and the functions are good to 24 ulp of
    their value, beside an exponential whose error grows with |z| and weighs z / (1 + exp(|z|)) or less."""
    f, _ = f64(name, z)
    if name in ("none", "relu"):
        return dz
    return 1.2 * dz + (24 * 2 * f.abs() + 8 * z.abs() * torch.exp(-z.abs().clamp(max=80) / 2)) * F32


def dense_case(moe, dev, M, N, K, act, fn, bias, residual, pre, seed):
    g = gen(seed)
    a, w = randn(g, M, K, act=act), randn(g, N, K, act=act, std=1.5 / math.sqrt(K))
    b = randn(g, N, act=act) if bias else None
    r = randn(g, M, N, act=act, std=3.0) if residual else None
    d = plain.DT[act]
    on = lambda t: t.to(dev) if t is not None else None  # noqa: E731
    out = on(r) if residual == "in place" else torch.empty((M, N), dtype=d, device=dev)
    z_out = torch.empty((M, N), dtype=d, device=dev) if pre else None
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_dense_gemm(on(a), moe.ACT_CODES[act], on(w), on(b), moe.FN_CODES[fn],
                       out if residual == "in place" else on(r), z_out, out, M, N, K, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    z, mag = a.double() @ w.double().T, a.double().abs() @ w.double().abs().T
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    dz = sum_slack(mag, K)
    if pre:
        plain.close(z_out, z, act, dz)
    ref, slack = f64(fn, z)[0], fn_error(fn, z, dz)
    if residual:
        ref = ref + r.double()
        slack = slack + ref.abs() * F32
    plain.close(out, ref, act, slack)
    return out, z_out


DENSE = [(1, 8, 8), (1, 2816, 2048), (2, 264, 1032), (3, 2048, 1408), (5, 72, 200), (8, 4104, 136), (9, 520, 264),
         (16, 2056, 72), (17, 136, 4104), (31, 1000, 520), (33, 264, 2056), (37, 4096, 776), (64, 72, 64),
         (100, 1032, 1032), (129, 520, 328), (257, 264, 136), (333, 2816, 264), (700, 136, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(DENSE)))
def test_dense_product_matches_the_formula(moe, dev, i):
    M, N, K = DENSE[i]
    for j in range(5):
        dense_case(moe, dev, M, N, K, ["bf16", "f16"][(i + j) % 2], FNS[j], (i + j) % 3 > 0,
                   [None, "apart", "in place"][(i + 2 * j) % 3], (i * j) % 2 == 0, 1000 * i + j)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (7, 28672, 1408), (13, 4096, 14336), (37, 4096, 14336),
                                   (61, 2048, 4096), (200, 4096, 4096), (1333, 2816, 2048), (2100, 4096, 1408)])
def test_dense_product_of_layers(moe, dev, M, N, K):
    act = "bf16"
    g = torch.Generator(device=dev).manual_seed(M)
    a = torch.randn((M, K), generator=g, device=dev).bfloat16()
    w = (torch.randn((N, K), generator=g, device=dev) * 0.02).bfloat16()
    b = torch.randn(N, generator=g, device=dev).bfloat16()
    r = torch.randn((M, N), generator=g, device=dev).bfloat16()
    outs = []
    for _ in range(2):
        out, z = torch.empty_like(r), torch.empty_like(r)
        moe.moe_dense_gemm(a, 0, w, b, moe.FN_CODES["gelu_tanh"], r, z, out, M, N, K)
        outs.append((out, z))
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    ref = a.double() @ w.double().T + b.double()
    dz = sum_slack(a.double().abs() @ w.double().abs().T + b.double().abs(), K)
    plain.close(z, ref.cpu(), act, dz.cpu())
    full = f64("gelu_tanh", ref)[0] + r.double()
    plain.close(out, full.cpu(), act, (fn_error("gelu_tanh", ref, dz) + full.abs() * F32).cpu())


# sizes at which products of one group take each of their forms: streaming with 8, 16 and 32 rows and several tiles a
# CTA, one to eight CTAs to a tile, one and several row tiles, pairs
FORMS = [(5, 9736, 72), (16, 9736, 136), (30, 9736, 200), (24, 136, 1032), (40, 264, 8192), (150, 520, 4096),
         (300, 264, 4104), (33, 1000, 1032), (600, 4104, 520), (614, 1648, 4336), (1000, 4096, 1032), (90, 28672, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", FORMS)
def test_products_of_one_group_in_every_form(moe, dev, M, N, K):
    """Without offsets, and with: the group's size is then known on the device alone."""
    g = torch.Generator(device=dev).manual_seed(M + N)
    for act, i in (("bf16", 0), ("f16", 1)):
        dt = plain.DT[act]
        w = (torch.randn((N, K), generator=g, device=dev) / math.sqrt(K)).to(dt)
        for tr in (False, True):
            a = torch.randn((M, N if tr else K), generator=g, device=dev).to(dt)
            outs = []
            for off in (None, torch.tensor([0, M], dtype=torch.int32, device=dev)):
                for _ in range(2):
                    out = torch.empty((M, K if tr else N), dtype=dt, device=dev)
                    moe.moe_ragged_gemm(a, i, w, tr, off, M, N, K, 1, out)
                    outs.append(out)
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3])
            we = w.double() if tr else w.double().T
            ref, mag = a.double() @ we, a.double().abs() @ we.abs()
            for out in outs[::2]:
                plain.close(out, ref.cpu(), act, sum_slack(mag, N if tr else K).cpu())
        b, r = torch.randn(N, generator=g, device=dev).to(dt), torch.randn((M, N), generator=g, device=dev).to(dt)
        a = torch.randn((M, K), generator=g, device=dev).to(dt)
        z = torch.empty_like(r)
        out = r.clone()
        moe.moe_dense_gemm(a, i, w, b, moe.FN_CODES["gelu"], out, z, out, M, N, K)
        ref = a.double() @ w.double().T + b.double()
        dz = sum_slack(a.double().abs() @ w.double().abs().T + b.double().abs(), K)
        plain.close(z, ref.cpu(), act, dz.cpu())
        full = f64("gelu", ref)[0] + r.double()
        plain.close(out, full.cpu(), act, (fn_error("gelu", ref, dz) + full.abs() * F32).cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [1, 100, 1500, 4000])
@pytest.mark.parametrize("M,N,K", [(40, 264, 8192), (150, 520, 4096), (300, 2056, 328)])
def test_split_product_ends_whatever_wait_runs_out(moe, dev, M, N, K, limit_ns):
    """Limits that may run out at its start, in its middle or not at all, with operands that are in no cache: the call
    ends, a result that is not the clean one is reported, and the next call at the default limit is the clean one."""
    g = torch.Generator(device=dev).manual_seed(1)
    a, w = (torch.randn(s, generator=g, device=dev).bfloat16() for s in ((M, K), (N, K)))
    want, out = (torch.empty((M, N), dtype=torch.bfloat16, device=dev) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_dense_gemm(a, 0, w, None, 0, None, None, want, M, N, K, err)
    torch.empty(1 << 28, device=dev).zero_()
    old = moe.moe_set_wait_limit_ns(limit_ns)
    try:
        moe.moe_dense_gemm(a, 0, w, None, 0, None, None, out, M, N, K, err)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(old)
    assert err.item() in (0, moe.MOE_DEV_ERR_TIMEOUT)
    assert err.item() or torch.equal(out, want)
    err.zero_()
    moe.moe_dense_gemm(a, 0, w, None, 0, None, None, out, M, N, K, err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [1, 100, 1500, 4000])
@pytest.mark.parametrize("counts,N,K", [([30, 0, 41, 29], 520, 4096), ([5] * 16, 136, 328)])
def test_split_groups_end_whatever_wait_runs_out(moe, dev, counts, N, K, limit_ns):
    """As above, few rows of several groups, both directions; and the gradient of one group's weight, whose tiles
    the same kernel splits."""
    rows, E = sum(counts), len(counts)
    g = torch.Generator(device=dev).manual_seed(2)
    a, b, w = (torch.randn(s, generator=g, device=dev).bfloat16() for s in ((rows, K), (rows, N), (E, N, K)))
    dy, x = (torch.randn(s, generator=g, device=dev).bfloat16() for s in ((4096, 264), (4096, 136)))
    off = offsets_of(counts).to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def calls():
        outs = [torch.empty(s, dtype=torch.bfloat16, device=dev) for s in ((rows, N), (rows, K))]
        outs.append(torch.zeros((264, 136), device=dev))
        return outs, (lambda: moe.moe_ragged_gemm(a, 0, w, False, off, rows, N, K, E, outs[0], err),
                      lambda: moe.moe_ragged_gemm(b, 0, w, True, off, rows, N, K, E, outs[1], err),
                      lambda: moe.moe_ragged_wgrad(dy, x, 0, None, 4096, 264, 136, 1, None, outs[2], True, err))

    want, run = calls()
    for f in run:
        f()
    outs, run = calls()
    for i, f in enumerate(run):
        torch.empty(1 << 28, device=dev).zero_()
        old = moe.moe_set_wait_limit_ns(limit_ns)
        try:
            f()
            torch.cuda.synchronize()
        finally:
            moe.moe_set_wait_limit_ns(old)
        assert err.item() in (0, moe.MOE_DEV_ERR_TIMEOUT)
        assert err.item() or torch.equal(outs[i], want[i])
        err.zero_()
        f()
        torch.cuda.synchronize()
        assert err.item() == 0 and torch.equal(outs[i], want[i])


@pytest.mark.gpu
def test_dense_block_refuses_its_own_buffers(moe, dev):
    from mixture_experts_grouped_gb300 import train
    bf = dict(dtype=torch.bfloat16, device=dev)
    block = train.DenseMlp(4, 64, 32, "bf16", "gelu", torch.zeros((32, 64), **bf), None, torch.zeros((64, 32), **bf), None)
    x = torch.ones((4, 64), **bf)
    out = block.forward(x)
    with pytest.raises(ValueError):
        block.forward(out)
    with pytest.raises(ValueError):
        block.forward(block.backward(x))
    block.forward(x, residual=out)  # (added in place, each element by the thread that writes it)


@pytest.mark.gpu
def test_tensors_past_32_bits_of_elements(moe, dev):
    """Rows, weights and gradients whose offsets pass 2^31 elements (4.3 GB each)."""
    H, R = 8192, 270000
    g = torch.Generator(device=dev).manual_seed(3)
    bf = dict(dtype=torch.bfloat16, device=dev)

    def near_rows(got, ref):
        assert float((got.double() - ref).abs().max()) <= 2 * plain.U["bf16"] * float(ref.abs().max())

    # a product with that many output elements: the last rows
    a, w = torch.randn((R, 64), generator=g, device=dev).bfloat16(), torch.randn((H, 64), generator=g, device=dev).bfloat16()
    big = torch.empty((R, H), **bf)
    moe.moe_dense_gemm(a, 0, w, None, 0, None, None, big, R, H, 64)
    for lo in (0, 262140, R - 40):
        near_rows(big[lo:lo + 40], a[lo:lo + 40].double() @ w.double().T)
    # its rows as the operand of the input's gradient, in two groups, and of the weight's gradient
    off = torch.tensor([0, 262150, R], dtype=torch.int32, device=dev)
    ww = torch.stack((w, w.flip(0))).contiguous()
    back = torch.empty((R, 64), **bf)
    moe.moe_ragged_gemm(big, 0, ww, True, off, R, H, 64, 2, back)
    near_rows(back[-40:], big[-40:].double() @ ww[1].double())
    near_rows(back[262100:262150], big[262100:262150].double() @ ww[0].double())
    dw = torch.empty((2, H, 64), device=dev)
    moe.moe_ragged_wgrad(big, a, 0, off, R, H, 64, 2, None, dw, True)
    ref = big[262150:].double().T @ a[262150:].double()
    assert float((dw[1].double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())
    # SwiGLU of a gate/up product that long, and its gradient
    h, dgu, dh = torch.empty((R, H // 2), **bf), torch.empty((R, H), **bf), a[:, :8].repeat(1, H // 16)
    moe.moe_swiglu(big, 0, R, H // 2, h)
    moe.moe_swiglu_backward(big, dh, 0, R, H // 2, dgu, None)
    t = big[-3:].double()
    near_rows(h[-3:], t[:, : H // 2] * torch.sigmoid(t[:, : H // 2]) * t[:, H // 2:])
    near_rows(dgu[-3:, H // 2:], dh[-3:].double() * t[:, : H // 2] * torch.sigmoid(t[:, : H // 2]))
    db = torch.empty(H, device=dev)
    moe.moe_bias_act_backward(big, dgu, 0, 1, R, H, dgu, db)
    t = torch.where(dgu[-3:] != 0, big[-3:], 0)
    assert torch.equal(dgu[-3:], t)
    # rows to such places, and the gradients back from them
    rows = torch.randperm(R, generator=gen(4))[:64].int()
    rows[:2] = torch.tensor([R - 1, R - 2])
    rows = rows.unique().to(dev)[-32:].contiguous()
    x = torch.randn((16, H), generator=g, device=dev).bfloat16()
    moe.moe_dispatch(x, 0, rows, big, 16, H, 2, R)
    assert torch.equal(big[rows.long()], x.repeat_interleave(2, 0))
    wt, d_w = torch.rand((16, 2), generator=g, device=dev), torch.empty((16, 2), device=dev)
    moe.moe_combine_backward(x, big, 0, rows, wt, big, d_w, 16, H, 2, R)
    near_rows(big[rows.long()].unflatten(0, (16, 2)), wt.double()[..., None] * x.double()[:, None])
    ref = (x.double() ** 2).sum(1, keepdim=True).expand(16, 2)
    assert torch.allclose(d_w.double(), ref, rtol=1e-5)
    del big, dgu, dh, h, a, back
    # a weight that long: 130 experts of 4096 x 4096
    E, N = 130, 4096
    w = torch.zeros((E, N, N), **bf)
    w[-1].normal_(generator=g)
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    off[-1] = 20
    x, out = torch.randn((20, N), generator=g, device=dev).bfloat16(), torch.empty((20, N), **bf)
    for tr in (False, True):
        moe.moe_ragged_gemm(x, 0, w, tr, off, 20, N, N, E, out)
        near_rows(out, x.double() @ (w[-1].double() if tr else w[-1].double().T))
    moe.moe_ragged_wgrad(x, out, 0, off, 20, N, N, E, None, w, False)
    near_rows(w[-1], x.double().T @ out.double())
    assert torch.all(w[:-1:43] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 20, 150])
def test_dense_product_keeps_non_finite_values_apart(moe, dev, M):
    N, K = 264, 200
    g = gen(M)
    a, w, b = randn(g, M, K), randn(g, N, K), randn(g, N)
    outs = []
    for bad in (False, True):
        if bad:
            a[1, 7], w[9, 3], b[20] = float("nan"), float("inf"), float("nan")
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        moe.moe_dense_gemm(a.to(dev), 0, w.to(dev), b.to(dev), 0, None, None, out, M, N, K)
        outs.append(out.cpu())
    rows, cols = torch.arange(M) != 1, (torch.arange(N) != 9) & (torch.arange(N) != 20)
    assert torch.equal(outs[0][rows][:, cols], outs[1][rows][:, cols])
    assert torch.isnan(outs[1][1]).all() and torch.isnan(outs[1][:, 20]).all()
    assert not torch.isfinite(outs[1][:, 9].float()).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_activation_functions_over_their_range(moe, dev, fn, act):
    """z from -inf to inf: the product of one column with 1 is z itself."""
    top = float(torch.finfo(plain.DT[act]).max)
    z = torch.cat([torch.linspace(-100, 100, 4001), torch.linspace(-8, 8, 4001),
                   torch.tensor([0.0, -0.0, top, -top, top / 3, -top / 3, 1e-4, -1e-4])]).to(plain.DT[act])
    z = z[: len(z) // 8 * 8]
    n = len(z)
    a = torch.zeros((1, 8), dtype=z.dtype)
    a[0, 0] = 1
    w = torch.zeros((n, 8), dtype=z.dtype)
    w[:, 0] = z
    out = torch.empty((1, n), dtype=z.dtype, device=dev)
    moe.moe_dense_gemm(a.to(dev), moe.ACT_CODES[act], w.to(dev), None, moe.FN_CODES[fn], None, None, out, 1, n, 8)
    ref, slope = f64(fn, z.double())
    # below f32's normal range, and silu below -87.3, values may count as 0
    tiny = 1.2e-36
    slack = (48 * ref.abs() + 8 * z.double().abs() * torch.exp(-z.double().abs().clamp(max=80) / 2)) * F32 + tiny
    plain.close(out[0], ref, act, slack)
    g = torch.full((1, n), 0.75, dtype=z.dtype, device=dev)
    moe.moe_bias_act_backward(g, z[None].to(dev), moe.ACT_CODES[act], moe.FN_CODES[fn], 1, n, out)
    # slopes lie within 1.2; their terms are each good to a few ulp beside an exponential as above
    slack = (48 + 16 * z.double().abs() * torch.exp(-z.double().abs().clamp(max=80) / 2)) * F32 + tiny
    plain.close(out[0], 0.75 * slope, act, slack)


@pytest.mark.gpu
def test_activation_functions_pass_nan_on(moe, dev):
    z = torch.tensor([float("nan")] * 8).bfloat16()[None].to(dev)
    g, out = torch.ones_like(z), torch.empty_like(z)
    for fn in FNS[1:]:
        moe.moe_bias_act_backward(g, z, 0, moe.FN_CODES[fn], 1, 8, out)
        assert torch.isnan(out).all(), fn
        a = torch.zeros((1, 8), dtype=torch.bfloat16, device=dev)
        a[0, 0] = float("nan")
        moe.moe_dense_gemm(a, 0, torch.ones((8, 8), device=dev).bfloat16(), None, moe.FN_CODES[fn], None, None, out, 1,
                           8, 8)
        assert torch.isnan(out).all(), fn


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 72), (31, 64), (33, 200), (65, 136), (300, 1032), (1333, 264)])
def test_bias_and_activation_gradient_matches_the_formula(moe, dev, M, N, act):
    for i, fn in enumerate(FNS):
        g = gen(M + N + i)
        d, z = randn(g, M, N, act=act), randn(g, M, N, act=act, std=2.0)
        dz = d.double() * f64(fn, z.double())[1]
        slack = d.double().abs() * (48 + 16) * F32
        for want in ("both", "dz", "bias", "sum"):
            dp = torch.empty((M, N), dtype=plain.DT[act], device=dev) if want in ("both", "dz") else None
            db = torch.full((N,), 2.0, device=dev) if want != "dz" else None
            moe.moe_bias_act_backward(d.to(dev), z.to(dev) if fn != "none" else None, moe.ACT_CODES[act],
                                      moe.FN_CODES[fn], M, N, dp, db, want == "sum")
            if dp is not None:
                plain.close(dp, dz, act, slack)
            if db is not None:
                ref = dz.sum(0) + (2.0 if want == "sum" else 0.0)
                assert torch.all((db.cpu().double() - ref).abs()
                                 <= (slack + dz.abs() * F32 * (M + 16)).sum(0) + 2 * (ref.abs() + 2) * F32)
    same = d.to(dev)
    moe.moe_bias_act_backward(same, z.to(dev), moe.ACT_CODES[act], 4, M, N, same)      # in place
    assert torch.equal(same, dp) if dp is not None else True


# ---- SwiGLU ---------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("rows,I", [(1, 8), (1, 768), (3, 136), (64, 1408), (1000, 72), (33, 14336), (255, 264)])
def test_swiglu_and_its_gradient_match_the_formula(moe, dev, act, rows, I):
    g = gen(rows + I)
    gu, dh = randn(g, rows, 2 * I, act=act, std=3.0), randn(g, rows, I, act=act)
    if rows > 2:
        gu[1] = 0
        gu[2, : I // 2] = -200.0  # exp overflows f32
    code = moe.ACT_CODES[act]
    h, dgu, h2 = (torch.full((rows, n), 9.0, dtype=plain.DT[act], device=dev) for n in (I, 2 * I, I))
    moe.moe_swiglu(gu.to(dev), code, rows, I, h)
    moe.moe_swiglu_backward(gu.to(dev), dh.to(dev), code, rows, I, dgu, h2)
    assert torch.equal(h, h2)
    gg, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    f, df = f64("silu", gg)
    # a few ulp of each factor, beside the exponential's error, which grows with |g| and weighs exp(-|g|) |g|
    e = (48 + 16 * gg.abs() * torch.exp(-gg.abs().clamp(max=80) / 2)) * F32
    plain.close(h, f * u, act, (f.abs() * e + 1.2e-36) * u.abs())
    ref = torch.cat((d * u * df, d * f), 1)
    slack = torch.cat(((d * u).abs() * (e + 1.2e-36), d.abs() * (f.abs() * e + 1.2e-36)), 1)
    plain.close(dgu, ref, act, slack)
    same, hh = gu.to(dev), dh.to(dev)
    moe.moe_swiglu_backward(same, hh, code, rows, I, same, hh)                          # both in place
    assert torch.equal(same, dgu) and torch.equal(hh, h)
    same = gu.to(dev)
    moe.moe_swiglu_backward(same, dh.to(dev), code, rows, I, same)                      # without h
    assert torch.equal(same, dgu)


# ---- rows to the experts, gradients of combine and routing ------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (5, 136, 2), (61, 2048, 8), (33, 4096, 3), (7, 8200, 16), (300, 72, 5)])
def test_dispatch_and_combine_gradient_match_the_formula(moe, dev, act, T, H, k):
    g, code = gen(T * k), moe.ACT_CODES[act]
    rows = T * k + 3
    row = torch.randperm(rows, generator=g)[: T * k].int()
    if T > 4:
        row[[1, 7]] = torch.tensor([-1, -5], dtype=torch.int32)       # dropped
        row[9] = rows                                                 # out of range
    x, d, y = randn(g, T, H, act=act), randn(g, T, H, act=act), randn(g, rows, H, act=act)
    w = torch.rand((T, k), generator=g)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    xs = torch.full((rows, H), 3.0, dtype=plain.DT[act], device=dev)
    moe.moe_dispatch(x.to(dev), code, row.to(dev), xs, T, H, k, rows, err)
    assert err.item() == (moe.MOE_DEV_ERR_PAIR_ID if T > 4 else 0)
    err.zero_()
    dy, dw = torch.full_like(xs, 3.0), torch.full((T, k), 9.0, device=dev)
    moe.moe_combine_backward(d.to(dev), y.to(dev), code, row.to(dev), w.to(dev), dy, dw, T, H, k, rows, err)
    assert err.item() == (moe.MOE_DEV_ERR_PAIR_ID if T > 4 else 0)
    ref_x, ref_dy = torch.full((rows, H), 3.0, dtype=x.dtype), torch.full((rows, H), 3.0, dtype=torch.float64)
    for p, r in enumerate(row.tolist()):
        t, j = divmod(p, k)
        if 0 <= r < rows:
            ref_x[r], ref_dy[r] = x[t], w[t, j].double() * d[t].double()
            prod = d[t].double() * y[r].double()
            assert abs(dw[t, j].item() - prod.sum().item()) <= prod.abs().sum().item() * (H / 8 + 24) * F32
        else:
            assert dw[t, j].item() == 0
    assert torch.equal(xs.cpu(), ref_x)
    plain.close(dy, ref_dy, act, ref_dy.abs() * F32)
    again = y.to(dev)
    moe.moe_combine_backward(d.to(dev), again, code, row.to(dev), w.to(dev), again, dw, T, H, k, rows, err)  # in place
    hit = row[(row >= 0) & (row < rows)].long().to(dev)
    assert torch.equal(again[hit], dy[hit])


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (61, 128, 8), (130, 256, 16), (9, 40, 3), (4, 33, 16)])
def test_routing_gradient_matches_the_formula_and_differences(moe, dev, T, E, k, renorm):
    g = gen(T + E)
    logits = 2 * torch.randn((T, E), generator=g)
    if T > 4:
        logits[3, E // 2:] = -math.inf if k <= E // 2 else 0.0   # experts that are masked away
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), device=dev)
    moe.moe_route_topk_softmax(logits.to(dev), ids, w, T, E, k, renorm)
    dw = torch.randn((T, k), generator=g)
    dl = torch.full((T, E), 9.0, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_route_backward(None if renorm else logits.to(dev), ids, w, dw.to(dev), dl, T, E, k, renorm, err)
    assert err.item() == 0
    at = ids.cpu().long()

    def loss(l):  # the weights of fixed ids
        p = torch.softmax(l.gather(1, at), 1) if renorm else torch.softmax(l, 1).gather(1, at)
        return (p * dw.double()).sum(1)

    l = logits.double()
    p = torch.softmax(torch.full_like(l, -math.inf).scatter(1, at, l.gather(1, at)) if renorm else l, 1)
    gr = torch.zeros_like(l).scatter(1, at, dw.double())
    ref = p * (gr - (p * gr).sum(1, keepdim=True))
    # the weights are f32, their sum of k products and the difference round a few times
    slack = p * (2 * gr.abs() + 4 * (p * gr.abs()).sum(1, keepdim=True)) * (k + 24) * F32 + 1e-38
    assert torch.all((dl.cpu().double() - ref).abs() <= slack)
    h = 1e-5
    for e in range(min(E, 6)):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        num = (loss(l + step) - loss(l - step)) / (2 * h)
        # central differences: h^2 / 6 times a third derivative below 6 |dw|, and rounding of 64-bit losses
        assert torch.all((num - dl[:, e].cpu().double()).abs() <= slack[:, e] + dw.abs().double().sum(1) * (h * h + 1e-10))


@pytest.mark.gpu
def test_routing_gradient_of_odd_ids(moe, dev):
    """An expert named twice gets both slots' parts; ids outside the experts take no part and are reported."""
    ids = torch.tensor([[1, 1, 3], [2, 9, -1]], dtype=torch.int32, device=dev)
    w = torch.tensor([[0.5, 0.25, 0.25], [0.7, 0.2, 0.1]], device=dev)
    dw = torch.tensor([[1.0, 2.0, 4.0], [3.0, 50.0, 60.0]], device=dev)
    dl, err = torch.empty((2, 4), device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_route_backward(None, ids, w, dw, dl, 2, 4, 3, True, err)
    assert err.item() == moe.MOE_DEV_ERR_EXPERT_ID
    m0, m1 = 0.5 + 0.5 + 1.0, 2.1
    want = torch.tensor([[0, 0.5 * (1 - m0) + 0.25 * (2 - m0), 0, 0.25 * (4 - m0)], [0, 0, 0.7 * (3 - m1), 0]])
    assert torch.allclose(dl.cpu(), want, rtol=1e-5, atol=1e-6)


# ---- together ---------------------------------------------------------------------------------------

def layer_f64(x, ids, w, wgu, wd):
    """The expert layer in 64 bits from leaves that may ask for gradients."""
    T, H = x.shape
    I = wd.shape[2]
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    for e in range(wgu.shape[0]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(tok):
            gu = x[tok] @ wgu[e].T
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            out = out.index_add(0, tok, (h @ wd[e].T) * w[tok, slot][:, None])
    return out


def near(got, ref, rel):
    got, ref = got.cpu().double(), ref.cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    assert float((got - ref).norm()) <= rel * float(ref.norm()), float((got - ref).norm() / ref.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,I,E,k,renorm", [(1, 64, 72, 4, 2, True), (37, 136, 200, 5, 3, False),
                                              (300, 512, 256, 16, 4, True), (5, 2048, 768, 128, 8, True)])
def test_training_step_of_the_layer(moe, dev, T, H, I, E, k, renorm, act):
    from mixture_experts_grouped_gb300 import train
    g, dt = gen(T + H), plain.DT[act]
    x, logits = randn(g, T, H, act=act).to(dev), torch.randn((T, E), generator=g).to(dev)
    wgu = randn(g, E, 2 * I, H, act=act, std=1 / math.sqrt(H)).to(dev)
    wd = randn(g, E, H, I, act=act, std=1 / math.sqrt(I)).to(dev)
    d_out = randn(g, T, H, act=act).to(dev)
    layer = train.MoeTrainLayer(T, H, I, E, k, act, wgu, wd, dev, renorm)
    out = layer.forward(x, logits).clone()
    dx, dl = (t.clone() for t in layer.backward(d_out))
    dgu, dd = layer.d_gate_up.clone(), layer.d_down.clone()
    assert layer.err.item() == 0
    leaves = [t.double().requires_grad_() for t in (x, logits, wgu, wd)]
    at = layer.topk_ids.long()
    l = leaves[1]
    w = torch.softmax(l.gather(1, at), 1) if renorm else torch.softmax(l, 1).gather(1, at)
    ref = layer_f64(leaves[0], at, w, leaves[2], leaves[3])
    ref.backward(d_out.double())
    # each quantity passes at most seven roundings to 16 bits of relative size u on its way (gate_up, h, y, d_y, d_h,
    # d_gate_up, its own), none of which a later step amplifies by more than a few in the 2-norm
    rel = 7 * 2 * plain.U[act]
    for got, leaf in zip((dx, dl, dgu, dd), leaves):
        near(got, leaf.grad, rel)
    near(out, ref.detach(), rel)
    # gradients accumulate; a second backward pass of one forward pass gives the same
    assert all(torch.equal(a, b) for a, b in zip((dx, dl), layer.backward(d_out, accumulate=True)))
    near(layer.d_gate_up, 2 * dgu, 8 * F32)
    near(layer.d_down, 2 * dd, 8 * F32)
    # a captured step on another stream's graph gives the same bits, also of changed inputs
    graph = torch.cuda.CUDAGraph()
    xg, lg, dg = x.clone(), logits.clone(), d_out.clone()
    with torch.cuda.graph(graph):
        layer.forward(xg, lg)
        layer.backward(dg)
    xg.mul_(-1)
    graph.replay()
    xg.copy_(x)
    for t in (layer.out, layer.d_x, layer.d_logits, layer.d_gate_up, layer.d_down):
        t.fill_(float("nan"))
    graph.replay()
    for a, b in zip((out, dx, dl, dgu, dd), (layer.out, layer.d_x, layer.d_logits, layer.d_gate_up, layer.d_down)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_training_objects_refuse_what_does_not_fit(moe, dev):
    from mixture_experts_grouped_gb300 import train
    T, H, I, E, k, bf = 4, 64, 32, 3, 2, dict(dtype=torch.bfloat16, device=dev)
    w = torch.zeros((E, 2 * I, H), **bf), torch.zeros((E, H, I), **bf)
    layer = train.MoeTrainLayer(T, H, I, E, k, "bf16", *w)
    assert torch.all(layer.d_gate_up == 0) and torch.all(layer.d_down == 0)
    x, logits = torch.zeros((T, H), **bf), torch.zeros((T, E), device=dev)
    n0 = moe.moe_launch_count()
    with pytest.raises(RuntimeError):
        layer.backward(x)
    for bad_x, bad_l in ((x[:3], logits), (x.half(), logits), (x.T.contiguous().T, logits), (x.cpu(), logits),
                         (x, logits.double()), (x, logits[:, :2]), (x, logits.cpu())):
        with pytest.raises(ValueError):
            layer.forward(bad_x, bad_l)
    for args in ((0, H, I, E, k, "bf16", *w), (T, H, I, E, k, "f16", *w), (T, H, I, E, k, "bf16", w[0][:, ::2], w[1]),
                 (T, H, I, E, k, "bf16", w[0].cpu(), w[1])):
        with pytest.raises(ValueError):
            train.MoeTrainLayer(*args)
    m = [torch.zeros(s, **bf) for s in ((I, H), (I,), (H, I), (H,))]
    block = train.DenseMlp(T, H, I, "bf16", "gelu", *m)
    with pytest.raises(RuntimeError):
        block.backward(x)
    for bad in (dict(x=x[:, ::2]), dict(x=x.cpu()), dict(x=x, residual=x.half())):
        with pytest.raises(ValueError):
            block.forward(**bad)
    with pytest.raises(ValueError):
        train.DenseMlp(T, H, I, "bf16", "gelu", m[0], m[3], m[2], m[3])
    assert moe.moe_launch_count() == n0
    layer.forward(x, logits)
    with pytest.raises(ValueError):
        layer.backward(x.float())


@pytest.mark.gpu
def test_training_gradient_against_differences(moe, dev):
    """The loss sum(out * d_out) along the gradient's own direction, by differences of the layer's own outputs."""
    from mixture_experts_grouped_gb300 import train
    T, H, I, E, k, act = 48, 128, 96, 6, 2, "f16"
    g = gen(1)
    x, logits = randn(g, T, H, act=act).to(dev), torch.randn((T, E), generator=g).to(dev)
    wgu, wd = randn(g, E, 2 * I, H, act=act, std=0.1).to(dev), randn(g, E, H, I, act=act, std=0.1).to(dev)
    d_out = randn(g, T, H, act=act).to(dev)
    layer = train.MoeTrainLayer(T, H, I, E, k, act, wgu, wd, dev)
    layer.forward(x, logits)
    dx, dl = (t.clone() for t in layer.backward(d_out))
    dgu = layer.d_gate_up.clone()
    w0, x0, ids = wgu.clone(), x.clone(), layer.topk_ids.clone()

    def loss():
        out = layer.forward(x, logits)
        assert torch.equal(layer.topk_ids, ids)
        return float((out.double() * d_out.double()).sum())

    def check(t, t0, grad):
        """+- s along grad, s so that t moves by 4% of its norm; what 16 bits leave of the step counts."""
        s = 0.04 * float(t0.double().norm()) / float(grad.double().norm())
        t.copy_(t0 + s * grad.to(t0.dtype) if t0.dtype == torch.float32 else (t0.double() + s * grad.double()).to(t0.dtype))
        up, hi = loss(), t.clone()
        t.copy_((t0.double() - s * grad.double()).to(t0.dtype))
        down, lo = loss(), t.clone()
        t.copy_(t0)
        want = float(((hi.double() - lo.double()) * grad.double()).sum())
        # curvature over a 4% step, third order: (0.04)^2; outputs in 11 bits, T H of them, of random signs
        noise = float(d_out.double().norm()) * plain.U[act] * 3
        assert abs((up - down) - want) <= 0.02 * abs(want) + noise

    check(x, x0, dx)
    check(wgu, w0, dgu)


@pytest.mark.gpu
@pytest.mark.parametrize("fn,bias,T,H,I", [("gelu", True, 33, 136, 264), ("relu", False, 1, 64, 72),
                                           ("silu", True, 300, 256, 1032), ("none", False, 5, 72, 136)])
def test_dense_block_and_its_gradients(moe, dev, fn, bias, T, H, I):
    from mixture_experts_grouped_gb300 import train
    act = "bf16"
    g = gen(T)
    x, r, d_out = (randn(g, T, H).to(dev) for _ in range(3))
    w1, w2 = randn(g, I, H, std=1 / math.sqrt(H)).to(dev), randn(g, H, I, std=1 / math.sqrt(I)).to(dev)
    b1, b2 = (randn(g, n).to(dev) if bias else None for n in (I, H))
    block = train.DenseMlp(T, H, I, act, fn, w1, b1, w2, b2, dev)
    out = block.forward(x, r).clone()
    dx = block.backward(d_out).clone()
    assert block.err.item() == 0
    got = [dx] + [t.clone() for t in (block.d_w1, block.d_w2, block.d_b1, block.d_b2) if t is not None]
    leaves = [t.double().requires_grad_() for t in (x, w1, w2, b1, b2) if t is not None]
    X, W1, W2 = leaves[:3]
    z = X @ W1.T + (leaves[3] if bias else 0.0)
    f = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[fn](z)
    ref = f @ W2.T + (leaves[4] if bias else 0.0) + r.double()
    ref.backward(d_out.double())
    rel = 5 * 2 * plain.U[act]  # pre, h, d_h, dz, and the last one
    near(out, ref.detach(), rel)
    for a, leaf in zip(got, leaves):
        if fn == "relu":  # a z whose rounding changes its sign changes its slope by 1: |z| < u of its scale, u of them
            near(a, leaf.grad, rel + math.sqrt(4 * plain.U[act]))
        else:
            near(a, leaf.grad, rel)
    block.backward(d_out, accumulate=True)
    for a, b in zip(got[1:], (t for t in (block.d_w1, block.d_w2, block.d_b1, block.d_b2) if t is not None)):
        near(b, 2 * a, 8 * F32)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
def test_feed_forward_block_with_a_16_bit_shared_expert(moe, dev, T):
    from mixture_experts_grouped_gb300 import ffn
    from mixture_experts_grouped_gb300 import layer as L
    H, I, S, E, k, act = 256, 128, 192, 8, 2, "bf16"
    g = gen(T)
    wgu, wd = randn(g, E, 2 * I, H, std=0.06).to(dev), randn(g, E, H, I, std=0.06).to(dev)
    sgu, sd = randn(g, 2 * S, H, std=0.06).to(dev), randn(g, H, S, std=0.06).to(dev)
    desc = [L.DeviceWeight(moe.MoeWeight(moe.MOE_W_BF16, 0, t.data_ptr(), None, None, None), [t]) for t in (wgu, wd)]
    nw, wr = torch.ones(H, dtype=torch.bfloat16, device=dev), torch.randn((H, E), generator=g).to(dev)
    x, r = randn(g, T, H).to(dev), randn(g, T, H).to(dev)
    shared = ffn.DenseExpert(T, H, S, act, sgu, sd, dev)
    block = ffn.FeedForward(T, H, I, E, k, act, nw, wr, *desc, shared, device=dev)
    out, res = block.forward(x, r)
    bare = ffn.FeedForward(T, H, I, E, k, act, nw, wr, *desc, device=dev)
    routed, res0 = bare.forward(x, r)
    assert torch.equal(res, res0)
    y = bare.y.double()
    gu = y @ sgu.double().T
    h = gu[:, :S] * torch.sigmoid(gu[:, :S]) * gu[:, S:]
    near(out, routed.double() + h @ sd.double().T, 4 * 2 * plain.U[act])
    assert shared.err.item() == 0
    with pytest.raises(ValueError):
        ffn.FeedForward(T + 1, H, I, E, k, act, nw, wr, *desc, shared, device=dev)
    with pytest.raises(ValueError):
        ffn.DenseExpert(T, H, S, "f16", sgu, sd, dev)
    with pytest.raises(ValueError):
        ffn.DenseExpert(T, H, S, act, sgu, sd.T, dev)


@pytest.mark.gpu
def test_calls_on_streams_do_not_disturb_each_other(moe, dev):
    """Two products at once on two streams, one of them given by argument."""
    g = torch.Generator(device=dev).manual_seed(1)
    a = torch.randn((700, 1024), generator=g, device=dev).bfloat16()
    w = torch.randn((4, 512, 1024), generator=g, device=dev).bfloat16()
    off = torch.tensor([0, 100, 100, 650, 700], dtype=torch.int32, device=dev)
    want = torch.empty((700, 512), dtype=torch.bfloat16, device=dev)
    dwant = torch.empty((4, 512, 1024), device=dev)
    moe.moe_ragged_gemm(a, 0, w, False, off, 700, 512, 1024, 4, want)
    moe.moe_ragged_wgrad(want, a, 0, off, 700, 512, 1024, 4, None, dwant, True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want) for _ in range(8)]
    dws = [torch.zeros_like(dwant) for _ in range(8)]
    torch.cuda.synchronize()
    for o, d in zip(outs, dws):
        with torch.cuda.stream(s1):
            moe.moe_ragged_gemm(a, 0, w, False, off, 700, 512, 1024, 4, o)
        moe.moe_ragged_wgrad(want, a, 0, off, 700, 512, 1024, 4, None, d, True, None, s2)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(d, dwant) for d in dws)


# ---- refusals (no GPU) --------------------------------------------------------------------------------

A = 1 << 20  # an aligned address that no call reaches


@pytest.mark.parametrize("call", [
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, (1 << 30) + 1, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 0, A, 4, (1 << 30) + 8, 64, 2, None, A, 1, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 0, A, 4, 1 << 24, 1 << 24, 2, None, A, 1, 0, 0),     # too many tiles
    lambda m: m.moe_dense_gemm(A, 0, A, None, 0, None, None, A, 4, 64, (1 << 30) + 8, 0, 0),
    lambda m: m.moe_bias_act_backward(A, A, 0, 1, (1 << 30) + 1, 64, A, None, 0, 0),
    lambda m: m.moe_swiglu(A, 0, 1 << 30, 1 << 20, A, 0),
    lambda m: m.moe_swiglu_backward(A, A, 0, 1 << 30, 1 << 20, A, None, 0),
])
def test_what_is_beyond_the_limits_is_unsupported(moe, call):
    n0 = moe.moe_launch_count()
    with pytest.raises(moe.MoeError) as e:
        call(moe)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED and e.value.message
    assert moe.moe_launch_count() == n0


@pytest.mark.parametrize("call", [
    lambda m: m.moe_ragged_gemm(A, 2, A, 0, A, 4, 64, 64, 2, A, 0, 0),        # act
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, -1, 64, 64, 2, A, 0, 0),       # rows
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 60, 64, 2, A, 0, 0),        # N % 8
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 4, 2, A, 0, 0),         # K % 8
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 0, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 64, 0, A, 0, 0),        # E
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 64, 257, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, None, 4, 64, 64, 2, A, 0, 0),     # no offsets of two groups
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A + 2, 4, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(None, 0, A, 0, A, 4, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, None, 0, A, 4, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 64, 2, None, 0, 0),
    lambda m: m.moe_ragged_gemm(A + 8, 0, A, 0, A, 4, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, A + 8, 0, A, 4, 64, 64, 2, A, 0, 0),
    lambda m: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 64, 2, A + 8, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 7, A, 4, 64, 64, 2, None, A, 1, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 0, A, 4, 64, 64, 2, A, A, 0, 0, 0),    # an addend of a 16-bit gradient
    lambda m: m.moe_ragged_wgrad(A, A, 0, A, 4, 64, 64, 2, None, None, 1, 0, 0),
    lambda m: m.moe_ragged_wgrad(None, A, 0, A, 4, 64, 64, 2, None, A, 1, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 0, A, 4, 64, 64, 2, A + 4, A, 1, 0, 0),
    lambda m: m.moe_ragged_wgrad(A, A, 0, None, 4, 64, 64, 3, None, A, 1, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, None, 5, None, None, A, 4, 64, 64, 0, 0),   # fn
    lambda m: m.moe_dense_gemm(A, 0, A, None, -1, None, None, A, 4, 64, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 3, A, None, 0, None, None, A, 4, 64, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, None, 0, None, None, A, 4, 62, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, A + 2, 0, None, None, A, 4, 64, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, None, 0, A + 2, None, A, 4, 64, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, None, 0, None, A + 2, A, 4, 64, 64, 0, 0),
    lambda m: m.moe_dense_gemm(A, 0, A, None, 0, None, None, None, 4, 64, 64, 0, 0),
    lambda m: m.moe_bias_act_backward(A, A, 0, 9, 4, 64, A, A, 0, 0),
    lambda m: m.moe_bias_act_backward(A, None, 0, 1, 4, 64, A, A, 0, 0),            # relu without pre
    lambda m: m.moe_bias_act_backward(A, A, 0, 1, 4, 64, None, None, 0, 0),
    lambda m: m.moe_bias_act_backward(A, A, 0, 1, 4, 63, A, None, 0, 0),
    lambda m: m.moe_bias_act_backward(A + 2, A, 0, 1, 4, 64, A, None, 0, 0),
    lambda m: m.moe_swiglu(A, 0, -1, 64, A, 0),
    lambda m: m.moe_swiglu(A, 0, 4, 60, A, 0),
    lambda m: m.moe_swiglu(A, 9, 4, 64, A, 0),
    lambda m: m.moe_swiglu(None, 0, 4, 64, A, 0),
    lambda m: m.moe_swiglu_backward(A, None, 0, 4, 64, A, None, 0),
    lambda m: m.moe_swiglu_backward(A, A, 0, 4, 64, A, A + 2, 0),
    lambda m: m.moe_dispatch(A, 0, A, A, 4, 60, 2, 8, 0, 0),
    lambda m: m.moe_dispatch(A, 0, A, A, 4, 64, 17, 8, 0, 0),
    lambda m: m.moe_dispatch(A, 0, A, None, 4, 64, 2, 8, 0, 0),
    lambda m: m.moe_dispatch(A, 0, None, A, 4, 64, 2, 8, 0, 0),
    lambda m: m.moe_combine_backward(A, A, 0, A, A, A, A, -4, 64, 2, 8, 0, 0),
    lambda m: m.moe_combine_backward(A, A, 0, A, None, A, A, 4, 64, 2, 8, 0, 0),
    lambda m: m.moe_combine_backward(A, A + 8, 0, A, A, A, A, 4, 64, 2, 8, 0, 0),
    lambda m: m.moe_route_backward(None, A, A, A, A, 4, 8, 2, 0, 0, 0),             # logits are needed
    lambda m: m.moe_route_backward(A, A, A, A, A, 4, 8, 9, 1, 0, 0),
    lambda m: m.moe_route_backward(A, A, A, A, A, 4, 257, 2, 1, 0, 0),
    lambda m: m.moe_route_backward(A, A, A, A, None, 4, 8, 2, 1, 0, 0),
])
def test_misuse_is_refused_before_any_launch(moe, call):
    n0 = moe.moe_launch_count()
    with pytest.raises(moe.MoeError) as e:
        call(moe)
    assert e.value.status == moe.MOE_ERR_INVALID and e.value.message
    assert moe.moe_launch_count() == n0


def test_no_rows_is_a_no_op(moe):
    n0 = moe.moe_launch_count()
    moe.moe_ragged_gemm(None, 0, A, 0, A, 0, 64, 64, 2, None, 0, 0)
    moe.moe_dense_gemm(None, 0, A, None, 0, None, None, None, 0, 64, 64, 0, 0)
    moe.moe_bias_act_backward(None, None, 0, 1, 0, 64, A, None, 0, 0)
    moe.moe_swiglu(None, 0, 0, 64, None, 0)
    moe.moe_swiglu_backward(None, None, 0, 0, 64, None, None, 0)
    moe.moe_dispatch(None, 0, None, None, 0, 64, 2, 0, 0, 0)
    moe.moe_combine_backward(None, None, 0, None, None, None, None, 0, 64, 2, 0, 0, 0)
    moe.moe_route_backward(None, None, None, None, None, 0, 8, 2, 1, 0, 0)
    assert moe.moe_launch_count() == n0


def test_products_without_a_device_fail_with_a_status(moe):
    calls = """
import sys
from mixture_experts_grouped_gb300 import moe as m
A = 1 << 20
for call in (lambda: m.moe_ragged_gemm(A, 0, A, 0, A, 4, 64, 64, 2, A, 0, 0),
             lambda: m.moe_ragged_gemm(A, 0, A, 1, None, 400, 64, 64, 1, A, 0, 0),
             lambda: m.moe_dense_gemm(A, 0, A, None, 0, None, None, A, 4, 64, 64, 0, 0),
             lambda: m.moe_ragged_wgrad(A, A, 0, None, 4, 64, 64, 1, None, A, 1, 0, 0),
             lambda: m.moe_ragged_wgrad(A, A, 0, A, 4, 64, 64, 2, None, A, 0, 0, 0),
             lambda: m.moe_bias_act_backward(A, A, 0, 1, 4, 64, A, A, 0, 0),
             lambda: m.moe_swiglu(A, 0, 4, 64, A, 0),
             lambda: m.moe_dispatch(A, 0, A, A, 4, 64, 2, 8, 0, 0)):
    try:
        call()
    except m.MoeError as e:
        assert e.status == m.MOE_ERR_CUDA, e
    else:
        sys.exit("a call went through")
"""
    root = pathlib.Path(__file__).resolve().parents[1]
    r = subprocess.run([sys.executable, "-c", calls], cwd=root, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)


@pytest.mark.gpu
def test_gradients_of_no_rows_are_zeros(moe, dev):
    dw = torch.ones((3, 16, 24), device=dev)
    moe.moe_ragged_wgrad(None, None, 0, torch.zeros(4, dtype=torch.int32, device=dev), 0, 16, 24, 3, None, dw, True)
    assert torch.all(dw == 0)
    moe.moe_ragged_wgrad(None, None, 0, None, 0, 16, 24, 1, None, dw[0].fill_(2.0), True)
    assert torch.all(dw == 0)
    db = torch.ones(16, device=dev)
    moe.moe_bias_act_backward(None, None, 0, 0, 0, 16, None, db)
    assert torch.all(db == 0)
