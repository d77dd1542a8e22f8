"""The serving operators against plain 64-bit forms (tests/plain.py), and their refusals."""
import math

import pytest
import torch

import plain

FMTS = ["bf16", "fp8", "nvfp4", "gptq"]


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


# ---- residual addition + norm --------------------------------------------------------

def norm_case(moe, dev, x, res, w, act, eps=1e-6, **out):
    T, H = x.shape
    d = plain.DT[act]
    xs = x.to(dev)
    rs = res.to(dev) if res is not None else None
    r_out, y = torch.empty((T, H), dtype=d, device=dev), torch.empty((T, H), dtype=d, device=dev)
    q = torch.empty((T, H), dtype=torch.uint8, device=dev)
    s = torch.empty((T, -(-H // 128)), device=dev)
    moe.moe_add_rmsnorm_quant(xs, rs, moe.ACT_CODES[act], w.to(dev), eps, T, H, r_out, y, q, s)
    torch.cuda.synchronize()
    return r_out, y, q, s


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,residual", [
    (1, 8, True), (1, 2048, True), (5, 136, False), (3, 256, True), (7, 264, True), (9, 512, False), (130, 520, True),
    (33, 4096, True), (2, 8192, False), (3, 8200, True), (2, 16392, True), (2, 32768, True), (1500, 1000, True)])
def test_norm_matches_the_formula(moe, dev, act, T, H, residual):
    g = gen(T * 31 + H)
    x = torch.randn((T, H), generator=g).to(plain.DT[act])
    res = (3 * torch.randn((T, H), generator=g)).to(plain.DT[act]) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(plain.DT[act])
    if T > 2:
        x[1] = 0                                     # a row of zeros (with a residual of zeros)
        if residual:
            res[1] = 0
        x[2, : H // 2] = 0
    r_out, y, q, s = norm_case(moe, dev, x, res, w, act)
    r = x.double() + (res.double() if residual else 0)
    ref = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6) * w.double()
    # f32: the sum of squares (every term non-negative, at most 64 terms in a row, then a tree), the
    # reciprocal root (2 ulp), two products and the addition
    rel = (64 + 16) * plain.F32 / 2 + 10 * plain.F32
    plain.close(r_out, r, act, r.abs() * plain.F32)
    plain.close(y, ref, act, ref.abs() * rel)
    plain.check_quant(ref, q, s, rel)


@pytest.mark.gpu
def test_norm_outputs_are_optional_and_in_place(moe, dev):
    T, H, act = 17, 1032, "bf16"
    g = gen(5)
    x = torch.randn((T, H), generator=g).bfloat16().to(dev)
    res = torch.randn((T, H), generator=g).bfloat16().to(dev)
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)
    r0, y0, q0, s0 = norm_case(moe, dev, x.cpu(), res.cpu(), w.cpu(), act)
    y = torch.empty_like(x)
    rr = res.clone()
    moe.moe_add_rmsnorm_quant(x, rr, 0, w, 1e-6, T, H, rr, y)                      # residual in place, no codes
    assert torch.equal(rr, r0) and torch.equal(y, y0)
    xx, q, s = x.clone(), torch.empty_like(q0), torch.empty_like(s0)
    moe.moe_add_rmsnorm_quant(xx, res, 0, w, 1e-6, T, H, xx, None, q, s)           # x in place, codes only
    assert torch.equal(xx, r0) and torch.equal(q, q0) and torch.equal(s, s0)


@pytest.mark.gpu
def test_norm_keeps_rows_apart_and_carries_non_finite_values(moe, dev):
    T, H = 4, 384
    x = torch.randn((T, H), generator=gen(1)).bfloat16()
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(H).bfloat16()
    _, y, q, s = norm_case(moe, dev, x, None, w, "bf16")
    clean = x.clone()
    clean[1:3] = 1.0
    _, y0, q0, s0 = norm_case(moe, dev, clean, None, w, "bf16")
    for a, b in ((y, y0), (q, q0), (s, s0)):
        assert torch.equal(a[[0, 3]], b[[0, 3]])
    assert torch.isnan(y[1]).all() and torch.isnan(s[1]).all()
    assert torch.all((q[1].cpu() & 0x7F) == 0x7F)
    # an infinite mean square: 1 / sqrt of it is 0, and inf * 0 is NaN in the one place
    yf = y[2].float().cpu()
    assert torch.isnan(yf[200]) and torch.all(yf[torch.arange(H) != 200] == 0)
    assert torch.isnan(s[2, 1]) and torch.all(s[2, [0, 2]].cpu() == 2.0 ** -126)


# ---- SiLU-mul -----------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,I", [(1, 8), (1, 1408), (3, 128), (7, 136), (5, 120), (64, 2056), (1000, 72), (33, 14336)])
def test_silu_matches_the_formula(moe, dev, act, T, I):
    x = (3 * torch.randn((T, 2 * I), generator=gen(T + I))).to(plain.DT[act])
    if T > 2:
        x[1] = 0
        x[2, : I // 2] = -200.0   # exp overflows f32: the product is a zero
    q = torch.empty((T, I), dtype=torch.uint8, device=dev)
    s = torch.empty((T, -(-I // 128)), device=dev)
    moe.moe_silu_mul_quant(x.to(dev), moe.ACT_CODES[act], T, I, q, s)
    v = plain.silu_mul(x[:, :I].double(), x[:, I:].double())
    # the fast exponential's error grows with |g| (2 + 1.16 |g| ulp), and weighs exp(-g) / (1 + exp(-g));
    # the fast division is good to 2 ulp: 24 ulp beside the group's largest value covers |g| <= 16
    plain.check_quant(v, q, s, 24 * 2 * plain.F32)


# ---- E4M3 product with block scales ---------------------------------------------------

def gemm_inputs(M, N, K, act, addend, seed):
    g = gen(seed)
    kb = -(-K // 128)
    a = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
    w = torch.randint(0, 256, (N, K), generator=g, dtype=torch.uint8)
    a[(a & 0x7F) == 0x7F] = 0x3A   # no NaN
    w[(w & 0x7F) == 0x7F] = 0xB9
    sa = torch.rand((M, kb), generator=g) * 0.02 + 1e-4
    sb = (torch.rand((-(-N // 128), kb), generator=g) - 0.3) * 0.02
    add = (torch.randn((M, N), generator=g) * 30).to(plain.DT[act]) if addend else None
    return a, sa, w, sb, add


def gemm_ref(a, sa, w, sb, add):
    N, K = w.shape
    av = plain.e4m3(a) * sa.double().repeat_interleave(128, 1)[:, :K]
    wv = plain.e4m3(w) * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, mag = av @ wv.T, av.abs() @ wv.abs().T
    if add is not None:
        ref, mag = ref + add.double(), mag + add.double().abs()
    return ref, mag


GEMMS = [(1, 8, 16), (1, 2816, 2048), (3, 136, 400), (8, 4096, 1408), (9, 24, 128), (16, 264, 144), (17, 1000, 272),
         (31, 520, 1040), (32, 2048, 2048), (33, 128, 512), (64, 256, 256), (65, 200, 4112), (100, 2816, 528),
         (127, 128, 128), (128, 128, 128), (129, 384, 2048), (200, 8, 16), (256, 2056, 640), (333, 2816, 2048),
         (600, 1544, 400), (1, 28672, 256), (1500, 5000, 1408)]


@pytest.mark.gpu
@pytest.mark.parametrize("act,addend", [("bf16", False), ("f16", True)])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_matches_the_formula(moe, dev, act, addend, M, N, K):
    a, sa, w, sb, add = gemm_inputs(M, N, K, act, addend, M + 3 * N + K)
    ref, mag = gemm_ref(a, sa, w, sb, add)
    out = torch.full((M, N), float("nan"), dtype=plain.DT[act], device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_block_fp8_gemm(a.to(dev), sa.to(dev), w.to(dev), sb.to(dev), add.to(dev) if addend else None, out,
                           moe.ACT_CODES[act], M, N, K, err)
    assert int(err.item()) == 0
    plain.close(out, ref, act, mag * (K + K / 64 + 8) * plain.F32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["huge", "tiny", "subnormal", "far apart", "zero"])
@pytest.mark.parametrize("M,N,K", [(5, 520, 528), (13, 264, 400), (29, 264, 528), (40, 520, 2064), (260, 4104, 144),
                                   (260, 1032, 2064), (778, 8456, 400), (446, 9752, 400), (513, 7696, 624)])
def test_gemm_takes_any_scales(moe, dev, M, N, K, kind):
    """Products of two scales that overflow f32, or lose bits below its normal range, while the outputs do not; rows of
    ordinary scales beside them."""
    g = gen(M + K)
    kb, nb = -(-K // 128), -(-N // 128)
    a = torch.randint(0x60, 0x7F, (M, K), generator=g, dtype=torch.uint8)      # 32 to 448, all positive
    w = torch.randint(0x60, 0x7F, (N, K), generator=g, dtype=torch.uint8)
    sa, sb = 1 + torch.rand((M, kb), generator=g), 1 + torch.rand((nb, kb), generator=g)
    odd = torch.arange(M) % 3 != 1
    if kind == "huge":                     # products from 1e39; the codes are 0 or the two smallest
        a, w = (torch.randint(0, 3, t.shape, generator=g, dtype=torch.uint8) for t in (a, w))
        a[odd, 128:256] = 0                # whole blocks of zeros
        sa[odd] *= 1e29
        sb *= 1e10
    elif kind == "tiny":                   # products about 1e-44, seven times the smallest f32
        sa[odd] *= 1e-34
        sb *= 1e-10
    elif kind == "subnormal":              # one scale below the normal range, the other about 1
        sa[odd] *= 1e-43
    elif kind == "far apart":              # the product is ordinary, a sum times the larger scale is not
        sa[odd] *= 1e37
        sb *= 1e-30
    else:
        sa[odd] = 0
        sb[:, ::2] = 0
    ref, mag = gemm_ref(a, sa, w, sb, None)
    assert ref.abs().max() < 3e38
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    moe.moe_block_fp8_gemm(a.to(dev), sa.to(dev), w.to(dev), sb.to(dev), None, out, 0, M, N, K)
    # terms and sums below the normal range are rounded to multiples of 2^-149 (a K-th of it for each term)
    plain.close(out, ref, "bf16", mag * (K + K / 64 + 8) * plain.F32 + (K / 32 + 8) * 2.0 ** -149)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 2048, 1024), (40, 512, 1024), (300, 2048, 1024)])
def test_gemm_keeps_non_finite_rows_apart_and_repeats_bit_for_bit(moe, dev, M, N, K):
    a, sa, w, sb, add = gemm_inputs(M, N, K, "bf16", True, 7)
    a[1, 3] = 0x7F                     # NaN code in row 1
    w[N - 5, K - 1] = 0xFF             # NaN code in column N - 5
    sa[2, 1] = float("inf")
    a, sa, w, sb, add = (t.to(dev) for t in (a, sa, w, sb, add))
    outs = []
    for _ in range(2):
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        moe.moe_block_fp8_gemm(a, sa, w, sb, add, out, 0, M, N, K)
        outs.append(out)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    bad = ~torch.isfinite(outs[0])
    want = torch.zeros((M, N), dtype=torch.bool, device=dev)
    want[1] = want[2] = True
    want[:, N - 5] = True
    assert torch.equal(bad, want)
    moe.moe_block_fp8_gemm(a, sa, w, sb, add, add, 0, M, N, K)   # the addend may be the output
    assert torch.equal(add.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("act,addend", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("M,N,K", [(1, 9736, 1424), (8, 9736, 1424), (16, 8200, 1296), (24, 8200, 2000), (32, 8200, 2000),
                                   (24, 5800, 1296), (32, 5800, 1424)])
def test_gemm_of_few_rows_takes_several_tiles(moe, dev, M, N, K, act, addend):
    """Two 32-row tiles and a part of one to a CTA (152 SMs), every warp with blocks of each, a short last block."""
    a, sa, w, sb, add = gemm_inputs(M, N, K, act, addend, M + N)
    ref, mag = gemm_ref(a, sa, w, sb, add)
    out = torch.full((M, N), float("nan"), dtype=plain.DT[act], device=dev)
    moe.moe_block_fp8_gemm(a.to(dev), sa.to(dev), w.to(dev), sb.to(dev), add.to(dev) if addend else None, out,
                           moe.ACT_CODES[act], M, N, K)
    plain.close(out, ref, act, mag * (K + K / 64 + 8) * plain.F32)


# on 152 SMs: tiles of 128, 64, 128 and 64 columns by one CTA each, 128 and 64 by two CTAs, 128 and 64 by four, and 256
# columns, one and two tiles to a CTA
FORMS = [(2000, 4104, 400), (520, 4104, 144), (260, 4104, 144), (130, 264, 400), (520, 1032, 4112), (260, 1032, 2064),
         (260, 1032, 4112), (40, 520, 2064), (268, 6712, 2064), (778, 8456, 2064)]


@pytest.mark.gpu
@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_gemm_forms_for_many_rows(moe, dev, M, N, K, addend):
    a, sa, w, sb, add = gemm_inputs(M, N, K, "bf16", addend, M + N)
    ref, mag = gemm_ref(a, sa, w, sb, add)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev)
    moe.moe_block_fp8_gemm(a.to(dev), sa.to(dev), w.to(dev), sb.to(dev), add.to(dev) if addend else None, out, 0, M, N,
                           K)
    plain.close(out, ref, "bf16", mag * (K + K / 64 + 8) * plain.F32)


# on 152 SMs: several tiles of 128 columns to a CTA (twice), of 64 columns (twice)
SEVERAL = [(446, 9752, 400), (257, 12808, 224), (513, 7696, 624), (2487, 928, 224)]


@pytest.mark.gpu
@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("M,N,K", SEVERAL)
def test_gemm_of_several_narrow_tiles(moe, dev, M, N, K, addend):
    a, sa, w, sb, add = gemm_inputs(M, N, K, "f16", addend, M + N)
    ref, mag = gemm_ref(a, sa, w, sb, add)
    out = torch.full((M, N), float("nan"), dtype=torch.float16, device=dev)
    moe.moe_block_fp8_gemm(a.to(dev), sa.to(dev), w.to(dev), sb.to(dev), add.to(dev) if addend else None, out, 1, M, N,
                           K)
    plain.close(out, ref, "f16", mag * (K + K / 64 + 8) * plain.F32)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(40, 512, 8192), (2000, 4096, 1024), (300, 7168, 2048)])
def test_gemm_wait_that_runs_out_is_reported(moe, dev, M, N, K):
    """As in test_gpu_timeout.py: ordinary waits with a limit too short for them, by a cluster and by single CTAs."""
    a, sa, w, sb, _ = (t.to(dev) if t is not None else None for t in gemm_inputs(M, N, K, "bf16", False, 5))
    out, err = torch.empty((M, N), dtype=torch.bfloat16, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_block_fp8_gemm(a, sa, w, sb, None, out, 0, M, N, K, err)
    clean = out.clone()
    prev = moe.moe_set_wait_limit_ns(300)
    try:
        moe.moe_block_fp8_gemm(a, sa, w, sb, None, out, 0, M, N, K, err)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(prev)
    assert int(err.item()) == moe.MOE_DEV_ERR_TIMEOUT
    err.zero_()
    moe.moe_block_fp8_gemm(a, sa, w, sb, None, out, 0, M, N, K, err)
    assert int(err.item()) == 0 and torch.equal(out.view(torch.int16), clean.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [100, 600, 1500, 4000])
@pytest.mark.parametrize("M,N,K", [(2000, 4104, 400), (260, 4104, 144), (778, 8456, 2064), (520, 1032, 4112),
                                   (260, 1032, 2064), (260, 1032, 4112), (40, 520, 2064), (446, 9752, 400),
                                   (513, 7696, 624)])
def test_gemm_ends_whatever_wait_runs_out(moe, dev, M, N, K, limit_ns):
    """Every form, with limits that run out at its start, in its middle or not at all: the call ends, a result that
    is not the clean one is reported, and the next call at the default limit is the clean one."""
    a, sa, w, sb, add = (t.to(dev) for t in gemm_inputs(M, N, K, "bf16", True, 5))
    out, err = torch.empty((M, N), dtype=torch.bfloat16, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    moe.moe_block_fp8_gemm(a, sa, w, sb, add, out, 0, M, N, K, err)
    clean = out.clone()
    prev = moe.moe_set_wait_limit_ns(limit_ns)
    try:
        moe.moe_block_fp8_gemm(a, sa, w, sb, add, out, 0, M, N, K, err)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(prev)
    code = int(err.item())
    assert code in (0, moe.MOE_DEV_ERR_TIMEOUT)
    assert code or torch.equal(out.view(torch.int16), clean.view(torch.int16))
    err.zero_()
    moe.moe_block_fp8_gemm(a, sa, w, sb, add, out, 0, M, N, K, err)
    assert int(err.item()) == 0 and torch.equal(out.view(torch.int16), clean.view(torch.int16))


# ---- offsets past 32 bits --------------------------------------------------------------

@pytest.mark.gpu
def test_rows_past_32_bits_of_bytes(moe, dev):
    """The last rows of tensors of more than 2^31 elements equal the same rows run by themselves."""
    T, H = 140001, 16384
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    x[:3] = 0
    x[-3:] = torch.randn((3, H), device=dev)
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)

    def buffers(t, n):
        return torch.empty((t, n), dtype=torch.uint8, device=dev), torch.empty((t, -(-n // 128)), device=dev)
    r, y, (q, s) = torch.empty_like(x), torch.empty_like(x), buffers(T, H)
    moe.moe_add_rmsnorm_quant(x, None, 0, w, 1e-6, T, H, r, y, q, s)
    r1, y1, (q1, s1) = torch.empty_like(x[:3]), torch.empty_like(x[:3]), buffers(3, H)
    moe.moe_add_rmsnorm_quant(x[-3:].clone(), None, 0, w, 1e-6, 3, H, r1, y1, q1, s1)
    for big, one in ((r, r1), (y, y1), (q, q1), (s, s1)):
        assert torch.equal(big[-3:], one)
    del r, y, q, s
    I = H // 2
    q, s = buffers(T, I)
    q1, s1 = buffers(3, I)
    moe.moe_silu_mul_quant(x, 0, T, I, q, s)
    moe.moe_silu_mul_quant(x[-3:].clone(), 0, 3, I, q1, s1)
    assert torch.equal(q[-3:], q1) and torch.equal(s[-3:], s1)
    del x, q, s
    # an output of more than 2^31 elements, 128 rows of it taken by themselves too
    K = 256
    a, sa, w8, sb, _ = (t.to(dev) if t is not None else None for t in gemm_inputs(1, H, K, "bf16", False, 3))
    T = T // 128 * 128
    a = torch.randint(0, 0x70, (T, K), dtype=torch.uint8, device=dev)
    sa = torch.rand((T, 2), device=dev)
    out, part = torch.empty((T, H), dtype=torch.bfloat16, device=dev), torch.empty((128, H), dtype=torch.bfloat16, device=dev)
    moe.moe_block_fp8_gemm(a, sa, w8, sb, None, out, 0, T, H, K)
    moe.moe_block_fp8_gemm(a[-128:].clone(), sa[-128:].clone(), w8, sb, None, part, 0, 128, H, K)
    # the two may cut the contraction differently: four sums of 64 terms, any order
    err = (out[-128:].double() - part.double()).abs()
    mag = (e4m3_abs(a[-128:], sa[-128:])) @ (e4m3_abs(w8, sb.repeat_interleave(128, 0))).T
    assert torch.all(err <= mag * (2 * (K + 8) * plain.F32) + part.double().abs() * 2 * plain.U["bf16"])


def e4m3_abs(codes, scales):
    return (codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)).abs()


@pytest.mark.gpu
def test_few_tokens_of_experts_past_32_bits_of_bytes(moe, dev):
    from mixture_experts_grouped_gb300 import ffn
    from mixture_experts_grouped_gb300 import layer as L
    T, H, I, E = 2, 2048, 2048, 256
    gu = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=dev)   # 4.3 GB
    down = torch.empty((E, H, I), dtype=torch.bfloat16, device=dev)
    g = gen(1)
    ge, de = weight("bf16", 1, 2 * I, H, 2, g)["w"], weight("bf16", 1, H, I, 1, g)["w"]
    gu[E - 1], down[E - 1] = ge[0].to(dev), de[0].to(dev)
    layer = ffn.FewTokensLayer(T, H, I, E, 1, "bf16",
                               L.DeviceWeight(moe.MoeWeight(0, 0, gu.data_ptr(), None, None, None), [gu]),
                               L.DeviceWeight(moe.MoeWeight(0, 0, down.data_ptr(), None, None, None), [down]), dev)
    layer.topk_ids.fill_(E - 1)
    layer.topk_weights.fill_(0.75)
    x = torch.randn((T, H), generator=g).bfloat16()
    out = layer.forward(x.to(dev))
    ids, w = torch.zeros((T, 1)).int(), torch.full((T, 1), 0.75)
    ref, slack = plain.few_tokens(x, ids, w, {"w": ge}, {"w": de}, "bf16", "bf16", I, 1)
    plain.close(out, ref, "bf16", slack)


# ---- the layer for a few tokens -------------------------------------------------------

def weight(fmt, e, n, k, groups2, g, group=128):
    if fmt == "bf16":
        return {"w": (torch.randn((e, n, k), generator=g) * 0.05).bfloat16()}
    if fmt == "fp8":
        w = torch.randint(0, 256, (e, n, k), generator=g, dtype=torch.uint8)
        w[(w & 0x7F) == 0x7F] = 0x3A
        return {"w": w, "scales": torch.rand((e, n), generator=g) * 4e-4 + 1e-4}
    if fmt == "nvfp4":
        return {"w": torch.randint(0, 256, (e, n, k // 2), generator=g, dtype=torch.uint8),
                "scales": torch.randint(0x20, 0x48, (e, k // 16, n), generator=g, dtype=torch.uint8),
                "scale2": torch.rand((groups2, e), generator=g) * 0.02 + 0.01}
    lim = 2 ** 31
    return {"w": torch.randint(-lim, lim, (e, k // 8, n), generator=g).int(),
            "scales": (torch.rand((e, k // group, n), generator=g) * 0.01 + 0.002).half(),
            "zeros": torch.randint(-lim, lim, (e, k // group, n // 8), generator=g).int()}


def device_weight(moe, w, fmt, dev, group=128):
    from mixture_experts_grouped_gb300 import layer as L
    d = {n: t.to(dev) for n, t in w.items()}

    def at(n):
        return d[n].data_ptr() if n in d else None
    return L.DeviceWeight(moe.MoeWeight(moe.WFMT_CODES[fmt], group if fmt == "gptq" else 0, at("w"), at("scales"),
                                        at("zeros"), at("scale2")), list(d.values()))


def few_layer(moe, dev, fmt, act, T, H, I, E, k, seed, renorm=True, group=128, change=None):
    from mixture_experts_grouped_gb300 import ffn
    g = gen(seed)
    gu, down = weight(fmt, E, 2 * I, H, 2, g, group), weight(fmt, E, H, I, 1, g, group)
    if change:
        change(gu, down)
    x = torch.randn((T, H), generator=g).to(plain.DT[act])
    logits = torch.randn((T, E), generator=g)
    layer = ffn.FewTokensLayer(T, H, I, E, k, act, device_weight(moe, gu, fmt, dev, group),
                               device_weight(moe, down, fmt, dev, group), dev, renorm)
    layer.out.fill_(float("nan"))
    return layer, x, logits, gu, down


SHAPES = [(1, 2048, 768, 16, 8), (1, 128, 128, 1, 1), (2, 256, 128, 4, 2), (5, 512, 384, 12, 5), (8, 1024, 128, 8, 2),
          (9, 256, 256, 256, 16), (16, 128, 640, 3, 3), (17, 384, 128, 7, 1), (32, 256, 256, 64, 6), (31, 128, 128, 2, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act", [("bf16", "bf16")] + [(f, a) for f in FMTS[1:] for a in ("bf16", "f16")])
@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
def test_few_tokens_matches_the_formula(moe, dev, fmt, act, T, H, I, E, k):
    renorm = (T + E) % 3 != 0
    layer, x, logits, gu, down = few_layer(moe, dev, fmt, act, T, H, I, E, k, T + H + I + E, renorm)
    out = layer.forward(x.to(dev), logits.to(dev))
    ids, w = torch.empty_like(layer.topk_ids), torch.empty_like(layer.topk_weights)
    moe.moe_route_topk_softmax(logits.to(dev), ids, w, T, E, k, renorm)
    assert torch.equal(layer.topk_ids, ids) and torch.equal(layer.topk_weights, w)
    assert int(layer.err.item()) == 0
    ref, slack = plain.few_tokens(x, ids.cpu(), w.cpu(), gu, down, fmt, act, I, E)
    plain.close(out, ref, act, slack)
    first = out.clone()
    layer.forward(x.to(dev), logits.to(dev))
    assert torch.equal(first.view(torch.int16), layer.out.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act,T,H,I,E,k,group", [
    ("bf16", "bf16", 3, 8, 8, 4, 2, 0), ("bf16", "bf16", 12, 136, 72, 5, 2, 0), ("bf16", "bf16", 2, 2056, 40, 3, 2, 0),
    ("fp8", "f16", 6, 144, 80, 5, 2, 0), ("nvfp4", "bf16", 4, 160, 96, 5, 3, 0), ("gptq", "f16", 4, 192, 64, 5, 3, 64),
    ("gptq", "bf16", 20, 320, 192, 6, 2, 64), ("gptq", "f16", 3, 256, 256, 4, 2, 256)])
def test_few_tokens_at_odd_sizes(moe, dev, fmt, act, T, H, I, E, k, group):
    layer, x, logits, gu, down = few_layer(moe, dev, fmt, act, T, H, I, E, k, H + I, group=group)
    out = layer.forward(x.to(dev), logits.to(dev))
    ref, slack = plain.few_tokens(x, layer.topk_ids.cpu(), layer.topk_weights.cpu(), gu, down, fmt, act, I, E)
    plain.close(out, ref, act, slack)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("gptq", "f16"), ("nvfp4", "bf16")])
def test_few_tokens_takes_given_routing(moe, dev, fmt, act):
    """Every token to one expert; bad ids dropped and flagged; an expert named twice; no pair left at all."""
    T, H, I, E, k = 32, 256, 128, 6, 3
    layer, x, _, gu, down = few_layer(moe, dev, fmt, act, T, H, I, E, k, 3)
    g = gen(9)
    w = torch.rand((T, k), generator=g)
    for kind in ("one", "bad", "twice", "none"):
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
        if kind == "one":
            ids[:, 0] = 4
            ids[:, 1:] = -1
        if kind == "bad":
            ids[3, 1], ids[7, 0], ids[31, 2] = -1, E, 2 ** 31 - 1
        if kind == "twice":
            ids[:, 1] = ids[:, 0]
            ids[5] = 2
        if kind == "none":
            ids[:] = E
        layer.err.zero_()
        layer.out.fill_(float("nan"))
        layer.topk_ids.copy_(ids)
        layer.topk_weights.copy_(w)
        out = layer.forward(x.to(dev))
        want = moe.MOE_DEV_ERR_EXPERT_ID if kind in ("one", "bad", "none") else 0
        assert int(layer.err.item()) == want, kind
        ref, slack = plain.few_tokens(x, ids, w, gu, down, fmt, act, I, E)
        plain.close(out, ref, act, slack + slack * 2.0 ** -20)
        assert torch.equal(layer.topk_ids.cpu(), ids)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_few_tokens_keeps_non_finite_experts_and_tokens_apart(moe, dev, fmt):
    T, H, I, E, k = 7, 256, 128, 5, 2
    bad = {"bf16": float("inf"), "fp8": 0x7F}[fmt]

    def spoil(gu, down):
        gu["w"][1, 5, 7] = bad
        down["w"][3, 2, 9] = bad
    layer, x, logits, gu, down = few_layer(moe, dev, fmt, "bf16", T, H, I, E, k, 11, change=spoil)
    x[0, 3] = float("nan")
    out = layer.forward(x.to(dev), logits.to(dev)).float().cpu()
    ids = layer.topk_ids.cpu()
    for t in range(1, T):
        hit = set(ids[t].tolist())
        fin = torch.isfinite(out[t])
        if 1 not in hit and 3 not in hit:
            assert fin.all(), t
        elif 1 not in hit:
            assert not fin[2] and fin[torch.arange(H) != 2].all(), t
    assert torch.isnan(out[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 12, 3), (32, 128, 8), (20, 200, 16), (9, 256, 4), (8, 5, 5)])
def test_few_tokens_routes_like_the_routing_call(moe, dev, T, E, k):
    """Ties, infinities, signed zeros and NaN among the logits; every softmax form."""
    layer, x, _, _, _ = few_layer(moe, dev, "bf16", "bf16", T, 8, 8, E, k, 1, renorm=T % 2 == 0)
    g = gen(T)
    logits = torch.randint(-3, 4, (T, E), generator=g).float()
    logits[0, ::3] = -0.0
    if T > 5:
        logits[1, 1] = float("inf")
        logits[2] = float("-inf")
        logits[3, E // 2] = float("nan")
        logits[4] = float("nan")
        logits[5] = 0.0
    logits = logits.to(dev)
    layer.forward(x.to(dev), logits)
    ids, w = torch.empty_like(layer.topk_ids), torch.empty_like(layer.topk_weights)
    moe.moe_route_topk_softmax(logits, ids, w, T, E, k, layer.renormalize)
    assert torch.equal(layer.topk_ids, ids)
    assert torch.equal(layer.topk_weights.view(torch.int32), w.view(torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act", [("gptq", "f16"), ("nvfp4", "bf16"), ("fp8", "f16")])
def test_few_tokens_of_many_rows(moe, dev, fmt, act):
    """Enough rows that a CTA's share is whole items: 64 experts of 1408 against 152 CTAs."""
    T, H, I, E, k = 16, 256, 1408, 64, 6
    layer, x, logits, gu, down = few_layer(moe, dev, fmt, act, T, H, I, E, k, 21)
    out = layer.forward(x.to(dev), logits.to(dev))
    ref, slack = plain.few_tokens(x, layer.topk_ids.cpu(), layer.topk_weights.cpu(), gu, down, fmt, act, I, E)
    plain.close(out, ref, act, slack)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("fp8", "bf16"), ("nvfp4", "f16"), ("gptq", "f16")])
def test_few_tokens_of_one_expert_among_many(moe, dev, fmt, act):
    """All 32 tokens to one expert of 128 (few tokens an expert by the batch's size, so it is listed four times), and
    the second choice to one of three others."""
    T, H, I, E, k = 32, 128, 128, 128, 2
    layer, x, _, gu, down = few_layer(moe, dev, fmt, act, T, H, I, E, k, 22)
    g = gen(23)
    ids = torch.stack((torch.full((T,), 77), torch.tensor([3, 76, 127])[torch.randint(0, 3, (T,), generator=g)]), 1).int()
    w = torch.rand((T, k), generator=g)
    layer.topk_ids.copy_(ids)
    layer.topk_weights.copy_(w)
    out = layer.forward(x.to(dev))
    assert int(layer.err.item()) == 0
    ref, slack = plain.few_tokens(x, ids, w, gu, down, fmt, act, I, E)
    plain.close(out, ref, act, slack)


@pytest.mark.gpu
def test_few_tokens_on_a_stream_and_in_a_graph(moe, dev):
    layer, x, logits, gu, down = few_layer(moe, dev, "bf16", "bf16", 4, 512, 256, 16, 4, 2)
    xs, ls = x.to(dev), logits.to(dev)
    want = layer.forward(xs, ls).clone()
    side = torch.cuda.Stream()
    layer.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    layer.forward(xs, ls, side)
    side.synchronize()
    assert torch.equal(layer.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(xs, ls)
    for _ in range(3):
        layer.out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 32, 33, 80])
def test_feed_forward_block(moe, dev, T):
    """Norm, router, routed experts (either path) and shared expert, run as one block."""
    from mixture_experts_grouped_gb300 import ffn
    H, I, E, k, act = 256, 128, 8, 2, "bf16"
    g = gen(T)
    gu, down = weight("bf16", E, 2 * I, H, 2, g), weight("bf16", E, H, I, 1, g)
    _, _, w1, s1, _ = gemm_inputs(1, 2 * I, H, act, False, 1)
    _, _, w2, s2, _ = gemm_inputs(1, H, I, act, False, 2)
    s1, s2 = s1 * 0.05, s2 * 0.05
    nw = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16()
    wr = torch.randn((H, E), generator=g) * 0.1
    x, res = torch.randn((T, H), generator=g).bfloat16(), torch.randn((T, H), generator=g).bfloat16()
    shared = ffn.SharedExpert(T, H, I, act, ffn.BlockFp8Weight(w1.to(dev), s1.to(dev)),
                              ffn.BlockFp8Weight(w2.to(dev), s2.to(dev)), dev)
    block = ffn.FeedForward(T, H, I, E, k, act, nw.to(dev), wr.to(dev), device_weight(moe, gu, "bf16", dev),
                            device_weight(moe, down, "bf16", dev), shared, device=dev)
    out, r = block.forward(x.to(dev), res.to(dev))
    # each step against the plain form of its own input, the routing as the library took it
    rr = x.double() + res.double()
    assert torch.equal(r.cpu(), rr.bfloat16())
    y, ids, wts = block.y.cpu(), block.experts.topk_ids.cpu(), block.experts.topk_weights.cpu()
    routed, slack = plain.few_tokens(y, ids, wts, gu, down, "bf16", act, I, E)
    # the grouped path also rounds its down products
    slack = slack + routed.abs() * 2.0 ** -8 + 2.0 ** -8 * slack
    if T > 32:
        mag = torch.zeros_like(routed)
        for e in range(E):
            tok, slot = torch.nonzero(ids == e, as_tuple=True)
            yy, _ = plain.few_tokens(y[tok], torch.zeros((len(tok), 1)).int() + e, torch.ones((len(tok), 1)), gu, down,
                                     "bf16", act, I, E)
            mag.index_add_(0, tok, yy.abs() * wts[tok, slot].double()[:, None])
        slack = slack + mag * 2.0 ** -8
    plain.close(block.experts.out, routed, act, slack)
    xq = (block.q.cpu(), block.q_scales.cpu())
    ref1, mag1 = gemm_ref(*xq, w1, s1, None)
    plain.close(shared.gate_up, ref1, act, mag1 * (H + 16) * plain.F32)
    gate_up = shared.gate_up.cpu().double()
    plain.check_quant(plain.silu_mul(gate_up[:, :I], gate_up[:, I:]), shared.q, shared.q_scales, 48 * plain.F32)
    ref2, mag2 = gemm_ref(shared.q.cpu(), shared.q_scales.cpu(), w2, s2, block.experts.out.cpu())
    plain.close(out, ref2, act, mag2 * (I + 16) * plain.F32)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("fu,fd", [("fp8", "bf16"), ("bf16", "fp8"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("gptq", "gptq")])
def test_feed_forward_takes_every_format_at_any_batch(moe, dev, fu, fd, T):
    """The grouped path takes gate/up and down weights of different formats, the few-token call does not: such a layer
    runs at every T."""
    from mixture_experts_grouped_gb300 import ffn
    H, I, E, k = 256, 128, 8, 2
    g = gen(T)
    gu, down = weight(fu, E, 2 * I, H, 2, g), weight(fd, E, H, I, 1, g)
    nw, wr = torch.ones(H).bfloat16(), torch.randn((H, E), generator=g) * 0.1
    block = ffn.FeedForward(T, H, I, E, k, "bf16", nw.to(dev), wr.to(dev), device_weight(moe, gu, fu, dev),
                            device_weight(moe, down, fd, dev), device=dev)
    x = torch.randn((T, H), generator=g).bfloat16()
    out, r = block.forward(x.to(dev))
    assert torch.equal(r.cpu(), x)
    ids, wts = block.experts.topk_ids.cpu(), block.experts.topk_weights.cpu()
    ref, slack, mag = torch.zeros((T, H)).double(), torch.zeros((T, H)).double(), torch.zeros((T, H)).double()
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        wg, wd = plain.dequant(gu, fu, e), plain.dequant(down, fd, e)
        # the plain form of one format, on the dequantised (f64) weights
        yy, ss = plain.few_tokens(block.y.cpu()[tok], torch.zeros((len(tok), 1)).int(), torch.ones((len(tok), 1)),
                                  {"w": wg[None]}, {"w": wd[None]}, "bf16", "bf16", I, 1)
        w = wts[tok, slot].double()[:, None]
        ref.index_add_(0, tok, yy * w)
        slack.index_add_(0, tok, ss * w)
        mag.index_add_(0, tok, yy.abs() * w)
    # the down products are rounded to bf16 too
    plain.close(out, ref, "bf16", slack * (1 + 2.0 ** -8) + mag * 2.0 ** -8)


# ---- refusals (no GPU) -------------------------------------------------------------------

def few_args(m, **kw):
    w = m.MoeWeight(0, 0, 16, None, None, None)
    a = dict(x=16, act=0, logits=16, ids=16, wts=16, gu=w, down=w, T=4, k=2, H=128, I=64, E=8, renorm=True, out=16,
             err=0, ws=16, wsb=1 << 20, stream=0)
    a.update(kw)
    return m.moe_few_tokens(*a.values())


@pytest.mark.parametrize("call", [
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 2, 16, 1e-6, 4, 128, 16, 16, 16, 16, 0),    # act
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, -1, 128, 16, 16, 16, 16, 0),   # T
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, 4, 100, 16, 16, 16, 16, 0),    # H % 8
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, 4, 0, 16, 16, 16, 16, 0),      # H
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, -1.0, 4, 128, 16, 16, 16, 16, 0),    # eps
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, math.nan, 4, 128, 16, 16, 16, 16, 0),
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, 4, 128, 16, None, None, None, 0),  # no output
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, 4, 128, 16, 16, 16, None, 0),  # codes without scales
    lambda m: m.moe_add_rmsnorm_quant(None, 16, 0, 16, 1e-6, 4, 128, 16, 16, 16, 16, 0),
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, None, 1e-6, 4, 128, 16, 16, 16, 16, 0),
    lambda m: m.moe_add_rmsnorm_quant(16, 24, 0, 16, 1e-6, 4, 128, 16, 16, 16, 16, 0),    # alignment
    lambda m: m.moe_silu_mul_quant(16, 3, 4, 128, 16, 16, 0),
    lambda m: m.moe_silu_mul_quant(16, 0, -4, 128, 16, 16, 0),
    lambda m: m.moe_silu_mul_quant(16, 0, 4, 100, 16, 16, 0),
    lambda m: m.moe_silu_mul_quant(16, 0, 4, 128, None, 16, 0),
    lambda m: m.moe_silu_mul_quant(24, 0, 4, 128, 16, 16, 0),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 2, 4, 128, 128, 0, 0),       # act
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, -1, 128, 128, 0, 0),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, 4, 100, 128, 0, 0),       # N % 8
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, 4, 128, 24, 0, 0),        # K % 16
    lambda m: m.moe_block_fp8_gemm(16, None, 16, 16, None, 16, 0, 4, 128, 128, 0, 0),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, 24, 16, 0, 4, 128, 128, 0, 0),         # alignment
    lambda m: m.moe_block_fp8_gemm(16, 18, 16, 16, None, 16, 0, 4, 128, 128, 0, 0),
    lambda m: few_args(m, act=2),
    lambda m: few_args(m, T=-1),
    lambda m: few_args(m, E=300),
    lambda m: few_args(m, k=9),
    lambda m: few_args(m, H=100),
    lambda m: few_args(m, I=60),
    lambda m: few_args(m, act=1),                                                          # bf16 weights, f16 act
    lambda m: few_args(m, gu=m.MoeWeight(0, 0, None, None, None, None)),
    lambda m: few_args(m, gu=m.MoeWeight(0, 0, 24, None, None, None)),
    lambda m: few_args(m, gu=m.MoeWeight(9, 0, 16, None, None, None)),
    lambda m: few_args(m, gu=m.MoeWeight(3, 0, 16, 16, None, None)),                       # two formats
    lambda m: few_args(m, gu=m.MoeWeight(1, 96, 16, 16, 16, None), down=m.MoeWeight(1, 64, 16, 16, 16, None)),
    lambda m: few_args(m, gu=m.MoeWeight(2, 0, 16, 16, None, None), down=m.MoeWeight(2, 0, 16, 16, None, 16)),
    lambda m: few_args(m, x=None),
    lambda m: few_args(m, ids=None),
    lambda m: few_args(m, x=24),
    lambda m: few_args(m, ws=None),
    lambda m: few_args(m, wsb=100),
])
def test_misuse_is_refused_before_any_launch(moe, call):
    n0 = moe.moe_launch_count()
    with pytest.raises(moe.MoeError) as ei:
        call(moe)
    assert ei.value.status == moe.MOE_ERR_INVALID and ei.value.message
    assert moe.moe_launch_count() == n0


@pytest.mark.parametrize("call", [
    lambda m: m.moe_add_rmsnorm_quant(16, 16, 0, 16, 1e-6, 4, 32776, 16, 16, 16, 16, 0),
    lambda m: few_args(m, T=33),
    lambda m: few_args(m, H=32768, I=16384),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, 4, 128, 2 ** 27 + 16, 0, 0),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, 4, 2 ** 30 + 8, 128, 0, 0),
    lambda m: m.moe_block_fp8_gemm(16, 16, 16, 16, None, 16, 0, 2 ** 31 - 1, 128, 128, 0, 0),
])
def test_what_is_beyond_the_limits_is_unsupported(moe, call):
    with pytest.raises(moe.MoeError) as ei:
        call(moe)
    assert ei.value.status == moe.MOE_ERR_UNSUPPORTED and ei.value.message


def test_rows_of_the_touched_experts_past_32_bits_are_unsupported(moe):
    """The kernels count the rows of the experts that a batch may touch (one that more than 8 tokens share counts
    again) in 32 bits."""
    nv, bf = moe.MoeWeight(2, 0, 16, 16, None, 16), moe.MoeWeight(0, 0, 16, None, None, None)
    wide = [dict(gu=nv, down=nv, T=32, k=16, E=256, H=32, I=2 ** 23), dict(gu=bf, down=bf, T=3, k=16, E=64, H=8, I=2 ** 26 - 8),
            dict(gu=nv, down=nv, T=32, k=16, E=256, H=32, I=6710912)]
    for kw in wide:
        with pytest.raises(moe.MoeError) as ei:
            few_args(moe, **kw, wsb=100)
        assert ei.value.status == moe.MOE_ERR_UNSUPPORTED and "rows" in ei.value.message
    # (256 + 64) x 6710880 is below 2^31: the next check is what refuses it
    with pytest.raises(moe.MoeError) as ei:
        few_args(moe, gu=nv, down=nv, T=32, k=16, E=256, H=32, I=6710880, wsb=100)
    assert ei.value.status == moe.MOE_ERR_INVALID and "workspace" in ei.value.message


def shared_expert(T, H, I, act="bf16", **kw):
    from mixture_experts_grouped_gb300 import ffn

    def w8(n, k):
        return ffn.BlockFp8Weight(torch.zeros((n, k), dtype=torch.uint8), torch.zeros((-(-n // 128), -(-k // 128))))
    return ffn.SharedExpert(T, H, I, act, kw.get("gu", w8(2 * I, H)), kw.get("down", w8(H, I)), "cpu"), w8


def test_blocks_of_unlike_shapes_are_refused(moe):
    """A shared expert of another T, H or type would read or write past the block's buffers."""
    from mixture_experts_grouped_gb300 import ffn
    from mixture_experts_grouped_gb300 import layer as L
    T, H, I, E, k = 4, 256, 128, 8, 2
    w = L.DeviceWeight(moe.MoeWeight(0, 0, 16, None, None, None), [])

    def block(shared, norm_weight=torch.zeros(H).bfloat16(), w_router=torch.zeros((H, E))):
        return ffn.FeedForward(T, H, I, E, k, "bf16", norm_weight, w_router, w, w, shared, device="cpu")
    good, w8 = shared_expert(T, H, 512)
    assert block(good).shared is good and block(None).shared is None
    for other in (shared_expert(T + 1, H, 512)[0], shared_expert(T, H + 128, 512)[0], shared_expert(T, H, 512, "f16")[0]):
        with pytest.raises(ValueError, match="shared expert"):
            block(other)
    with pytest.raises(ValueError, match="norm_weight"):
        block(good, norm_weight=torch.zeros(H - 8).bfloat16())
    with pytest.raises(ValueError, match="w_router"):
        block(good, w_router=torch.zeros((E, H)))
    for kw in (dict(gu=w8(1016, H)), dict(gu=w8(1024, H - 16)), dict(down=w8(H, 1024)), dict(down=w8(H + 8, 512)),
               dict(gu=ffn.BlockFp8Weight(w8(1024, H).codes, torch.zeros((8, 1))))):
        with pytest.raises(ValueError, match="weight"):
            shared_expert(T, H, 512, **kw)


@pytest.mark.parametrize("fmt,T,H,I,E,k,few", [
    (0, 1, 4096, 14336, 8, 2, True), (0, 2, 4096, 14336, 8, 2, False), (0, 32, 4096, 14336, 8, 2, False),
    (0, 24, 4096, 2048, 16, 4, False), (0, 24, 2048, 768, 32, 8, True), (0, 32, 2048, 768, 32, 8, False),
    (0, 16, 2048, 768, 128, 8, True), (0, 32, 1024, 512, 8, 2, True), (3, 16, 4096, 14336, 8, 2, True),
    (3, 32, 4096, 14336, 8, 2, False), (3, 32, 4096, 2048, 16, 4, True), (2, 32, 4096, 14336, 8, 2, True),
    (1, 16, 4096, 14336, 8, 2, True), (1, 32, 4096, 14336, 8, 2, False), (1, 32, 4096, 2048, 16, 4, False),
    (1, 32, 2048, 1408, 64, 6, True), (1, 32, 512, 512, 16, 2, True), (0, 33, 512, 512, 16, 2, False)])
def test_feed_forward_takes_the_faster_path(moe, fmt, T, H, I, E, k, few):
    """The path that measured faster (or as fast, within a few percent) on these layers."""
    from mixture_experts_grouped_gb300 import ffn
    from mixture_experts_grouped_gb300 import layer as L
    w = L.DeviceWeight(moe.MoeWeight(fmt, 128, 16, 16, 16, 16), [])
    block = ffn.FeedForward(T, H, I, E, k, "bf16", torch.zeros(H), torch.zeros((H, E)), w, w, device="cpu")
    assert isinstance(block.experts, ffn.FewTokensLayer) == few
    assert isinstance(block.experts, L.MoeLayer) != few


def test_no_rows_is_a_no_op(moe):
    n0 = moe.moe_launch_count()
    moe.moe_add_rmsnorm_quant(None, None, 0, None, 1e-6, 0, 128, None, 16, None, None, 0)
    moe.moe_silu_mul_quant(None, 0, 0, 128, None, None, 0)
    moe.moe_block_fp8_gemm(None, None, None, None, None, None, 0, 0, 128, 128, 0, 0)
    few_args(moe, T=0, x=None, out=None, ws=None, wsb=0)
    assert moe.moe_launch_count() == n0 and moe.moe_few_tokens_workspace_size(4, 2, 64) == 1024
