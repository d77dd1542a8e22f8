"""The training operators at the edges of what they take: infinities, tails, long sums, outputs in place of inputs,
tensors of other devices, and an object's own buffers as its inputs."""
import math
from types import SimpleNamespace

import pytest
import torch

import plain
from test_training_ops import FNS, dev, f64, moe, offsets_of  # noqa: F401

F32 = plain.F32


# ---- infinities ------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("fn", FNS[1:])
def test_slopes_of_infinite_values_are_their_limits(moe, dev, fn, act):
    """0 at -inf and 1 at +inf, in every column of a vector, and in the bias' sums."""
    z = torch.tensor([-math.inf, math.inf] * 8, dtype=plain.DT[act], device=dev).repeat(40, 1)
    d = torch.full_like(z, 0.75)
    dz, db = torch.empty_like(z), torch.empty(16, device=dev)
    moe.moe_bias_act_backward(d, z, moe.ACT_CODES[act], moe.FN_CODES[fn], 40, 16, dz, db)
    assert torch.all(dz[:, ::2] == 0) and torch.all(dz[:, 1::2] == 0.75)
    assert torch.all(db[::2] == 0) and torch.all(db[1::2] == 30.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", FNS[1:])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_gradient_through_a_pre_that_overflows_f16(moe, dev, fn, M):
    """z = +-76800 is finite in f32, where its function is taken, and infinite in the f16 that the gradient reads."""
    N, K = 72, 64
    a, w = torch.zeros((M, K), dtype=torch.float16), torch.zeros((N, K), dtype=torch.float16)
    a[:, 0], w[:, 0] = 256.0, 1.0
    w[3, 0], w[5, 0] = -300.0, 300.0
    out, pre = (torch.empty((M, N), dtype=torch.float16, device=dev) for _ in range(2))
    code = moe.FN_CODES[fn]
    moe.moe_dense_gemm(a.to(dev), 1, w.to(dev), None, code, None, pre, out, M, N, K)
    assert torch.all(pre[:, 3] == -math.inf) and torch.all(pre[:, 5] == math.inf)
    assert torch.all(out[:, 3] == 0) and torch.all(out[:, 5] == math.inf)
    d = torch.full((M, N), 0.5, dtype=torch.float16, device=dev)
    dz, db = torch.empty_like(d), torch.empty(N, device=dev)
    moe.moe_bias_act_backward(d, pre, 1, code, M, N, dz, db)
    want = torch.full((M, N), 0.5, dtype=torch.float16, device=dev)  # slopes at 256 are 1
    want[:, 3] = 0
    assert torch.equal(dz, want) and torch.equal(db, want.float().sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_swiglu_of_infinite_gates_is_its_limit(moe, dev, act):
    """A gate that overflowed to -inf gives 0 and has no gradient, one of +inf has the slope 1; a NaN stays."""
    rows, I, dt = 3, 24, plain.DT[act]
    g = torch.tensor([-math.inf, math.inf, math.nan, 1.0], dtype=dt, device=dev).repeat(rows, I // 4)
    u, dh = torch.full((rows, I), 2.0, dtype=dt, device=dev), torch.full((rows, I), 0.5, dtype=dt, device=dev)
    gu = torch.cat((g, u), 1).contiguous()
    h, h2, dgu = torch.empty_like(u), torch.empty_like(u), torch.empty_like(gu)
    moe.moe_swiglu(gu, moe.ACT_CODES[act], rows, I, h)
    moe.moe_swiglu_backward(gu, dh, moe.ACT_CODES[act], rows, I, dgu, h2)
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    dg, du = dgu[:, :I], dgu[:, I:]
    assert torch.all(h[:, ::4] == 0) and torch.all(h[:, 1::4] == math.inf) and torch.isnan(h[:, 2::4]).all()
    assert torch.all(dg[:, ::4] == 0) and torch.all(dg[:, 1::4] == 1.0) and torch.isnan(dg[:, 2::4]).all()
    assert torch.all(du[:, ::4] == 0) and torch.all(du[:, 1::4] == math.inf) and torch.isnan(du[:, 2::4]).all()


# ---- outputs in place of inputs ---------------------------------------------------------------------

# one row, the narrow form with one and several batches of rows a thread, the wide form (whose columns fill the GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("M,N", [(1, 8), (33, 200), (5000, 72), (1333, 264), (300, 9736), (1100, 16384)])
def test_bias_and_activation_gradient_in_place(moe, dev, M, N, fn, act):
    """d_pre in the place of d_out, and in that of pre, has the bits that it has in a tensor of its own, and so has
    d_bias; without d_pre too."""
    g = torch.Generator(device=dev).manual_seed(M)
    d, z = (torch.randn((M, N), generator=g, device=dev).to(plain.DT[act]) for _ in range(2))
    codes = moe.ACT_CODES[act], moe.FN_CODES[fn]
    dz, db = torch.empty_like(d), torch.empty(N, device=dev)
    moe.moe_bias_act_backward(d, z, *codes, M, N, dz, db)
    ref = d.double() * f64(fn, z.double())[1]
    assert torch.all((dz.double() - ref).abs()
                     <= ref.abs() * plain.U[act] + d.double().abs() * 64 * F32 + plain.TINY[act])
    for place in ("d_out", "pre", "none"):
        di, zi, db2 = d.clone(), z.clone(), torch.empty(N, device=dev)
        into = {"d_out": di, "pre": zi, "none": None}[place]
        moe.moe_bias_act_backward(di, zi, *codes, M, N, into, db2)
        assert torch.equal(db2, db), place
        assert into is None or torch.equal(into, dz), place
        assert place == "d_out" or torch.equal(di, d)
        assert place == "pre" or torch.equal(zi, z)


# ---- the tail of gelu -------------------------------------------------------------------------------

def gelu_part(z):
    """The part of itself by which the normal distribution of z may be off: 9e-7 of its polynomial; 24 half steps of
    its evaluation, and of the hardware's 2^x and reciprocal; and the roundings of the exponent z^2 / 2, of two half
    steps of itself at most."""
    return 9e-7 + (24 + z * z) * F32


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_gelu_keeps_its_relative_accuracy_in_the_tail(moe, dev, act):
    """To where the density leaves f32's normal range (-13): a half step of the type beside gelu_part, value and slope."""
    z = torch.cat([torch.linspace(-13, 0, 3001), torch.linspace(0, 9, 1001), -torch.logspace(-6, 0, 1002)])
    z = z.to(plain.DT[act])[: 5000]
    n = len(z)
    a = torch.zeros((1, 8), dtype=z.dtype)
    a[0, 0] = 1
    w = torch.zeros((n, 8), dtype=z.dtype)
    w[:, 0] = z
    out = torch.empty((1, n), dtype=z.dtype, device=dev)
    moe.moe_dense_gemm(a.to(dev), moe.ACT_CODES[act], w.to(dev), None, moe.MOE_FN_GELU, None, None, out, 1, n, 8)
    z = z.double()
    cdf, density = torch.exp(torch.special.log_ndtr(z)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    part = gelu_part(z)
    plain.close(out[0], z * cdf, act, z.abs() * cdf * part)
    one = torch.ones((1, n), dtype=plain.DT[act], device=dev)
    moe.moe_bias_act_backward(one, z[None].to(plain.DT[act]).to(dev), moe.ACT_CODES[act], moe.MOE_FN_GELU, 1, n, out)
    plain.close(out[0], cdf + z * density, act, (cdf + z.abs() * density) * part)
    # and in f32, as the bias' gradient: one row, each column its own sum
    db = torch.empty(n, device=dev)
    moe.moe_bias_act_backward(one, z[None].to(plain.DT[act]).to(dev), moe.ACT_CODES[act], moe.MOE_FN_GELU, 1, n, None, db)
    assert torch.all((db.cpu().double() - (cdf + z * density)).abs() <= (cdf + z.abs() * density) * part + 1e-38)


# ---- long sums --------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act,rows,chunk", [("f16", 1200000, 16384), ("bf16", 4000000, 131072)])
@pytest.mark.parametrize("N,K,counts", [(64, 72, None), (72, 64, "one"), (136, 264, "few")])
def test_weight_gradient_in_16_bits_of_very_many_rows(moe, dev, act, rows, chunk, N, K, counts):
    """Sums of one sign, of which n rows in one accumulator come out up to n 2^-27 short: a chunk loses a quarter of
    the output's half step. Columns of many scales, so that the rounding of the outputs has no common sign."""
    if counts == "few":
        rows //= 4
    g = torch.Generator(device=dev).manual_seed(N)
    dt = plain.DT[act]
    dy, x = (torch.empty((rows, n), dtype=dt, device=dev).uniform_(0.05, 0.15, generator=g) for n in (N, K))
    dy *= torch.empty(N, dtype=dt, device=dev).uniform_(0.5, 2.0, generator=g)
    split = {None: None, "one": [0, rows], "few": [0, 77, 77, rows // 5, rows - 3, rows - 3]}[counts]
    off = torch.tensor(split, dtype=torch.int32, device=dev) if split else None
    E = len(split) - 1 if split else 1
    dw, again = (torch.empty((E, N, K), dtype=dt, device=dev) for _ in range(2))
    for o in (dw, again):
        moe.moe_ragged_wgrad(dy, x, moe.ACT_CODES[act], off, rows, N, K, E, None, o, False)
    assert torch.equal(dw, again)
    bounds = split or [0, rows]
    for e in range(E):
        ref = torch.zeros((N, K), dtype=torch.float64, device=dev)
        for lo in range(bounds[e], bounds[e + 1], 1 << 19):
            hi = min(lo + (1 << 19), bounds[e + 1])
            ref += dy[lo:hi].double().T @ x[lo:hi].double()
        n = bounds[e + 1] - bounds[e]
        lost = min(chunk, n) * 2.0 ** -27 + (n // chunk + 16) * F32  # and the sum of the chunks
        plain.close(dw[e], ref.cpu(), act, ref.cpu() * lost)
        if n > chunk:  # the rounding's mean over N K outputs: six of its deviations, U / sqrt(3 N K) each
            mean = float(((dw[e].double() - ref) / ref).mean())
            assert abs(mean) <= lost + 6 * plain.U[act] / math.sqrt(3 * N * K)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("addend", [None, "apart", "in place"])
@pytest.mark.parametrize("rows,N,K,counts", [
    (600, 264, 136, None), (5000, 264, 520, None), (4200, 136, 72, None), (30000, 520, 264, None),
    (200000, 136, 264, None), (4100, 1032, 1000, None), (9000, 2816, 2048, None),
    (641, 72, 136, "one"), (5000, 520, 264, "one"), (12000, 512, 520, "few"), (40000, 264, 1032, "few"),
    (9000, 136, 72, "many"), (70000, 520, 1416, "many"), (4100, 264, 520, "uneven"), (9000, 72, 1032, "uneven")])
def test_f32_gradients_are_as_good_as_sums_in_f32(moe, dev, act, addend, rows, N, K, counts):
    """Rows of random signs, as gradients are: off by 1e-6 of their 2-norm at most however many rows, which is what a
    plain f32 product of 4096 rows has. (640 rows in one accumulator, 40 steps of 16: measured 8.0e-7 in f16 and 6.0e-7 in
    bf16. The chunks are added in f32.)"""
    g = torch.Generator(device=dev).manual_seed(rows + N)
    dt = plain.DT[act]
    dy, x = (torch.randn((rows, n), generator=g, device=dev).to(dt) for n in (N, K))
    split = {None: None, "one": [0, rows], "few": [5, 5, rows // 3, rows // 3 + 511, rows - 2],
             "many": list(range(0, rows + 1, rows // 40))[:41],
             "uneven": [0, rows - 90] + list(range(rows - 89, rows - 69)) + [rows]}[counts]  # one long group, many short
    off = torch.tensor(split, dtype=torch.int32, device=dev) if split else None
    bounds = split or [0, rows]
    E = len(bounds) - 1
    add = torch.randn((E, N, K), generator=g, device=dev) if addend else None
    outs = []
    for _ in range(2):
        dw = add.clone() if addend == "in place" else torch.full((E, N, K), 7.0, device=dev)
        moe.moe_ragged_wgrad(dy, x, moe.ACT_CODES[act], off, rows, N, K, E, dw if addend == "in place" else add, dw, True)
        outs.append(dw)
    assert torch.equal(*outs)
    for e in range(E):
        at = slice(bounds[e], bounds[e + 1])
        ref = torch.zeros((N, K), dtype=torch.float64, device=dev)
        for lo in range(bounds[e], bounds[e + 1], 1 << 17):
            hi = min(lo + (1 << 17), bounds[e + 1])
            ref += dy[lo:hi].double().T @ x[lo:hi].double()
        size = float(ref.norm())
        if addend:
            ref += add[e].double()
        assert float((outs[0][e].double() - ref).norm()) <= 1e-6 * size + F32 * float(ref.norm()), (e, at)
        if bounds[e] == bounds[e + 1]:
            assert torch.equal(outs[0][e].double(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N,K,one", [(3000, 264, 520, False), (3000, 264, 520, True), (100000, 136, 72, False),
                                          (40000, 520, 264, True)])
def test_f32_gradients_of_one_sign(moe, dev, act, rows, N, K, one):
    """640 rows in one accumulator come out 640 2^-27 = 4.8e-6 short at most; the chunks are added in f32."""
    g = torch.Generator(device=dev).manual_seed(N)
    dy, x = (torch.empty((rows, n), dtype=plain.DT[act], device=dev).uniform_(0.05, 0.15, generator=g) for n in (N, K))
    off = torch.tensor([0, rows], dtype=torch.int32, device=dev) if one else None
    dw = torch.empty((N, K), device=dev)
    moe.moe_ragged_wgrad(dy, x, moe.ACT_CODES[act], off, rows, N, K, 1, None, dw, True)
    ref = dy.double().T @ x.double()
    assert torch.all((dw.double() - ref).abs() <= ref * (640 * 2.0 ** -27 + (rows / 640 + 8) * F32))


@pytest.mark.gpu
@pytest.mark.parametrize("act,f32,rows", [("bf16", True, 640), ("f16", True, 1280), ("bf16", True, 5120),
                                          ("f16", False, 16384), ("f16", False, 131072), ("bf16", False, 131072)])
@pytest.mark.parametrize("grouped", [False, True])
def test_gradients_around_a_chunk(moe, dev, act, f32, rows, grouped):
    """One row, a few and a unit of 16 less and more than a whole number of chunks, of one group in the split form and
    of two in the pairs'."""
    N, K, dt, code = 136, 72, plain.DT[act], moe.ACT_CODES[act]
    g = torch.Generator(device=dev).manual_seed(rows)
    dy, x = (torch.randn((rows + 40, n), generator=g, device=dev).to(dt) for n in (N, K))
    dy[rows + 17:], x[rows + 17:] = math.nan, math.inf  # no group's
    for n in (rows - 17, rows - 16, rows - 1, rows, rows + 1, rows + 16, rows + 17):
        off = torch.tensor([0, n, n], dtype=torch.int32, device=dev) if grouped else None
        E = 2 if grouped else 1
        dw = torch.full((E, N, K), 7.0, dtype=torch.float32 if f32 else dt, device=dev)
        moe.moe_ragged_wgrad(dy, x, code, off, rows + 40 if grouped else n, N, K, E, None, dw, f32)
        d, xe = dy[:n].double(), x[:n].double()
        ref, mag = d.T @ xe, d.abs().T @ xe.abs()
        lost = mag * (min(n, 640 if f32 else 16384 if act == "f16" else 131072) * 2.0 ** -27 + 300 * F32)
        if f32:
            assert torch.all((dw[0].double() - ref).abs() <= lost), n
        else:
            plain.close(dw[0], ref.cpu(), act, lost.cpu())
        assert not grouped or torch.all(dw[1] == 0)


# ---- waits that run out -----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("limit_ns", [1, 300])
@pytest.mark.parametrize("call", ["dense", "groups", "transposed", "gradient", "gradient in chunks"])
def test_split_form_reports_a_wait_that_runs_out(moe, dev, call, limit_ns):
    """Contractions so long that the wait for a tile's last product (45 us and more) outlasts any first look at its
    barrier, with a limit far below: the call ends, the status is there, and the next call is the clean one."""
    g = torch.Generator(device=dev).manual_seed(1)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    chunks = call == "gradient in chunks"  # f16: of 16384 rows each, 60 us (those of an f32 gradient are too short)
    dtype = torch.float16 if chunks else torch.bfloat16

    def randn16(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    if call == "dense":
        M, N, K = 40, 264, 131072
        a, w = randn16(M, K), randn16(N, K)

        def run(out):
            moe.moe_dense_gemm(a, 0, w, None, 0, None, None, out, M, N, K, err)
        shape = M, N
    elif call.startswith("gradient"):
        rows, N, K = 300000 if chunks else 100000, 264, 136
        a, w = randn16(rows, N), randn16(rows, K)

        def run(out):
            moe.moe_ragged_wgrad(a, w, 1 if chunks else 0, None, rows, N, K, 1, None, out, False, err)
        shape = N, K
    else:
        tr, counts = call == "transposed", [30, 0, 41, 29]
        N, K = (65536, 520) if tr else (520, 65536)
        a, w, off = randn16(100, N if tr else K), randn16(4, N, K), offsets_of(counts).to(dev)

        def run(out):
            moe.moe_ragged_gemm(a, 0, w, tr, off, 100, N, K, 4, out, err)
        shape = 100, K if tr else N
    want, out = (torch.empty(shape, dtype=dtype, device=dev) for _ in range(2))
    run(want)
    assert err.item() == 0
    old = moe.moe_set_wait_limit_ns(limit_ns)
    try:
        run(out)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(old)
    assert err.item() == moe.MOE_DEV_ERR_TIMEOUT
    err.zero_()
    run(out)
    assert err.item() == 0 and torch.equal(out, want)


# ---- devices ----------------------------------------------------------------------------------------

def test_tensors_and_devices_have_to_fit_the_object(monkeypatch):
    """The checks themselves, with stand-ins for tensors and for the current device."""
    from mixture_experts_grouped_gb300 import ffn
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        ffn._cuda_device("cpu")
    here = ffn._cuda_device("cuda")
    assert here == torch.device("cuda:1") and ffn._cuda_device("cuda:0") == torch.device("cuda:0")
    ffn._require_current(here)
    with pytest.raises(ValueError):
        ffn._require_current(torch.device("cuda:0"))

    def tensor(device="cuda:1", dtype=torch.float16, shape=(4, 8), dense=True):
        return SimpleNamespace(device=torch.device(device), dtype=dtype, shape=shape, is_contiguous=lambda: dense)

    ffn._require("x", tensor(), here, torch.float16, 4, 8)
    for bad in (tensor("cuda:0"), tensor("cpu"), tensor(dtype=torch.bfloat16), tensor(shape=(4, 7)), tensor(dense=False)):
        with pytest.raises(ValueError):
            ffn._require("x", bad, here, torch.float16, 4, 8)


def training_objects(dev, device):
    from mixture_experts_grouped_gb300 import train
    T, H, I, E, k, bf = 4, 64, 32, 3, 2, dict(dtype=torch.bfloat16, device=dev)
    layer = train.MoeTrainLayer(T, H, I, E, k, "bf16", torch.zeros((E, 2 * I, H), **bf), torch.zeros((E, H, I), **bf),
                                device)
    block = train.DenseMlp(T, H, I, "bf16", "gelu", *(torch.zeros(s, **bf) for s in ((I, H), (I,), (H, I), (H,))),
                           device)
    return layer, block, torch.zeros((T, H), **bf), torch.zeros((T, E), device=dev)


def test_training_objects_need_a_cuda_device():
    from mixture_experts_grouped_gb300 import train
    w = torch.zeros((3, 64, 64)), torch.zeros((3, 64, 32))
    with pytest.raises(ValueError):
        train.MoeTrainLayer(4, 64, 32, 3, 2, "bf16", *w, device="cpu")
    with pytest.raises(ValueError):
        train.DenseMlp(4, 64, 32, "bf16", "gelu", w[0], None, w[1], None, device="cpu")


@pytest.mark.gpu
def test_training_objects_run_on_their_own_device_alone(moe, dev, monkeypatch):
    layer, block, x, logits = training_objects(dev, "cuda")
    layer.forward(x, logits)
    block.forward(x)
    n0 = moe.moe_launch_count()
    for device in ("cpu", "cuda:1"):  # buffers apart from the weights
        with pytest.raises(ValueError):
            training_objects(dev, device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: layer.forward(x, logits), lambda: layer.backward(x), lambda: block.forward(x),
                 lambda: block.backward(x)):
        with pytest.raises(ValueError):
            call()
    assert moe.moe_launch_count() == n0


@pytest.mark.gpu
def test_dense_expert_refuses_what_does_not_fit(moe, dev, monkeypatch):
    from mixture_experts_grouped_gb300 import ffn
    from mixture_experts_grouped_gb300 import layer as L
    T, H, I, bf = 4, 64, 32, dict(dtype=torch.bfloat16, device=dev)
    w = torch.zeros((2 * I, H), **bf), torch.zeros((H, I), **bf)
    expert = ffn.DenseExpert(T, H, I, "bf16", *w)
    x = torch.ones((T, H), **bf)
    assert torch.equal(expert.forward(x, x), x)
    n0 = moe.moe_launch_count()
    for bad in (x[:3], x[:, :32], x.half(), x.float(), x.T.contiguous().T, x.cpu()):
        for args in ((bad,), (bad, x), (x, bad)):
            with pytest.raises(ValueError):
                expert.forward(*args)
    for bad in ((w[0].cpu(), w[1]), (w[0], w[1].half()), (w[1], w[0])):
        with pytest.raises(ValueError):
            ffn.DenseExpert(T, H, I, "bf16", *bad)
    for device in ("cpu", "cuda:1"):
        with pytest.raises(ValueError):
            ffn.DenseExpert(T, H, I, "bf16", *w, device=device)
    desc = [L.DeviceWeight(moe.MoeWeight(moe.MOE_W_BF16, 0, t.data_ptr(), None, None, None), [t])
            for t in (torch.zeros((3, 2 * I, H), **bf), torch.zeros((3, H, I), **bf))]
    norm, router = torch.ones(H, **bf), torch.zeros((H, 3), device=dev)
    for device in ("cpu", "cuda:1"):
        with pytest.raises(ValueError):
            ffn.FeedForward(T, H, I, 3, 2, "bf16", norm, router, *desc, expert, device=device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        expert.forward(x)
    assert moe.moe_launch_count() == n0


# ---- an object's own buffers as its inputs -----------------------------------------------------------

def test_buffers_that_an_input_must_not_share():
    from mixture_experts_grouped_gb300 import ffn
    pool = torch.zeros(64)
    own = ffn._Buffers(SimpleNamespace(a=pool[:16], b=pool[16:32], none=None), "a", "b", "none")
    own.refuse("x", pool[32:])
    own.refuse("x", pool[:16], ("b",))
    own.refuse("x", pool[16:32], in_place="b")
    own.refuse("x", torch.zeros(0))
    for bad in (pool[:16], pool[15:16], pool[8:24], pool[31:40], pool):
        with pytest.raises(ValueError):
            own.refuse("x", bad)
    for bad in (pool[16:24], pool[20:32], pool[24:40], pool[8:24]):  # not exactly b
        with pytest.raises(ValueError):
            own.refuse("x", bad, ("b",), in_place="b")


@pytest.mark.gpu
def test_dense_block_refuses_every_buffer_that_it_overwrites(moe, dev):
    from mixture_experts_grouped_gb300 import train
    T, H, bf = 8, 64, dict(dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    w = [torch.randn(s, generator=g, device=dev).bfloat16() / 8 for s in ((H, H), (H,), (H, H), (H,))]
    block = train.DenseMlp(T, H, H, "bf16", "gelu", *w)  # H = I: every buffer has x's shape
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    out = block.forward(x).clone()
    dx = block.backward(x).clone()
    n0 = moe.moe_launch_count()
    whole = {n: getattr(block, n) for n in ("pre", "h", "out", "d_h", "d_x")}
    whole["d_w1"] = block.d_w1.view(torch.bfloat16).flatten()[16: 16 + T * H].view(T, H)  # within
    for t in whole.values():
        with pytest.raises(ValueError):
            block.forward(t)
    for n in ("pre", "h"):
        with pytest.raises(ValueError):
            block.forward(x, residual=whole[n])
    with pytest.raises(ValueError):
        block.backward(whole["d_h"])
    assert moe.moe_launch_count() == n0
    # what a pass has read before it writes it: the last output added in place, gradients that are outputs
    added = block.forward(x, residual=x).clone()
    assert torch.equal(block.forward(x, residual=block.d_x.copy_(x)), added)
    assert torch.equal(block.forward(x, residual=block.out.copy_(x)), added)
    assert torch.equal(block.forward(x), out)
    assert torch.equal(block.backward(block.d_x.copy_(x)), dx)


@pytest.mark.gpu
def test_expert_layer_refuses_every_buffer_that_it_overwrites(moe, dev):
    from mixture_experts_grouped_gb300 import train
    T, H, E = 8, 64, 2
    g = torch.Generator(device=dev).manual_seed(2)
    w = [torch.randn(s, generator=g, device=dev).bfloat16() / 8 for s in ((E, 2 * H, H), (E, H, H))]
    layer = train.MoeTrainLayer(T, H, H, E, 1, "bf16", *w, renormalize=False)  # one expert a token: rows are tokens
    both = train.MoeTrainLayer(T, H, H, E, E, "bf16", *w)                      # all: weights have the logits' shape
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    logits = torch.randn((T, E), generator=g, device=dev)
    out = layer.forward(x, logits).clone()
    dx, dl = (t.clone() for t in layer.backward(x))
    n0 = moe.moe_launch_count()
    for call in (lambda: layer.forward(layer.xs, logits), lambda: layer.forward(x, layer.d_logits),
                 lambda: both.forward(x, both.topk_weights), lambda: both.forward(x, both.d_weights),
                 lambda: layer.backward(layer.d_y),
                 lambda: layer.forward(x, layer.d_down.flatten()[3: 3 + T * E].view(T, E))):
        with pytest.raises(ValueError):
            call()
    assert moe.moe_launch_count() == n0
    # what a pass has read before it writes it
    assert torch.equal(layer.forward(layer.out.copy_(x), logits), out)
    assert torch.equal(layer.forward(layer.d_x.copy_(x), logits), out)
    assert all(torch.equal(a, b) for a, b in zip(layer.backward(layer.d_x.copy_(x)), (dx, dl)))


@pytest.mark.gpu
def test_dense_expert_refuses_every_buffer_that_it_overwrites(moe, dev):
    from mixture_experts_grouped_gb300 import ffn
    T, H = 8, 64
    g = torch.Generator(device=dev).manual_seed(3)
    w = [torch.randn(s, generator=g, device=dev).bfloat16() / 8 for s in ((2 * H, H), (H, H))]
    expert = ffn.DenseExpert(T, H, H, "bf16", *w)
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    out = expert.forward(x, x).clone()
    n0 = moe.moe_launch_count()
    within = expert.gate_up.flatten()[8: 8 + T * H].view(T, H)
    for args in ((within,), (x, within), (x, expert.h)):
        with pytest.raises(ValueError):
            expert.forward(*args)
    assert moe.moe_launch_count() == n0
    assert torch.equal(expert.forward(x, expert.out.copy_(x)), out)
    assert torch.equal(expert.forward(expert.out.copy_(x), x), out)
    assert torch.equal(expert.forward(expert.h.copy_(x), x), out)


@pytest.mark.gpu
def test_a_pass_that_was_refused_midway_has_no_backward_pass(moe, dev):
    """E above the routing's limit: the layer's first call refuses it, and what is left in the buffers is no forward
    pass."""
    from mixture_experts_grouped_gb300 import train
    T, H, I, E, k, bf = 4, 64, 32, moe.MOE_MAX_EXPERTS + 1, 2, dict(dtype=torch.bfloat16, device=dev)
    layer = train.MoeTrainLayer(T, H, I, E, k, "bf16", torch.zeros((E, 2 * I, H), **bf), torch.zeros((E, H, I), **bf))
    x, logits = torch.zeros((T, H), **bf), torch.zeros((T, E), device=dev)
    with pytest.raises(moe.MoeError):
        layer.forward(x, logits)
    with pytest.raises(RuntimeError, match="without a forward pass"):
        layer.backward(x)
    block = train.DenseMlp(T, 60, I, "bf16", "gelu", torch.zeros((I, 60), **bf), None, torch.zeros((60, I), **bf), None)
    with pytest.raises(moe.MoeError):
        block.forward(torch.zeros((T, 60), **bf))
    with pytest.raises(RuntimeError, match="without a forward pass"):
        block.backward(torch.zeros((T, 60), **bf))
