"""GPU channel-wise operators (layer norm, 8-bit checkpoints, channel product) against plain 64-bit forms, within
bounds derived from the operations (channel_ref.py counts the roundings)."""
import pytest
import torch

import channel_ref as ref
import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = [c3.ACT_NONE, c3.ACT_SILU, c3.ACT_GELU]


def rand(shape, seed, stream, std=1.0, dtype=torch.bfloat16, mean=0.0):
    return (si.tensor(shape, seed, stream, std, torch.float32, "cuda") + mean).to(dtype)


def sync_ok():
    assert c3.poll_status() == c3.Status.OK, c3.last_error()


def guarded(n, dtype, extra=512):
    """A buffer of n elements between canaries: (view of the n, checker)."""
    es = torch.empty((), dtype=dtype).element_size()
    pad = extra // es
    raw = torch.full((n + 2 * pad,), 77, dtype=dtype, device="cuda")

    def intact():
        assert (raw[:pad] == 77).all() and (raw[pad + n:] == 77).all(), "written outside the output"
    return raw[pad:pad + n], intact


def ckpt(rows, C, seed, std=1.0):
    return ref.checkpoint(si.tensor((rows, C), seed, 9, std, torch.float32, "cuda").double(), "cuda")


# ---------------------------------------------------------------- layer norm

LN_SHAPES = [(1, 8), (3, 24), (257, 40), (2, 64), (1001, 72), (130, 128), (77, 136), (4099, 256), (5, 264), (611, 512),
             (1, 520), (333, 1000), (64, 1024), (9, 1032), (37, 2048), (301, 2056), (6, 4096), (3, 8192)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layernorm_forward(rows, C, dtype):
    dt = DT[dtype]
    x = rand((rows, C), 1, 0, 1.5, dt, 3.0)
    gamma, beta = rand((C,), 1, 1, 0.3, dt, 1.0), rand((C,), 1, 2, 0.3, dt)
    y, mean, rstd = c3.layernorm(x, gamma, beta, 1e-5, with_stats=True)
    sync_ok()
    ry, rmean, rrstd, rxh = ref.layernorm(x.double(), gamma.double(), beta.double(), 1e-5)
    # fp32: at most 2^5 roundings of values up to max|x| in the mean and the deviations
    off = (x.double().abs().amax(-1) + rmean.abs()) * 2.0 ** -19
    ref.check(mean, rmean, off, "mean")
    ref.check(rstd, rrstd, rrstd * 2.0 ** -18 + off * rrstd * rrstd, "rstd")
    xh_off = (off * rrstd)[:, None] + rxh.abs() * (2.0 ** -18 + (off * rrstd)[:, None])
    bound = ref.rounding(ry, dt) * 1.01 + gamma.double().abs() * xh_off + beta.double().abs() * 2.0 ** -22
    ref.check(y, ry, bound, "y")
    # with the checkpoint of the normalised values: the same y, and codes within half a step of them
    y8, a, rstd8 = c3.layernorm(x, gamma, beta, 1e-5, checkpoint8=True)
    sync_ok()
    assert torch.equal(y8, y) and torch.equal(rstd8, rstd)
    nb = -(-C // 32)
    assert tuple(a.codes.shape) == (rows, 32 * nb) and tuple(a.exponents.shape) == (rows, nb)
    if C % 32:
        assert (a.codes[:, C:] == 0).all()
    step = ref.step_of(a)
    clamped = (a.codes[:, :C].abs() == 127).double()
    ref.check(ref.decode(a), rxh, step * (0.5 + 0.5 * clamped) + xh_off, "checkpoint")
    _, e = ref.codes(rxh)
    differ = (a.exponents.long() != e)
    assert differ.double().mean().item() <= 1e-3        # only a maximum beside a power of two


@pytest.mark.parametrize("C", [64, 520, 2048])
def test_layernorm_without_parameters_in_place_and_nothing_outside(C):
    rows = 61
    x = rand((rows, C), 2, 0, 1.0, torch.bfloat16)
    want = c3.layernorm(x)
    ones, zeros = torch.ones(C, dtype=x.dtype, device="cuda"), torch.zeros(C, dtype=x.dtype, device="cuda")
    assert torch.equal(want, c3.layernorm(x, ones, zeros))
    buf, intact = guarded(rows * C, torch.bfloat16)
    y = buf.view(rows, C)
    y.copy_(x)
    assert c3.layernorm(y, y=y) is y
    sync_ok()
    assert torch.equal(y, want)
    intact()


def test_layernorm_rows_are_independent_of_their_neighbours():
    """Rows of NaN, infinities and constants beside ordinary ones."""
    C = 256
    x = rand((9, C), 3, 0)
    want = c3.layernorm(x)
    x[2], x[4], x[6] = float("nan"), 5.0, float("inf")
    y, a, rstd = c3.layernorm(x, checkpoint8=True)
    sync_ok()
    for r in (0, 1, 3, 5, 7, 8):
        assert torch.equal(y[r], want[r])
    assert torch.isnan(y[2]).all() and torch.isnan(y[6]).all() and (y[4] == 0).all()
    assert (a.exponents[2] == 255).all() and (a.exponents[6] == 255).all() and (a.exponents[4] == 7).all()
    v = c3.act8_unpack(a, x.dtype)
    assert torch.isnan(v[2]).all() and (v[4] == 0).all() and torch.isfinite(v[3]).all()


@pytest.mark.parametrize("from_codes", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layernorm_backward(rows, C, dtype, from_codes):
    dt = DT[dtype]
    dy, gamma = rand((rows, C), 4, 0, 1.0, dt), rand((C,), 4, 1, 0.3, dt, 1.0)
    dres = rand((rows, C), 4, 2, 1.0, dt) if rows % 2 else None
    if from_codes:
        saved, mean = ckpt(rows, C, 4), None
        rstd = torch.rand((rows,), device="cuda") + 0.5
        xh, xh_off = ref.decode(saved), 0.0
    else:
        saved = rand((rows, C), 4, 3, 1.5, dt, 0.5)
        _, mean, rstd, _ = ref.layernorm(saved.double(), 1.0, 0.0, 1e-6)
        mean, rstd = mean.float(), rstd.float()
        xh = (saved.double() - mean.double()[:, None]) * rstd.double()[:, None]
        xh_off = 2.0 ** -22 * (saved.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    dx, dg, db = c3.layernorm_bwd(dy, saved, rstd, mean, gamma, dres)
    sync_ok()
    rdx, rdg, rdb = ref.layernorm_bwd(dy.double(), xh, rstd.double(), gamma.double())
    g = (dy.double() * gamma.double()).abs()
    # fp32 sums over C (at most 2^6 roundings deep), then a handful of operations
    c2 = (g * xh.abs()).mean(-1, keepdim=True)
    terms = g + g.mean(-1, keepdim=True) + xh.abs() * c2
    bound = rstd.double()[:, None] * (2.0 ** -17 * terms + xh_off * c2 + xh.abs() * (g * xh_off).mean(-1, keepdim=True))
    if dres is not None:
        rdx = rdx + dres.double()
    ref.check(dx, rdx, ref.rounding(rdx, dt) * 1.01 + bound + 2.0 ** -23 * rdx.abs(), "dx")
    # fp32 sums of a thread's, a block's and the blocks' terms: at most 2^8 roundings deep
    ref.check(dg, rdg, ref.rounding(rdg, dt) * 1.01 + (dy.double().abs() * (2.0 ** -16 * xh.abs() + xh_off)).sum(0), "dgamma")
    ref.check(db, rdb, ref.rounding(rdb, dt) * 1.01 + 2.0 ** -16 * dy.double().abs().sum(0), "dbeta")
    # again: the same bits; without parameter gradients: the same dx, no workspace
    again = c3.layernorm_bwd(dy, saved, rstd, mean, gamma, dres)
    only = c3.layernorm_bwd(dy, saved, rstd, mean, gamma, dres, with_params=False)
    sync_ok()
    assert all(torch.equal(p, q) for p, q in zip((dx, dg, db), again))
    assert torch.equal(only[0], dx) and only[1] is None


@pytest.mark.parametrize("C", [72, 512, 1032])
def test_layernorm_backward_in_place(C):
    rows = 75
    dy, x, dres = (rand((rows, C), 5, i) for i in range(3))
    _, mean, rstd = c3.layernorm(x, with_stats=True)
    want = c3.layernorm_bwd(dy, x, rstd, mean, None, dres)
    for target in ("dy", "x", "dres"):
        t = {"dy": dy.clone(), "x": x.clone(), "dres": dres.clone()}
        got = c3.layernorm_bwd(t["dy"], t["x"], rstd, mean, None, t["dres"], dx=t[target])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), target
    buf, intact = guarded(rows * C, torch.bfloat16)
    c3.layernorm_bwd(dy, x, rstd, mean, None, dres, dx=buf.view(rows, C))
    sync_ok()
    intact()


# ---------------------------------------------------------------- 8-bit checkpoints

A8_SHAPES = [(1, 8), (1, 32), (5, 16), (33, 40), (100, 64), (7, 136), (1000, 520), (4097, 256), (3, 9000)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,C", A8_SHAPES)
def test_pack_codes_and_unpacked_values_are_exact(rows, C, dtype):
    dt = DT[dtype]
    x = rand((rows, C), 6, 0, 1.0, dt) * torch.exp2(torch.arange(rows, device="cuda") % 9 - 4.0)[:, None].to(dt)
    x[:, ::7] = 0
    x[0] = 0                                              # a block of zeros
    a = c3.act8_pack(x)
    v = c3.act8_unpack(a, dt)
    sync_ok()
    k, e = ref.codes(x.double())
    assert torch.equal(a.codes.long(), k) and torch.equal(a.exponents.long(), e)
    assert torch.equal(v.double(), ref.decode(a))         # every code is exact in the type it came from


def test_pack_at_the_ends_of_the_range():
    """The smallest and largest values, infinities and NaN, block by block."""
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros((1, 32 * 7), dtype=torch.bfloat16, device="cuda")
    x[0, 0] = big
    x[0, 33] = 2.0 ** -126                                # smallest normal
    x[0, 70] = 2.0 ** -133                                # smallest subnormal: below half a step of 2^-126
    x[0, 100], x[0, 101] = float("inf"), 1.0
    x[0, 130], x[0, 131] = float("nan"), 1.0
    x[0, 160], x[0, 161] = -1.0, 0.0078125
    x[0, 195] = float("-inf")
    a = c3.act8_pack(x)
    v = c3.act8_unpack(a, torch.bfloat16).view(7, 32)
    d = c3.act8_bwd(torch.ones_like(x), a, c3.ACT_SILU).view(7, 32)
    sync_ok()
    assert a.exponents.tolist() == [[254, 7, 7, 255, 255, 127, 255]]
    assert v[0, 0].item() == 127 * 2.0 ** 121             # 127.5 steps and more clamp to 127
    assert v[1, 1].item() == 2.0 ** -126 and (v[2] == 0).all()
    assert torch.isnan(v[[3, 4, 6]]).all() and torch.isnan(d[[3, 4, 6]]).all()
    assert v[5, 0].item() == -1.0 and v[5, 1].item() == 0.0   # half a step rounds to even
    assert d[0, 0].item() == 1.0 and torch.isfinite(d[[0, 1, 2, 5]]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,C", A8_SHAPES)
def test_unpack_recomputes(rows, C, dtype, affine, act):
    dt = DT[dtype]
    a = ckpt(rows, C, 7, 2.0)
    gamma, beta = (rand((C,), 7, 1, 0.3, dt, 1.0), rand((C,), 7, 2, 0.3, dt)) if affine else (None, None)
    buf, intact = guarded(rows * C, dt)
    y = c3.act8_unpack(a, dt, gamma, beta, act, y=buf.view(rows, C))
    sync_ok()
    v = ref.decode(a)
    off = torch.zeros_like(v)
    if affine:
        off = 2.0 ** -23 * ((v * gamma.double()).abs() + beta.double().abs())
        v = v * gamma.double() + beta.double()
    want = ref.act(v, act)
    ref.check(y, want, ref.rounding(want, dt) * 1.01 + 1.2 * off + ref.act_error(v, act), "y")
    intact()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,C", A8_SHAPES)
def test_activation_gradient_from_the_checkpoint(rows, C, dtype, act):
    dt = DT[dtype]
    a = ckpt(rows, C, 8, 2.0)
    dy = rand((rows, C), 8, 1, 1.0, dt)
    dx = c3.act8_bwd(dy, a, act)
    sync_ok()
    v = ref.decode(a)
    want = dy.double() * ref.slope(v, act)
    bound = dy.double().abs() * ref.slope_error(v, act)
    ref.check(dx, want, ref.rounding(want, dt) * 1.01 + bound, "dx")
    inplace = dy.clone()
    assert c3.act8_bwd(inplace, a, act, dx=inplace) is inplace and torch.equal(inplace, dx)


def test_activations_far_from_zero():
    """Saturated arguments: the derivative is 0 or 1, the value v or 0."""
    v = torch.tensor([[1.0, 8.0, 30.0, 1e4, 1e19, 3e38, -1.0, -8.0, -30.0, -1e4, -1e19, -3e38] * 4], dtype=torch.float64)
    a = ref.checkpoint(v.T.reshape(-1, 1).repeat(1, 8), "cuda")       # every value its own block
    val = ref.decode(a)
    for act in (c3.ACT_SILU, c3.ACT_GELU):
        y = c3.act8_unpack(a, torch.bfloat16, act=act).double()
        d = c3.act8_bwd(torch.ones((48, 8), dtype=torch.bfloat16, device="cuda"), a, act).double()
        sync_ok()
        want = torch.where(val < -1e5, torch.zeros_like(val), ref.act(val, act))
        big = val.abs() > 1e5
        assert torch.isfinite(y).all() and torch.isfinite(d).all()
        ref.check(y, want, torch.where(big, want.abs() * 2.0 ** -8, ref.rounding(want, torch.bfloat16) * 1.01 + ref.act_error(val, act)), "y")
        ref.check(d, torch.where(big, (val > 0).double(), ref.slope(val.clamp(-1e5, 1e5), act)),
                  # beyond 25 the derivative is within (|v| + 1) e^-|v| <= 26 e^-25 < 2^-31 of 0 or 1, which is returned
                  torch.where(val.abs() > 25, torch.full_like(val, 2.0 ** -31), 2.0 ** -8 + ref.slope_error(val, act)), "slope")


# ---------------------------------------------------------------- channel product

def product_case(M, K, N, dt, seed=11):
    return dict(x=rand((M, K), seed, 0, 1.0, dt), w=rand((N, K), seed, 1, K ** -0.5, dt),
                bias=rand((N,), seed, 2, 0.3, dt), residual=rand((M, N), seed, 3, 1.0, dt))


def sum_error(x, w):
    """fp32 accumulation in any order, truncating: one step of 2^-23 per product."""
    return (w.shape[1] + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t())


LIN_SHAPES = [(1, 8, 8), (1, 512, 2048), (2, 64, 136), (16, 520, 264), (17, 1024, 96), (61, 1024, 1000), (128, 72, 512),
              (129, 512, 520), (300, 264, 40), (1000, 128, 512), (2049, 200, 1032), (4100, 512, 512)]


def run_linear(p, act, bias, residual, checkpoint8):
    return c3.linear(p["x"], p["w"], p["bias"] if bias else None, p["residual"] if residual else None, act,
                     checkpoint8=checkpoint8)


def check_linear(p, dt, act, bias, residual, y, a):
    pre = p["x"].double() @ p["w"].double().t()
    off = sum_error(p["x"], p["w"])
    if bias:
        pre = pre + p["bias"].double()
        off = off + 2.0 ** -23 * pre.abs()
    want = ref.act(pre, act)
    bound = 1.13 * off + ref.act_error(pre, act)          # |act'| < 1.13
    if residual:
        want = want + p["residual"].double()
        bound = bound + 2.0 ** -23 * want.abs()
    ref.check(y, want, ref.rounding(want, dt) * 1.01 + bound, "y")
    if a is not None:
        C = a.channels
        if C % 32:
            assert (a.codes[..., C:] == 0).all()
        step = ref.step_of(a)
        clamped = (a.codes[:, :C].abs() == 127).double()
        ref.check(ref.decode(a), pre, step * (0.5 + 0.5 * clamped) + off, "pre")
        _, e = ref.codes(pre)
        differ = a.exponents.long() != e
        assert ((a.exponents.long() - e).abs() <= 1).all() and differ.double().mean().item() <= max(1e-3, 1.0 / e.numel())


@pytest.mark.parametrize("kernel", ["", "1", "128", "256"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", LIN_SHAPES)
def test_linear_forward(M, K, N, dtype, kernel, monkeypatch):
    """Every size through the chosen kernel and through each of them by force."""
    if kernel:
        monkeypatch.setenv("CONV3D_LINEAR", kernel)
    dt = DT[dtype]
    p = product_case(M, K, N, dt)
    for act, bias, residual, checkpoint8 in ((0, False, False, False), (0, True, True, True), (1, True, False, True),
                                             (2, True, True, True), (2, True, False, False), (1, False, True, False)):
        out = run_linear(p, act, bias, residual, checkpoint8)
        sync_ok()
        y, a = out if checkpoint8 else (out, None)
        check_linear(p, dt, act, bias, residual, y, a)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_linear_of_a_token_or_a_few(M, dtype, monkeypatch):
    """The dot products, chosen and by force: odd sizes, one and two shares of the contraction, contractions that are
    too long for them (another kernel takes those), guarded outputs, the same bits with and without a checkpoint."""
    dt = DT[dtype]
    for K, N in ((8, 8), (24, 40), (512, 2048), (1000, 136), (1024, 520), (1032, 72), (2048, 264), (4096, 64), (4104, 1000),
                 (8192, 32), (20000, 96), (72, 5000)):
        p = product_case(M, K, N, dt, 21)
        for kernel in ("0", "2"):
            monkeypatch.setenv("CONV3D_LINEAR", kernel)
            for act, bias, residual in ((0, False, False), (1, True, True), (2, True, False)):
                y, a = run_linear(p, act, bias, residual, True)
                plain = run_linear(p, act, bias, residual, False)
                sync_ok()
                check_linear(p, dt, act, bias, residual, y, a)
                assert torch.equal(y, plain)
    monkeypatch.setenv("CONV3D_LINEAR", "2")
    K, N = 520, 200
    p = product_case(M, K, N, dt, 22)
    y, y_ok = guarded(M * N, dt)
    q, q_ok = guarded(M * 224, torch.int8)
    e, e_ok = guarded(M * 7, torch.uint8)
    y.copy_(p["residual"].flatten())
    code = c3.BF16 if dt == torch.bfloat16 else c3.F16
    assert c3.linear_fwd_ptr(p["x"].data_ptr(), p["w"].data_ptr(), p["bias"].data_ptr(), y.data_ptr(), y.data_ptr(),
                             q.data_ptr(), e.data_ptr(), M, K, N, 2, code, torch.cuda.current_stream().cuda_stream) == c3.Status.OK
    sync_ok()
    check_linear(p, dt, 2, True, True, y.view(M, N), c3.Act8(q.view(M, -1), e.view(M, 7), N))
    for ok in (y_ok, q_ok, e_ok):
        ok()
    p["x"][M - 1, 3] = float("nan")                     # a row of NaN leaves the others alone
    z, a = run_linear(p, 2, True, True, True)
    assert torch.equal(z[:M - 1], y.view(M, N)[:M - 1]) and torch.isnan(z[M - 1]).all() and (a.exponents[M - 1] == 255).all()


@pytest.mark.parametrize("split", ["1", "2", "3", "8"])
def test_linear_split_along_the_contraction(split, monkeypatch):
    monkeypatch.setenv("CONV3D_LINEAR", "1")
    monkeypatch.setenv("CONV3D_LINEAR_SPLIT", split)
    for M, K, N in ((1, 512, 256), (40, 712, 136), (200, 1024, 512)):
        p = product_case(M, K, N, torch.bfloat16, 12)
        y, a = run_linear(p, 2, True, True, True)
        y2, a2 = run_linear(p, 2, True, True, True)
        sync_ok()
        check_linear(p, torch.bfloat16, 2, True, True, y, a)
        assert torch.equal(y, y2) and torch.equal(a.codes, a2.codes)     # the same bits again


@pytest.mark.parametrize("kernel", ["1", "128", "256"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (61, 72, 1000), (300, 136, 520)])
def test_linear_writes_nothing_outside(M, K, N, kernel, monkeypatch):
    monkeypatch.setenv("CONV3D_LINEAR", kernel)
    p = product_case(M, K, N, torch.bfloat16, 13)
    nb = -(-N // 32)
    y, y_ok = guarded(M * N, torch.bfloat16)
    q, q_ok = guarded(M * nb * 32, torch.int8)
    e, e_ok = guarded(M * nb, torch.uint8)
    y.copy_(p["residual"].flatten())                       # in place: y is the residual
    assert c3.linear_fwd_ptr(p["x"].data_ptr(), p["w"].data_ptr(), p["bias"].data_ptr(), y.data_ptr(), y.data_ptr(),
                             q.data_ptr(), e.data_ptr(), M, K, N, 1, c3.BF16,
                             torch.cuda.current_stream().cuda_stream) == c3.Status.OK
    sync_ok()
    check_linear(p, torch.bfloat16, 1, True, True, y.view(M, N), c3.Act8(q.view(M, -1), e.view(M, nb), N))
    for ok in (y_ok, q_ok, e_ok):
        ok()
    d, d_ok = guarded(M * K, torch.bfloat16)
    c3.linear_bwd_data(p["residual"], p["w"], dx=d.view(M, K))
    sync_ok()
    d_ok()


def test_linear_does_not_mix_rows():
    """A row of NaN and one with infinities leave the others' bits alone; their blocks are marked."""
    for M in (20, 700):
        p = product_case(M, 256, 512, torch.bfloat16, 14)
        y0, _ = run_linear(p, 2, True, False, True)
        p["x"][3], p["x"][M - 1, 0] = float("nan"), float("inf")
        y, a = run_linear(p, 2, True, False, True)
        sync_ok()
        keep = [r for r in range(M) if r not in (3, M - 1)]
        assert torch.equal(y[keep], y0[keep])
        assert torch.isnan(y[3]).all() and (a.exponents[3] == 255).all() and (a.exponents[M - 1] == 255).all()


@pytest.mark.parametrize("kernel", ["", "1", "128", "256"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", LIN_SHAPES)
def test_linear_data_gradient(M, K, N, dtype, kernel, monkeypatch):
    if kernel:
        monkeypatch.setenv("CONV3D_LINEAR", kernel)
    dt = DT[dtype]
    dy, w = rand((M, N), 15, 0, 1.0, dt), rand((N, K), 15, 1, K ** -0.5, dt)
    pre = ckpt(M, K, 15, 1.5)
    v = ref.decode(pre)
    plain = dy.double() @ w.double()
    off = (N + 8) * 2.0 ** -23 * (dy.double().abs() @ w.double().abs())
    for act in ACTS:
        dx = c3.linear_bwd_data(dy, w, pre, act)
        sync_ok()
        s = ref.slope(v, act)
        want = plain * s
        bound = off * (s.abs() + ref.slope_error(v, act)) + plain.abs() * ref.slope_error(v, act) * (act != 0)
        ref.check(dx, want, ref.rounding(want, dt) * 1.01 + bound + 2.0 ** -23 * want.abs(), "dx")
        if act:
            again, x = c3.linear_bwd_data(dy, w, pre, act, with_x=True)
            sync_ok()
            assert torch.equal(again, dx) and torch.equal(x, c3.act8_unpack(pre, dt, act=act))


@pytest.mark.parametrize("rows", ["16", "32", "64", "128"])
@pytest.mark.parametrize("split", ["1", "2", "3", "5", "6", "7", "8"])
def test_linear_few_rows_in_any_pieces(split, rows, monkeypatch):
    """Every number of pieces hands every row to one rank, whatever the rows per tile; the same bits again."""
    monkeypatch.setenv("CONV3D_LINEAR", "1")
    monkeypatch.setenv("CONV3D_LINEAR_SPLIT", split)
    monkeypatch.setenv("CONV3D_LINEAR_ROWS", rows)
    for M, K, N in ((1, 136, 712), (5, 264, 512), (61, 72, 1000), (131, 136, 520)):
        p = product_case(M, N, K, torch.bfloat16, 19)              # forward: [M, N] -> [M, K]
        out = run_linear(p, 1, True, True, True)
        again = run_linear(p, 1, True, True, True)
        check_linear(p, torch.bfloat16, 1, True, True, *out)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1].codes, again[1].codes)
        dy, w = rand((M, N), 19, 4), rand((N, K), 19, 5, K ** -0.5)
        pre = ckpt(M, K, 19, 1.5)
        dx, x = c3.linear_bwd_data(dy, w, pre, 2, with_x=True)
        sync_ok()
        v = ref.decode(pre)
        s = ref.slope(v, 2)
        plain = dy.double() @ w.double()
        off = (N + 8) * 2.0 ** -23 * (dy.double().abs() @ w.double().abs())
        want = plain * s
        bound = off * (s.abs() + ref.slope_error(v, 2)) + plain.abs() * ref.slope_error(v, 2)
        ref.check(dx, want, ref.rounding(want, dx.dtype) * 1.01 + bound + 2.0 ** -23 * want.abs(), "dx")
        assert torch.equal(x, c3.act8_unpack(pre, dx.dtype, act=2))


@pytest.mark.parametrize("kernel", ["1", "128", "256"])
@pytest.mark.parametrize("M,K,N", [(1, 8, 64), (61, 1000, 72), (300, 520, 136)])
def test_linear_gradient_writes_nothing_outside(M, K, N, kernel, monkeypatch):
    monkeypatch.setenv("CONV3D_LINEAR", kernel)
    dy, w, pre = rand((M, N), 20, 0), rand((N, K), 20, 1, K ** -0.5), ckpt(M, K, 20, 1.5)
    d, d_ok = guarded(M * K, torch.bfloat16)
    x, x_ok = guarded(M * K, torch.bfloat16)
    assert c3.linear_bwd_data_ptr(dy.data_ptr(), w.data_ptr(), pre.codes.data_ptr(), pre.exponents.data_ptr(), 1, d.data_ptr(),
                                  x.data_ptr(), M, K, N, c3.BF16, torch.cuda.current_stream().cuda_stream) == c3.Status.OK
    sync_ok()
    d_ok()
    x_ok()
    assert torch.equal(d.view(M, K), c3.linear_bwd_data(dy, w, pre, 1))
    assert torch.equal(x.view(M, K), c3.act8_unpack(pre, torch.bfloat16, act=1))


@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("M", [37, 700])
def test_linear_data_gradient_recomputes_any_checkpoint(M, act):
    """Blocks whose values pass 64 (where the derivative's argument is cut off and the
    value's is not), tiny ones, and ones that hold an infinity or a NaN."""
    K, N = 1032, 256
    v = rand((M, K), 18, 0, 1.5)
    v[1::7] *= 100.0
    v[2::7] *= 1e30
    v[3::7] *= 1e-37
    v[4::7, 40] = float("inf")
    v[5::7, 1031] = float("nan")
    v[6::7, ::3] *= 50.0
    pre = c3.act8_pack(v)
    dy, w = rand((M, N), 18, 1), rand((N, K), 18, 2, K ** -0.5)
    dx = c3.linear_bwd_data(dy, w, pre, act)
    again, x = c3.linear_bwd_data(dy, w, pre, act, with_x=True)
    sync_ok()
    torch.testing.assert_close(again, dx, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(x, c3.act8_unpack(pre, v.dtype, act=act), rtol=0, atol=0, equal_nan=True)
    assert torch.isnan(x[4::7, 32:64]).all() and torch.isfinite(x[4::7, :32]).all()


@pytest.mark.parametrize("splits", ["", "1", "2", "5"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (1, 64, 72), (37, 520, 136), (128, 256, 256), (129, 264, 40), (3000, 256, 512),
                                   (20001, 72, 1000), (70000, 64, 96)])
def test_linear_weight_gradient(M, K, N, dtype, splits, monkeypatch):
    if splits:
        monkeypatch.setenv("CONV3D_LINEAR_WGRAD_SPLITS", splits)
    dt = DT[dtype]
    x, dy = rand((M, K), 16, 0, 1.0, dt), rand((M, N), 16, 1, 1.0, dt)
    dw, db = c3.linear_bwd_weight(x, dy)
    dw2, none = c3.linear_bwd_weight(x, dy, with_bias=False)
    dw3, db3 = c3.linear_bwd_weight(x, dy)
    sync_ok()
    rdw, rdb = dy.double().t() @ x.double(), dy.double().sum(0)
    ref.check(dw, rdw, ref.rounding(rdw, dt) * 1.01 + (M + 8) * 2.0 ** -23 * (dy.double().abs().t() @ x.double().abs()), "dw")
    ref.check(db, rdb, ref.rounding(rdb, dt) * 1.01 + (M + 8) * 2.0 ** -23 * dy.double().abs().sum(0), "dbias")
    assert none is None and torch.equal(dw2, dw) and torch.equal(dw3, dw) and torch.equal(db3, db)


@pytest.mark.parametrize("splits", ["1", "3"])
def test_linear_weight_gradient_writes_nothing_outside(splits, monkeypatch):
    monkeypatch.setenv("CONV3D_LINEAR_WGRAD_SPLITS", splits)
    M, K, N = 5000, 136, 264
    x, dy = rand((M, K), 18, 0), rand((M, N), 18, 1)
    dw, dw_ok = guarded(N * K, torch.bfloat16)
    db, db_ok = guarded(N, torch.bfloat16)
    need = c3.linear_bwd_weight_workspace_bytes(M, K, N)
    ws, ws_ok = guarded(max(need, 256), torch.uint8)
    ws.fill_(0xFF)                                         # NaN in every place that is read before it is written
    assert c3.linear_bwd_weight_ptr(x.data_ptr(), dy.data_ptr(), dw.data_ptr(), db.data_ptr(), M, K, N, c3.BF16,
                                    ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == c3.Status.OK
    sync_ok()
    want = c3.linear_bwd_weight(x, dy)
    assert torch.equal(dw.view(N, K), want[0]) and torch.equal(db, want[1])
    for ok in (dw_ok, db_ok, ws_ok):
        ok()


def test_offsets_beyond_32_bits(monkeypatch):
    """Rows whose byte and element offsets pass 2^32: the last rows agree with the same rows alone (through the same
    kernel: the two sum in different orders)."""
    monkeypatch.setenv("CONV3D_LINEAR", "256")
    rows, C = (1 << 32) // 2048 + 300, 2048
    x = torch.zeros((rows, C), dtype=torch.bfloat16, device="cuda")
    tail = rand((300, C), 17, 0)
    x[-300:] = tail
    a = c3.act8_pack(x)
    want = c3.act8_pack(tail)
    assert torch.equal(a.codes[-300:], want.codes) and torch.equal(a.exponents[-300:], want.exponents)
    y = c3.act8_unpack(a, x.dtype, act=c3.ACT_SILU)
    assert torch.equal(y[-300:], c3.act8_unpack(want, x.dtype, act=c3.ACT_SILU))
    c3.layernorm(x, y=y)
    assert torch.equal(y[-300:], c3.layernorm(tail))
    w = rand((64, C), 17, 1, C ** -0.5)
    assert torch.equal(c3.linear(x, w)[-300:], c3.linear(x[-812:].contiguous(), w)[-300:])
    back = rand((300, 64), 17, 2)
    dy = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    dy[-300:] = back
    c3.linear_bwd_data(dy, w, a, c3.ACT_GELU, dx=y)
    assert torch.equal(y[-300:], c3.linear_bwd_data(dy[-812:].contiguous(), w,
                                                   c3.Act8(a.codes[-812:].contiguous(), a.exponents[-812:].contiguous(), C),
                                                   c3.ACT_GELU)[-300:])
    sync_ok()
