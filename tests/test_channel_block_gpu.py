"""The channel-wise operators as they are used together: the channel MLP block and its backward pass from 8-bit
checkpoints, the autograd wrappers against 64-bit formulas and differences, graphs, streams, launch counts and the
bounded waits of the product kernels."""
import threading
import time

import pytest
import torch

import channel_ref as ref
import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3
from test_channel_ops_gpu import check_linear, ckpt, product_case, rand, run_linear, sum_error, sync_ok

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
MLP_SHAPES = [(1, 64, 128), (37, 72, 200), (700, 256, 512), (3001, 512, 1024)]


def block(rows, C, H, seed, dt=BF):
    return dict(x=rand((rows, C), seed, 0, 1.0, dt, 0.3), gamma=rand((C,), seed, 1, 0.2, dt, 1.0),
                beta=rand((C,), seed, 2, 0.2, dt), w1=rand((H, C), seed, 3, C ** -0.5, dt), b1=rand((H,), seed, 4, 0.2, dt),
                w2=rand((C, H), seed, 5, H ** -0.5, dt), b2=rand((C,), seed, 6, 0.2, dt))


def formula(p, act, eps=1e-6):
    """fp64 forward pass: (y, n, xhat, rstd, pre, h)."""
    d = {k: v.double() for k, v in p.items()}
    n, _, rstd, xh = ref.layernorm(d["x"], d["gamma"], d["beta"], eps)
    pre = n @ d["w1"].t() + d["b1"]
    h = ref.act(pre, act)
    return d["x"] + h @ d["w2"].t() + d["b2"], n, xh, rstd, pre, h


@pytest.mark.parametrize("act", [c3.ACT_SILU, c3.ACT_GELU])
@pytest.mark.parametrize("rows,C,H", MLP_SHAPES)
def test_block_forward(rows, C, H, act):
    p = block(rows, C, H, 21)
    want, n, _, _, pre, h = formula(p, act)
    y = c3.channel_mlp(**p, act=act)
    y2, saved = c3.channel_mlp(**p, act=act, save=True)
    sync_ok()
    assert torch.equal(y, y2)
    w1, w2 = p["w1"].double().abs(), p["w2"].double().abs()
    n_off = n.abs() * 2.0 ** -8 * 1.01 + 2.0 ** -14            # n rounded to bf16 (and its fp32 operations)
    pre_off = n_off @ w1.t() + sum_error(n, p["w1"].double())
    h_off = 1.13 * pre_off + ref.act_error(pre, act) + h.abs() * 2.0 ** -8 * 1.01
    bound = h_off @ w2.t() + sum_error(h, p["w2"].double()) + ref.rounding(want, BF) * 1.01
    ref.check(y, want, bound, "y")
    assert saved.xhat.channels == C and saved.pre.channels == H and tuple(saved.rstd.shape) == (rows,)


def grad_bounds(p, dy, xh, rstd, pre, e_x, e_pre, act):
    """fp64 gradients of the block from (xh, rstd, pre) and bounds of the library's, whose checkpoints are off by
    e_x and e_pre at most: every 16-bit rounding (h, dpre, n, dn and the results) and fp32 sum is counted."""
    d = {k: v.double() for k, v in p.items()}
    dy = dy.double()
    u = 2.0 ** -8 * 1.01
    h, s = ref.act(pre, act), ref.slope(pre, act)
    h_off = 1.13 * e_pre + ref.act_error(pre, act) + u * h.abs()
    dw2, dw2_off = dy.t() @ h, dy.abs().t() @ h_off + (len(dy) + 8) * 2.0 ** -23 * (dy.abs().t() @ (h.abs() + h_off))
    dh = dy @ d["w2"]
    dh_off = sum_error(dy, d["w2"].t())
    s_off = 0.85 * e_pre + ref.slope_error(pre, act)           # |act''| < 0.85
    dpre = dh * s
    dpre_off = dh_off * (s.abs() + s_off) + dh.abs() * s_off
    dpre_off = dpre_off + u * (dpre.abs() + dpre_off)
    n = xh * d["gamma"] + d["beta"]
    n_off = d["gamma"].abs() * e_x + u * n.abs() + 2.0 ** -20
    big = dpre.abs() + dpre_off
    dw1 = dpre.t() @ n
    dw1_off = big.t() @ n_off + dpre_off.t() @ n.abs() + (len(dy) + 8) * 2.0 ** -23 * (big.t() @ (n.abs() + n_off))
    dn = dpre @ d["w1"]
    dn_off = dpre_off @ d["w1"].abs() + sum_error(big, d["w1"].t())
    dn_off = dn_off + u * (dn.abs() + dn_off)
    g, g_off = dn * d["gamma"], dn_off * d["gamma"].abs()
    c2, c2_off = (g * xh).mean(-1, keepdim=True), (g_off * (xh.abs() + e_x) + g.abs() * e_x).mean(-1, keepdim=True)
    dx, dgamma, dbeta = ref.layernorm_bwd(dn, xh, rstd, d["gamma"])
    dx_off = rstd[:, None] * (g_off + g_off.mean(-1, keepdim=True) + (xh.abs() + e_x) * c2_off + e_x * c2.abs() +
                              2.0 ** -16 * (g.abs() + g.abs().mean(-1, keepdim=True) + xh.abs() * c2.abs()))
    dgamma_off = (dn_off * (xh.abs() + e_x) + dn.abs() * e_x + 2.0 ** -15 * dn.abs() * xh.abs()).sum(0)
    dbeta_off = (dn_off + 2.0 ** -15 * dn.abs()).sum(0)
    sums = (len(dy) + 8) * 2.0 ** -23
    pairs = dict(dx=(dx + dy, dx_off), dgamma=(dgamma, dgamma_off), dbeta=(dbeta, dbeta_off), dw1=(dw1, dw1_off),
                 db1=(dpre.sum(0), (dpre_off + sums * big).sum(0)), dw2=(dw2, dw2_off),
                 db2=(dy.sum(0), sums * dy.abs().sum(0)))
    return {k: (v, off + ref.rounding(v.abs() + off, BF) * 1.01) for k, (v, off) in pairs.items()}


NAMES = ("dx", "dgamma", "dbeta", "dw1", "db1", "dw2", "db2")


@pytest.mark.parametrize("act", [c3.ACT_SILU, c3.ACT_GELU])
@pytest.mark.parametrize("rows,C,H", MLP_SHAPES)
def test_block_backward_from_given_checkpoints(rows, C, H, act):
    p = block(rows, C, H, 22)
    saved = c3.ChannelMlpSaved(ckpt(rows, C, 22), torch.rand((rows,), device="cuda") + 0.5, ckpt(rows, H, 23, 1.5))
    dy = rand((rows, C), 22, 7)
    got = c3.channel_mlp_bwd(dy, saved, p["gamma"], p["beta"], p["w1"], p["w2"], act)
    sync_ok()
    want = grad_bounds(p, dy, ref.decode(saved.xhat), saved.rstd.double(), ref.decode(saved.pre), 0.0, 0.0, act)
    for name, g in zip(NAMES, got):
        ref.check(g, want[name][0], want[name][1], name)


@pytest.mark.parametrize("rows,C,H", MLP_SHAPES)
def test_block_autograd_against_the_formula_and_differences(rows, C, H):
    act = c3.ACT_GELU
    p = {k: v.requires_grad_() for k, v in block(rows, C, H, 24).items()}
    dy = rand((rows, C), 24, 7)
    y = c3.channel_mlp_autograd(**p, act=act)
    y.backward(dy)
    sync_ok()
    q = {k: v.detach() for k, v in p.items()}
    _, n, xh, rstd, pre, _ = formula(q, act)
    # the kept checkpoints: half a step (a whole one where a value clamps) of 2^-6 of the block's largest
    # magnitude at most, plus the forward pass's own error in what is coded
    def coded(v, off):
        blocks = torch.nn.functional.pad(v.abs() + off, (0, -v.shape[1] % 32)).view(len(v), -1, 32).amax(-1)
        return off + (blocks * 2.0 ** -6).clamp_min(2.0 ** -126).repeat_interleave(32, 1)[:, :v.shape[1]]
    n_off = n.abs() * 2.0 ** -8 * 1.01 + 2.0 ** -14
    pre_off = n_off @ q["w1"].double().abs().t() + sum_error(n, q["w1"].double())
    want = grad_bounds(q, dy, xh, rstd, pre, coded(xh, xh.abs() * 2.0 ** -16 + 2.0 ** -16), coded(pre, pre_off), act)
    grads = [p[k].grad for k in ("x", "gamma", "beta", "w1", "b1", "w2", "b2")]
    for name, g in zip(NAMES, grads):
        ref.check(g, want[name][0], want[name][1] * 1.01, name)
    # differences of the 64-bit formula along a random direction of every input
    t = 2.0 ** -13
    step = {k: si.tensor(tuple(v.shape), 25, i, 1.0, torch.float32, "cuda").double() * t for i, (k, v) in enumerate(q.items())}
    ahead = formula({k: v.double() + step[k] for k, v in q.items()}, act)[0]
    behind = formula({k: v.double() - step[k] for k, v in q.items()}, act)[0]
    quotient = ((ahead - behind) * dy.double()).sum().item() / 2
    along = bound = 0.0
    for name, k, g in zip(NAMES, q, grads):
        along += (g.double() * step[k]).sum().item()
        bound += (want[name][1] * step[k].abs()).sum().item()
    # the quotient's own error is of third order in t: compared with the first order term of the bound it is small
    assert abs(along - quotient) <= 1.05 * bound, (along, quotient, bound)


@pytest.mark.parametrize("checkpoint8", [False, True])
def test_layernorm_autograd(checkpoint8):
    rows, C = 123, 264
    x, g, b = (rand((rows, C), 26, 0, 1.5, BF, 0.5).requires_grad_(), rand((C,), 26, 1, 0.2, BF, 1.0).requires_grad_(),
               rand((C,), 26, 2).requires_grad_())
    dy = rand((rows, C), 26, 3)
    c3.layernorm_autograd(x, g, b, 1e-6, checkpoint8).backward(dy)
    sync_ok()
    xd, gd = x.detach().double(), g.detach().double()
    _, _, rstd, xh = ref.layernorm(xd, gd, b.detach().double(), 1e-6)
    dx, dg, db = ref.layernorm_bwd(dy.double(), xh, rstd, gd)
    blocks = torch.nn.functional.pad(xh.abs(), (0, -C % 32)).view(rows, -1, 32).amax(-1) * 2.0 ** -6
    e = blocks.repeat_interleave(32, 1)[:, :C] if checkpoint8 else torch.zeros_like(xh)
    e = e + 2.0 ** -18 * (xh.abs() + xd.abs() * rstd[:, None])
    gy = (dy.double() * gd).abs()
    off = rstd[:, None] * ((xh.abs() + e) * (gy * e).mean(-1, keepdim=True) + e * (gy * xh.abs()).mean(-1, keepdim=True) +
                           2.0 ** -17 * (gy + gy.mean(-1, keepdim=True) + xh.abs() * (gy * xh.abs()).mean(-1, keepdim=True)))
    ref.check(x.grad, dx, off + ref.rounding(dx.abs() + off, BF) * 1.01, "dx")
    off = (dy.double().abs() * (e + 2.0 ** -16 * xh.abs())).sum(0)
    ref.check(g.grad, dg, off + ref.rounding(dg.abs() + off, BF) * 1.01, "dgamma")
    ref.check(b.grad, db, 2.0 ** -16 * dy.double().abs().sum(0) + ref.rounding(db, BF) * 1.01, "dbeta")


@pytest.mark.parametrize("act", [c3.ACT_NONE, c3.ACT_SILU, c3.ACT_GELU])
def test_linear_autograd(act):
    M, K, N = 210, 136, 264
    p = {k: v.requires_grad_() for k, v in product_case(M, K, N, BF, 27).items()}
    dy = rand((M, N), 27, 5)
    c3.linear_autograd(p["x"], p["w"].view(N, 1, 1, 1, K), p["bias"], p["residual"], act).backward(dy)
    sync_ok()
    x, w = p["x"].detach().double(), p["w"].detach().double()
    pre = x @ w.t() + p["bias"].detach().double()
    blocks = torch.nn.functional.pad(pre.abs(), (0, -N % 32)).view(M, -1, 32).amax(-1) * 2.0 ** -6
    e = sum_error(x, w) + (blocks.repeat_interleave(32, 1)[:, :N] if act else 0.0)
    d, s = dy.double(), ref.slope(pre, act)
    dpre = d * s
    off = d.abs() * (0.85 * e + ref.slope_error(pre, act)) if act else torch.zeros_like(d)
    off = off + (2.0 ** -8 * 1.01 * (dpre.abs() + off) if act else 0.0)
    big = dpre.abs() + off

    def close(got, want, o, what):
        ref.check(got, want, o + ref.rounding(want.abs() + o, BF) * 1.01, what)
    close(p["x"].grad, dpre @ w, off @ w.abs() + sum_error(big, w.t()), "dx")
    close(p["w"].grad, dpre.t() @ x, off.t() @ x.abs() + (M + 8) * 2.0 ** -23 * (big.t() @ x.abs()), "dw")
    close(p["bias"].grad, dpre.sum(0), (off + (M + 8) * 2.0 ** -23 * big).sum(0), "dbias")
    assert torch.equal(p["residual"].grad, dy)


def test_conv3d_autograd_keeps_its_input_in_8_bits():
    x, w = rand((1, 3, 10, 12, 64), 28, 0), rand((96, 3, 3, 3, 64), 28, 1, (27 * 64) ** -0.5)
    dy = rand((1, 3, 10, 12, 96), 28, 2)
    grads = []
    for checkpoint8 in (False, True):
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        c3.conv3d_autograd(a, b, checkpoint8=checkpoint8).backward(dy)
        grads.append((a.grad, b.grad))
    sync_ok()
    assert torch.equal(grads[0][0], grads[1][0])                   # dx does not read x
    back = c3.act8_unpack(c3.act8_pack(x), x.dtype)
    dw, _ = c3.conv3d_bwd_weight(back, dy, (3, 3, 3))
    sync_ok()
    # the same kernel on the values read back: fp32 sums whose order varies, rounded once
    ref.check(grads[1][1], dw.double(), 2.0 ** -7 * dw.double().abs() + 1e-3, "dw")


def test_block_in_a_graph_and_on_another_stream():
    rows, C, H = 300, 128, 256
    p = block(rows, C, H, 29)
    dy = rand((rows, C), 29, 7)

    def step():
        y, saved = c3.channel_mlp(**p, save=True)
        return (y, *c3.channel_mlp_bwd(dy, saved, p["gamma"], p["beta"], p["w1"], p["w2"]))
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()                                             # the current stream is the side stream
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert c3.poll_status() == c3.Status.OK
        for name, a, b, c in zip(("y", *NAMES), want, out, other):
            for got in (b, c):
                assert torch.equal(got, a), name


def test_two_streams_at_once():
    """Calls of every operator on two streams, overlapping: each as it is alone."""
    sizes = ((9000, 512, 1024), (8100, 256, 512))
    ps = [block(r, C, H, 30 + i) for i, (r, C, H) in enumerate(sizes)]
    ys = [rand((r, C), 32, i) for i, (r, C, _) in enumerate(sizes)]

    def step(p, dy):
        y, saved = c3.channel_mlp(**p, save=True)
        return (y, *c3.channel_mlp_bwd(dy, saved, p["gamma"], p["beta"], p["w1"], p["w2"]))
    alone = [step(p, dy) for p, dy in zip(ps, ys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    out = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[i].append(step(ps[i], ys[i]))
    torch.cuda.synchronize()
    assert c3.poll_status() == c3.Status.OK
    for i in range(2):
        for got in out[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, alone[i]))


def test_stream_argument_and_leading_extents():
    x = rand((2, 3, 4, 5, 64), 33, 0)
    w = rand((96, 1, 1, 1, 64), 33, 1, 0.125)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = c3.layernorm(x, stream=s)
    z = c3.linear(y, w, act=c3.ACT_SILU, stream=s)
    a = c3.act8_pack(z, stream=s.cuda_stream)
    s.synchronize()
    flat = c3.linear(c3.layernorm(x.view(-1, 64)), w.view(96, 64), act=c3.ACT_SILU)
    b = c3.act8_pack(flat)
    sync_ok()
    assert tuple(z.shape) == (2, 3, 4, 5, 96) and torch.equal(z.view(-1, 96), flat)
    assert tuple(a.codes.shape) == (2, 3, 4, 5, 96) and torch.equal(a.codes.view(-1, 96), b.codes)


def test_first_call_of_a_thread():
    """A thread without a CUDA context of its own (autograd's, a worker) makes a call whose first step
    on the device is a tensor map: the driver needs a context to encode it."""
    x, w = rand((64, 64), 38, 0), rand((64, 64), 38, 1, 0.125)
    clip, kernel = rand((1, 2, 8, 8, 64), 38, 2), rand((64, 1, 3, 3, 64), 38, 3, 0.04)
    calls = [lambda: c3.linear(x, w), lambda: c3.linear_bwd_data(x, w), lambda: c3.linear_bwd_weight(x, x)[0],
             lambda: c3.conv3d(clip, kernel)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    for call, expect in zip(calls, want):
        got = []

        def work():
            try:
                got.append(call())
            except Exception as e:   # noqa: BLE001 -- shown by the assertion below
                got.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert torch.is_tensor(got[0]), got[0]
        assert torch.equal(got[0], expect)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    c3.linear_autograd(a, b).backward(x)   # autograd's thread: the first call is the product
    assert torch.equal(a.grad, c3.linear_bwd_data(x, w))
    sync_ok()


def test_memory_of_a_call_on_a_given_stream_belongs_to_that_stream():
    """What a call allocates must not go to the current stream's next tensor when it is
    freed: the kernels that write or read it may still be waiting on theirs."""
    x, w = rand((64, 64), 35, 0), rand((64, 64), 35, 1, 0.125)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c3.linear(x, w, stream=s)   # the allocator's pools of both streams hold blocks
    torch.empty_like(x)
    for call in (lambda: c3.layernorm(x, stream=s), lambda: c3.linear(x, w, stream=s.cuda_stream),
                 lambda: c3.act8_unpack(c3.act8_pack(x, stream=s), BF, stream=s),
                 lambda: c3.linear_bwd_weight(x, x, stream=s)[0]):
        y = call()
        at = y.data_ptr()
        del y
        other = [torch.empty_like(x) for _ in range(4)]
        assert at not in [t.data_ptr() for t in other]
    for handle in (0, 1, 2):   # the default streams by CUDA's handles
        torch.cuda.synchronize()
        y = c3.linear(x, w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(y, c3.linear(x, w))
    sync_ok()


def test_refusals_on_the_gpu():
    x = rand((4, 64), 34, 0)
    with pytest.raises(TypeError):
        c3.layernorm(x.float())
    with pytest.raises(TypeError):
        c3.layernorm(x, torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        c3.layernorm(x.t())
    with pytest.raises(ValueError):
        c3.layernorm(x, torch.ones(32, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        c3.linear(x, rand((8, 32), 34, 1))
    with pytest.raises(ValueError):
        c3.linear(x, rand((8, 64), 34, 1).cpu())
    with pytest.raises(ValueError):
        c3.act8_bwd(x, ckpt(4, 32, 34), c3.ACT_SILU)
    with pytest.raises(ValueError):
        c3.layernorm_bwd(x, x, torch.ones(4, device="cuda"))
    with pytest.raises(c3.Conv3dError) as e:
        c3.layernorm(x[:, :60].contiguous())
    assert e.value.status == c3.Status.UNSUPPORTED and "multiple of 8" in str(e.value)
    with pytest.raises(c3.Conv3dError):
        c3.layernorm(x[:0])
    with pytest.raises(c3.Conv3dError):
        c3.linear(x, rand((64, 64), 34, 1), y=x)


def test_launch_counts():
    x, w = rand((300, 256), 35, 0), rand((512, 256), 35, 1)
    saved = c3.act8_pack(x)
    rstd = torch.ones(300, device="cuda")

    def count(fn):
        torch.cuda.synchronize()
        before = c3.kernel_launches()
        fn()
        return c3.kernel_launches() - before
    assert count(lambda: c3.layernorm(x, checkpoint8=True)) == 1
    assert count(lambda: c3.layernorm_bwd(x, saved, rstd)) == 2
    assert count(lambda: c3.layernorm_bwd(x, saved, rstd, with_params=False)) == 1
    assert count(lambda: c3.act8_unpack(saved, BF, act=c3.ACT_GELU)) == 1
    assert count(lambda: c3.linear(x, w, act=c3.ACT_GELU, checkpoint8=True)) == 1
    assert count(lambda: c3.linear(x[:1], w)) == 1
    assert count(lambda: c3.linear_bwd_data(rand((300, 512), 35, 2), w, saved, c3.ACT_GELU)) == 1
    sync_ok()


@pytest.fixture
def _disarm():
    yield
    c3.test_arm_stall(0)
    c3.poll_status()


STALLS = {"rows": {"CONV3D_LINEAR": "1", "CONV3D_LINEAR_SPLIT": "1"}, "rows split": {"CONV3D_LINEAR": "1", "CONV3D_LINEAR_SPLIT": "4"},
          "pair streamed": {"CONV3D_LINEAR": "256", "CONV3D_LINEAR_RESIDENT": "0"},
          "pair resident": {"CONV3D_LINEAR": "256", "CONV3D_LINEAR_RESIDENT": "1"}}


@pytest.mark.parametrize("variant", sorted(STALLS))
def test_product_kernels_time_out_and_recover(variant, monkeypatch, _disarm):
    """A pipeline stage that never fills: the bounded wait ends the kernel, the status says so, and the next call on
    the same context is correct."""
    for k, v in STALLS[variant].items():
        monkeypatch.setenv(k, v)
    p = product_case(700, 256, 264, BF, 36)
    sync_ok()
    c3.test_arm_stall(1, 50)
    t0 = time.perf_counter()
    run_linear(p, 2, True, True, True)
    status = c3.poll_status()
    assert status == c3.Status.TIMEOUT, c3.status_string(status)
    assert time.perf_counter() - t0 < 5.0
    y, a = run_linear(p, 2, True, True, True)
    sync_ok()
    check_linear(p, BF, 2, True, True, y, a)


@pytest.mark.parametrize("variant", sorted(STALLS))
def test_gradient_kernels_time_out_and_recover(variant, monkeypatch, _disarm):
    for k, v in STALLS[variant].items():
        monkeypatch.setenv(k, v)
    dy, w, pre = rand((700, 264), 39, 0), rand((264, 512), 39, 1, 0.05), ckpt(700, 512, 39)
    want = c3.linear_bwd_data(dy, w, pre, c3.ACT_GELU, with_x=True)
    sync_ok()
    c3.test_arm_stall(1, 50)
    t0 = time.perf_counter()
    c3.linear_bwd_data(dy, w, pre, c3.ACT_GELU, with_x=True)
    status = c3.poll_status()
    assert status == c3.Status.TIMEOUT, c3.status_string(status)
    assert time.perf_counter() - t0 < 5.0
    again = c3.linear_bwd_data(dy, w, pre, c3.ACT_GELU, with_x=True)
    sync_ok()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("splits", ["1", "2"])
def test_weight_gradient_kernel_times_out_and_recovers(splits, monkeypatch, _disarm):
    monkeypatch.setenv("CONV3D_LINEAR_WGRAD_SPLITS", splits)
    x, dy = rand((30000, 264), 38, 0), rand((30000, 520), 38, 1)
    want = c3.linear_bwd_weight(x, dy)
    sync_ok()
    c3.test_arm_stall(1, 50)
    t0 = time.perf_counter()
    c3.linear_bwd_weight(x, dy)
    assert c3.poll_status() == c3.Status.TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    again = c3.linear_bwd_weight(x, dy)
    sync_ok()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("M,K,N", [(300, 64, 512), (2000, 256, 264), (5000, 448, 520), (20000, 320, 1032)])
def test_resident_and_streamed_weight_agree(M, K, N, monkeypatch):
    """The same products in the same order: the same bits, however B reaches shared memory."""
    monkeypatch.setenv("CONV3D_LINEAR", "256")
    p = product_case(M, K, N, BF, 37)
    dy = rand((M, K), 37, 7)
    pre = ckpt(M, N, 37)
    out = []
    for resident in ("0", "1"):
        monkeypatch.setenv("CONV3D_LINEAR_RESIDENT", resident)
        y, a = run_linear(p, 2, True, True, True)
        dx = c3.linear_bwd_data(dy, rand((K, N), 37, 8, K ** -0.5), pre, c3.ACT_SILU)
        both = c3.linear_bwd_data(dy, rand((K, N), 37, 8, K ** -0.5), pre, c3.ACT_SILU, with_x=True)
        sync_ok()
        out.append((y, a.codes, a.exponents, dx, *both))
    check_linear(p, BF, 2, True, True, out[0][0], c3.Act8(out[0][1], out[0][2], N))
    assert all(torch.equal(a, b) for a, b in zip(*out))
