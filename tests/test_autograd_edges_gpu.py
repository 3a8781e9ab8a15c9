"""Edges of the torch.autograd wrappers: what is kept where little is asked for,
second derivatives, and tensors that a call overwrites in place."""
import pytest
import torch

import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(shape, k, scale=1.0, dtype=BF):
    return si.tensor(shape, 91, k, scale, dtype, "cuda")


def _launches(call):
    before = c3.kernel_launches()
    out = call()
    return c3.kernel_launches() - before, out


def test_conv3d_keeps_no_checkpoint_that_nothing_reads():
    x, w, b = rand((1, 3, 12, 16, 64), 0), rand((64, 3, 3, 3, 64), 1, 0.025), rand((64,), 2)
    dy = rand((1, 3, 12, 16, 64), 3)
    plain, y = _launches(lambda: c3.conv3d(x, w, b))

    def run(needs, grad=True):
        leaves = [t.clone().requires_grad_(n) for t, n in zip((x, w, b), needs)]
        with torch.set_grad_enabled(grad):
            n, out = _launches(lambda: c3.conv3d_autograd(*leaves, checkpoint8=True))
        assert torch.equal(out, y)
        if grad and any(needs):
            out.backward(dy)
        return n - plain, [t.grad for t in leaves]

    packs, (dx, dw, db) = run((True, False, False))        # frozen weights
    assert packs == 0 and dw is None and db is None
    assert torch.equal(dx, c3.conv3d_bwd_data(dy, w, x.shape))
    assert run((False, False, False))[0] == 0
    assert run((True, True, True), grad=False)[0] == 0     # no graph is recorded
    for needs in ((True, True, False), (False, True, True), (False, False, True)):
        packs, grads = run(needs)
        assert packs == 1 and [g is not None for g in grads] == list(needs)
    # the bias's gradient reads dy alone
    _, db = c3.conv3d_bwd_weight(x, dy, (3, 3, 3))
    torch.testing.assert_close(grads[2].float(), db.float(), rtol=2.0 ** -7, atol=0)
    assert c3.poll_status() == c3.Status.OK


def _calls():
    x, w, b = rand((64, 64), 10), rand((64, 64), 11, 0.125), rand((64,), 12)
    clip, kernel = rand((1, 2, 8, 8, 64), 13), rand((64, 3, 3, 3, 64), 14, 0.025)
    return {
        "layernorm": (c3.layernorm_autograd, (x, b, b)),
        "layernorm checkpoint": (lambda *t: c3.layernorm_autograd(*t, checkpoint8=True), (x, b, b)),
        "linear": (c3.linear_autograd, (x, w, b)),
        "linear gelu": (lambda *t: c3.linear_autograd(*t, act=c3.ACT_GELU), (x, w, b)),
        "mlp": (c3.channel_mlp_autograd, (x, b, b, w, b, w, b)),
        "conv3d": (c3.conv3d_autograd, (clip, kernel, b)),
    }


@pytest.mark.parametrize("name", ["layernorm", "layernorm checkpoint", "linear", "linear gelu", "mlp", "conv3d"])
def test_second_derivatives_are_refused(name):
    """The gradients of these calls carry no graph: a loss with a gradient in it would
    lose that term without a word."""
    call, tensors = _calls()[name]
    leaves = [t.clone().requires_grad_() for t in tensors]
    y = call(*leaves)
    dy = rand(tuple(y.shape), 15)
    plain = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    grads = torch.autograd.grad(y, leaves, dy, create_graph=True)
    for g, p in zip(grads, plain):
        # (the convolution's weight gradient adds its parts in any order)
        torch.testing.assert_close(g, p, rtol=0 if name != "conv3d" else 2.0 ** -7, atol=0 if name != "conv3d" else 1e-3)
    for g in grads:
        with pytest.raises(RuntimeError, match="differentiable once"):   # whatever dy depends on
            g.float().square().sum().backward(retain_graph=True)
    assert c3.poll_status() == c3.Status.OK


def _in_place_calls():
    """name: (a tensor that a call will overwrite, the call)"""
    x, w, b = rand((64, 64), 20), rand((64, 64), 21, 0.125), rand((64,), 22)
    clip, kernel = rand((1, 2, 8, 8, 64), 23), rand((64, 1, 1, 1, 64), 24, 0.125)
    a8 = c3.act8_pack(x)
    _, mean, rstd = c3.layernorm(x, with_stats=True)
    stats = c3.groupnorm_stats(clip, 8)
    flat = dict(pad=(0, 0, 0), tpad=c3.TPAD_ZERO)
    return {
        "layernorm": (x, lambda t: c3.layernorm(t, y=t)),
        "layernorm_bwd": (x, lambda t: c3.layernorm_bwd(t, x, rstd, mean, dx=t)),
        "act8_unpack": (x, lambda t: c3.act8_unpack(a8, BF, y=t)),
        "act8_bwd": (x, lambda t: c3.act8_bwd(t, a8, c3.ACT_SILU, dx=t)),
        "linear": (x, lambda t: c3.linear(x, w, b, t, y=t)),
        "linear_bwd_data": (x, lambda t: c3.linear_bwd_data(x, w, dx=t)),
        "conv3d_fwd": (clip, lambda t: c3.conv3d_fwd(clip, kernel, b, None, t, **flat)),
        "conv3d_gn": (clip, lambda t: c3.conv3d_gn(clip, None, None, None, kernel, y=t, **flat)),
        "groupnorm_silu": (clip, lambda t: c3.groupnorm_silu(t, stats, y=t)),
        "groupnorm_stats": (stats, lambda t: c3.groupnorm_stats(clip, 8, stats=t)),
        "conv3d_bwd_data": (clip, lambda t: c3.conv3d_bwd_data(clip, kernel, clip.shape, dx=t, **flat)),
    }


@pytest.mark.parametrize("name", [
    "layernorm", "layernorm_bwd", "act8_unpack", "act8_bwd", "linear", "linear_bwd_data", "conv3d_fwd", "conv3d_gn",
    "groupnorm_silu", "groupnorm_stats", "conv3d_bwd_data"])
def test_autograd_notices_an_overwritten_tensor(name):
    tensor, call = _in_place_calls()[name]
    t = tensor.clone()
    leaf = torch.ones_like(t).requires_grad_()
    z = (leaf * t).sum()              # saves t
    call(t)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.inference_mode():      # tensors without a version
        call(tensor.clone())
    assert c3.poll_status() == c3.Status.OK
