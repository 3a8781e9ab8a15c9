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
