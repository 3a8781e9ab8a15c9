"""Relative accuracy of the activations and their derivatives, out to the smallest results.

silu(v) = v s, gelu(v) = v s with s = 1 / (1 + 2^w), w = -log2(e) v or -2 log2(e) u(v).
Counted in units of 2^-24: w takes four roundings (its constants, v^2, the fused sum, the
product), at most 4 |w|, which move 2^w by ln 2 times that, 2.8 |w|; 2^w itself is off by
at most 4 (2^-22), the sum 1, the reciprocal 2 (2^-23), the product with v 1.  Together
3 |w| + 12.  The derivative is s + c s (1 - s) = s (1 + c 2^w s), c = v or 2 v u'(v), whose
second term has the error of s (2.8 |w| + 7) twice, of 2^w and of c (4), and three
roundings: 9 |w| + 24 of s (1 + |c| (1 - s)).  s below 2^-126 may come out as 0.  Then one
rounding to the type.
"""
import math

import pytest
import torch

import channel_ref as ref
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
ACTS = [c3.ACT_SILU, c3.ACT_GELU]
UNIT = 2.0 ** -24


def parts(v, kind):
    """(s, 1 - s, |w|, c) in fp64"""
    arg = v if kind == c3.ACT_SILU else 2 * ref.A * (v + ref.B * v ** 3)
    c = v if kind == c3.ACT_SILU else v * 2 * ref.A * (1 + 3 * ref.B * v ** 2)
    return torch.sigmoid(arg), torch.sigmoid(-arg), (arg.abs() / math.log(2)).clamp(max=130.0), c


def value_and_bound(v, kind, dtype):
    s, _, w, _ = parts(v, kind)
    want = v * s
    off = want.abs() * (3 * w + 12) * UNIT + v.abs() * torch.where(s < 2.0 ** -125, s, 0.0)
    return want, off + ref.rounding(want.abs() + off, dtype)


def slope_and_bound(v, kind, dtype):
    s, r, w, c = parts(v, kind)
    want = s * (1 + c * r)
    size = s * (1 + c.abs() * r)
    off = size * (9 * w + 24) * UNIT + torch.where(s < 2.0 ** -125, size, 0.0)
    return want, off + ref.rounding(want.abs() + off, dtype)


def every_value(dtype):
    """All finite values of the type whose magnitude is at most 2^60."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).cuda()
    return v[(v.double().abs() <= 2.0 ** 60).nonzero().flatten()]


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kernel,C", [("1", 64), ("128", 128), ("2", 2048)], ids=["few rows", "pair", "dot"])
def test_product_with_the_identity(kernel, C, dtype, kind, monkeypatch):
    """y = act(x I): x is the pre-activation exactly, in each of the product's kernels."""
    monkeypatch.setenv("CONV3D_LINEAR", kernel)
    v = every_value(dtype)
    v = v[:v.numel() // C * C].view(-1, C)
    eye = torch.eye(C, dtype=dtype, device="cuda")
    step = 4 if kernel == "2" else v.shape[0]
    y = torch.cat([c3.linear(v[i:i + step], eye, act=kind) for i in range(0, v.shape[0], step)])
    assert c3.poll_status() == c3.Status.OK
    want, bound = value_and_bound(v.double(), kind, dtype)
    ref.check(y, want, bound, f"act {kind}")


def checkpoint_of(rows, C):
    """Random codes under steps from 2^-33 to 2^7 (|v| up to 16256)."""
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(-127, 128, (rows, C), generator=g).to(torch.int8)
    exps = torch.randint(100, 141, (rows, C // 32), generator=g)
    exps[:, ::2] = torch.randint(126, 133, (rows, C // 64), generator=g)   # most |v| from 1 to 32
    return c3.Act8(codes.cuda(), exps.to(torch.uint8).cuda(), C)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_checkpoint_reads(dtype, kind):
    a = checkpoint_of(512, 256)
    v = ref.decode(a)
    ref.check(c3.act8_unpack(a, dtype, act=kind), *value_and_bound(v, kind, dtype), "unpack")
    dx = c3.act8_bwd(torch.ones(512, 256, dtype=dtype, device="cuda"), a, kind)
    ref.check(dx, *slope_and_bound(v, kind, dtype), "act8_bwd")
    assert c3.poll_status() == c3.Status.OK


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kernel", ["1", "128", "256"])
def test_gradient_with_a_product_of_one(kernel, dtype, kind, monkeypatch):
    """dx = (dy w) act'(v) with dy w = 1, and the recomputed activation beside it."""
    monkeypatch.setenv("CONV3D_LINEAR", kernel)
    rows, K, N = 512, 256, 64
    a = checkpoint_of(rows, K)
    dy = torch.zeros(rows, N, dtype=dtype, device="cuda")
    w = torch.zeros(N, K, dtype=dtype, device="cuda")
    dy[:, 0], w[0] = 1, 1
    v = ref.decode(a)
    alone = c3.linear_bwd_data(dy, w, a, kind)
    dx, x = c3.linear_bwd_data(dy, w, a, kind, with_x=True)
    assert c3.poll_status() == c3.Status.OK
    ref.check(alone, *slope_and_bound(v, kind, dtype), "act'")
    ref.check(dx, *slope_and_bound(v, kind, dtype), "act' beside x")
    assert torch.equal(x.view(torch.int16), c3.act8_unpack(a, dtype, act=kind).view(torch.int16))
