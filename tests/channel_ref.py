"""Plain 64-bit forms of the channel-wise operators and the error bounds of their tests.

A rounding to the output type is off by at most half a step, finfo.eps / 2 of the value (2^-8 for bf16, 2^-11
for fp16), plus half the smallest subnormal step of fp16.  fp32 steps before it are counted at 2^-24 each.
The hardware tanh has a relative error of at most 2^-10.987 (CUDA's documented bound): TANH below.
"""
import math

import torch

TANH = 2.0 ** -10.98
A = math.sqrt(2.0 / math.pi)
B = 0.044715
NAMES = {0: "none", 1: "silu", 2: "gelu"}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(ref, dtype):
    """Bound of one rounding of ``ref`` to ``dtype``."""
    return ref.abs() * half_step(dtype) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def act(v, kind):
    if kind == 0:
        return v
    arg = v if kind == 1 else 2 * A * (v + B * v ** 3)
    return v * torch.sigmoid(arg)


def slope(v, kind):
    if kind == 0:
        return torch.ones_like(v)
    if kind == 1:
        s = torch.sigmoid(v)
        return s + v * s * (1 - s)
    s = torch.sigmoid(2 * A * (v + B * v ** 3))
    return s + v * s * (1 - s) * 2 * A * (1 + 3 * B * v ** 2)


def act_error(v, kind):
    """h + h tanh: |h| TANH, and a few fp32 roundings (the argument's included: its relative error of 2^-22
    moves the tanh by at most 2^-22 * max |u| sech^2(u) < 2^-22)."""
    return v.abs() * (0.5 * TANH + 2.0 ** -21) if kind else torch.zeros_like(v)


def codes(v):
    """(codes int64 [rows, 32 nb], exponents int64 [rows, nb]) of a finite fp64 [rows, C] matrix."""
    rows, C = v.shape
    nb = -(-C // 32)
    b = torch.zeros((rows, nb * 32), dtype=torch.float64, device=v.device)
    b[:, :C] = v
    b = b.view(rows, nb, 32)
    _, e = torch.frexp(b.abs().amax(-1))           # amax = m 2^e, m in [1/2, 1)
    byte = (e.long() - 1 + 127).clamp(min=7)
    byte[b.abs().amax(-1) == 0] = 7
    k = torch.round(torch.ldexp(b, (133 - byte)[..., None])).clamp(-127, 127)
    return k.long().view(rows, -1), byte


def decode(a):
    """fp64 [rows, C] values of an Act8 (NaN where the block is marked)."""
    C = a.channels
    q = a.codes.double().reshape(-1, a.codes.shape[-1])
    e = a.exponents.long().reshape(-1, a.exponents.shape[-1])
    step = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e - 133)
    step = torch.where(e == 255, torch.full_like(step, float("nan")), step)
    return (q * step.repeat_interleave(32, dim=1))[:, :C]


def step_of(a):
    """fp64 [rows, C] step of each value of an Act8."""
    e = a.exponents.long().reshape(-1, a.exponents.shape[-1])
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e - 133).repeat_interleave(32, dim=1)[:, :a.channels]


def checkpoint(v, device):
    """The Act8 of a finite fp64 [rows, C] matrix, made without the library's kernels."""
    import video_vae_convolution_implicit_b200 as c3
    k, e = codes(v)
    return c3.Act8(k.to(torch.int8).to(device), e.to(torch.uint8).to(device), v.shape[1])


def layernorm(x, gamma, beta, eps):
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = (d.square().mean(-1) + eps).rsqrt()
    xh = d * rstd[:, None]
    return xh * gamma + beta, mean, rstd, xh


def layernorm_bwd(dy, xh, rstd, gamma):
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def check(got, ref, bound, what):
    """Every element of ``got`` within ``bound`` of ``ref`` (both fp64)."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    worst = over.max().item()
    if worst > 0:
        i = over.argmax().item()
        raise AssertionError(f"{what}: element {i} is {got.flatten()[i].item()}, expected {ref.flatten()[i].item()} "
                             f"within {bound.expand_as(ref).flatten()[i].item()}")


def slope_error(v, kind):
    """slope = (1 + t)/2 + c (1 - t^2), t = tanh(arg) with relative error TANH; c = v/4 (silu), (v/2) u'(v) (gelu).
    dt <= |t| TANH moves the two terms by dt/2 and 2 |c t| dt, with 1 - t^2 in place of its limit far out: where
    |t| is within TANH of 1 the hardware's t may be 1, and the second term is then off by itself, c (1 - t^2)."""
    if kind == 0:
        return torch.zeros_like(v)
    if kind == 1:
        t, c = torch.tanh(v / 2), v / 4
    else:
        t, c = torch.tanh(A * (v + B * v ** 3)), v / 2 * A * (1 + 3 * B * v ** 2)
    return t.abs() * TANH * (0.5 + 2 * c.abs() * t.abs()) + 2.0 ** -20
