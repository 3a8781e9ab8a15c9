"""What is measured of the channel-wise operators beside the convolutions: layer norm over the channels of
each pixel (forward and backward), 8-bit activation checkpoints (written, read back, and used in the backward
pass), the channel product (bias, activation and residual in its epilogue; its gradients) and the backward pass
of the channel MLP block that is made of them.

Activations are [rows, C], one row a pixel (or token) with its channels innermost, as the decoder layers hold
them.  An 8-bit checkpoint holds blocks of 32 channels: int8 codes [rows, 32 * ceil(C / 32)] and one exponent
byte per block [rows, ceil(C / 32)]; a code k under exponent byte b stands for k * 2^(b - 133).

``own`` false: the plain form, elementary torch operations in fp32, rounded once at the end.  ``own`` true: the
calls a user makes of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = {"none": 0, "silu": 1, "gelu": 2}
EPS = 1e-6
GELU_A = math.sqrt(2.0 / math.pi)
GELU_B = 0.044715


def listed():
    return [
        # one pixel / one token in front of a single-row product: call latency
        dict(name="ln_one_row", op="layernorm", rows=1, C=512, dtype="bf16"),
        # the 256-channel 9x128x128 decoder activation, with the statistics that training keeps
        dict(name="ln_9x128x128x256", op="layernorm", rows=147456, C=256, dtype="bf16"),
        # a ragged row count and a channel count that fills no whole block of 32, fp16, gradients from x itself
        dict(name="ln_bwd_ragged", op="layernorm_bwd", rows=16381, C=520, dtype="f16", ckpt=False, dres=False),
        # the 512-channel 17x64x96 mid-block, gradients from its 8-bit checkpoint plus the skip branch's gradient
        dict(name="ln_bwd8_17x64x96x512", op="layernorm_bwd", rows=104448, C=512, dtype="bf16", ckpt=True, dres=True),
        # an activation kept for the backward pass in 8 bits and read back
        dict(name="act8_9x128x128x256", op="act8", rows=147456, C=256, dtype="bf16"),
        # a small activation recomputed from its checkpoint (normalised value -> affine -> SiLU)
        dict(name="act8_recompute_small", op="act8_unpack", rows=1000, C=136, dtype="f16", act="silu", affine=True),
        # the activation's gradient at the hidden width of a 9x64x64 channel MLP
        dict(name="act8_bwd_9x64x64x2048", op="act8_bwd", rows=36864, C=2048, dtype="bf16", act="gelu"),
        # a single token / pixel through the expanding product
        dict(name="linear_one_row", op="linear", rows=1, K=512, N=2048, dtype="bf16", act="silu", residual=False, ckpt=False),
        # a few rows, sizes that fill no tile
        dict(name="linear_61_rows", op="linear", rows=61, K=1024, N=1000, dtype="f16", act="gelu", residual=True, ckpt=False),
        # the expanding product of a training step on 9x64x64 pixels; its pre-activation goes to an 8-bit checkpoint
        dict(name="linear_9x64x64", op="linear", rows=36864, K=512, N=2048, dtype="bf16", act="gelu", residual=False, ckpt=True),
        # the contracting product's input gradient times the activation's derivative from the checkpoint
        dict(name="linear_bwd_9x64x64", op="linear_bwd", rows=36864, K=2048, N=512, dtype="bf16", act="gelu", ckpt=True),
        # the whole backward pass of a channel MLP block on the 17x64x96 mid-block
        dict(name="mlp_bwd_17x64x96", op="mlp_bwd", rows=104448, C=512, hidden=2048, dtype="bf16", act="gelu"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, step * int(round(v / step))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_bwd", "act8", "act8_unpack", "act8_bwd", "linear", "linear", "linear_bwd",
                     "mlp_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("linear", "linear_bwd", "mlp_bwd"):
        rows, K, N = _log_int(rng, 1, 104448), _log_int(rng, 64, 2048, 8), _log_int(rng, 64, 2048, 8)
        rows = max(1, min(rows, int(104448 * 512 * 2048 / (K * N))))
        act = rng.choice(["none", "silu", "gelu"])
        if op == "linear":
            return dict(op=op, rows=rows, K=K, N=N, dtype=dtype, act=act, residual=rng.random() < 0.5,
                        ckpt=rng.random() < 0.5)
        if op == "linear_bwd":
            return dict(op=op, rows=rows, K=K, N=N, dtype=dtype, act=act, ckpt=act != "none")
        return dict(op=op, rows=rows, C=K, hidden=N, dtype=dtype, act=rng.choice(["silu", "gelu"]))
    rows, C = _log_int(rng, 1, 147456), _log_int(rng, 64, 2048, 8)
    rows = max(1, min(rows, int(104448 * 512 / C)))
    case = dict(op=op, rows=rows, C=C, dtype=dtype)
    if op == "layernorm_bwd":
        case.update(ckpt=rng.random() < 0.5, dres=rng.random() < 0.5)
    if op == "act8_unpack":
        case.update(act=rng.choice(["none", "silu", "gelu"]), affine=rng.random() < 0.5)
    if op == "act8_bwd":
        case.update(act=rng.choice(["silu", "gelu"]))
    return case


# ---------------------------------------------------------------- inputs


def _randn(gen, shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def _blocks(v):
    """[rows, C] fp32 -> [rows, blocks, 32], zeros behind the last channel."""
    rows, C = v.shape
    nb = -(-C // 32)
    if nb * 32 != C:
        v = torch.nn.functional.pad(v, (0, nb * 32 - C))
    return v.view(rows, nb, 32)


def _exponent_bytes(blocks):
    """The biased exponent of each block's largest magnitude, at least 7: uint8 [rows, blocks]."""
    e = torch.frexp(blocks.abs().amax(-1)).exponent + 126
    return e.clamp(7, 254).to(torch.uint8)


def _step(scales):
    # 2^(b - 133), exact: fp32 holds 2^n as the exponent field n + 127
    return ((scales.to(torch.int32) - 6) << 23).view(torch.float32)


def _codes(v):
    """(codes, exponent bytes) of a [rows, C] fp32 tensor."""
    b = _blocks(v)
    s = _exponent_bytes(b)
    q = torch.round(b / _step(s)[..., None]).clamp(-127, 127).to(torch.int8)
    return q.view(v.shape[0], -1), s


def _make_checkpoint(gen, rows, C, scale=1.0):
    """A checkpoint as a forward pass would have left it."""
    return _codes(torch.randn((rows, C), generator=gen, device="cuda") * scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    s["dt"] = dt
    rows, op = case["rows"], case["op"]

    def params(C):
        return _randn(gen, (C,), dt, 0.2, 1.0), _randn(gen, (C,), dt, 0.2)

    if op == "layernorm":
        # activations off centre: the statistics matter
        s["x"] = _randn(gen, (rows, case["C"]), dt, 1.5, 0.5)
        s["gamma"], s["beta"] = params(case["C"])
    elif op == "layernorm_bwd":
        C = case["C"]
        s["gamma"], _ = params(C)
        s["dy"] = _randn(gen, (rows, C), dt)
        s["dskip"] = _randn(gen, (rows, C), dt) if case["dres"] else None
        if case["ckpt"]:
            s["q"], s["scales"] = _make_checkpoint(gen, rows, C)
            s["rstd"] = torch.rand((rows,), generator=gen, device="cuda") + 0.5
        else:
            s["x"] = _randn(gen, (rows, C), dt, 1.5, 0.5)
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = (xf.var(-1, correction=0) + EPS).rsqrt()
    elif op == "act8":
        s["x"] = _randn(gen, (rows, case["C"]), dt, 1.5, 0.5)
    elif op == "act8_unpack":
        s["q"], s["scales"] = _make_checkpoint(gen, rows, case["C"])
        if case["affine"]:
            s["gamma"], s["beta"] = params(case["C"])
        else:
            s["gamma"] = s["beta"] = None
    elif op == "act8_bwd":
        s["q"], s["scales"] = _make_checkpoint(gen, rows, case["C"], 1.5)
        s["dy"] = _randn(gen, (rows, case["C"]), dt)
    elif op == "linear":
        K, N = case["K"], case["N"]
        s["x"] = _randn(gen, (rows, K), dt)
        s["w"] = _randn(gen, (N, K), dt, K ** -0.5)
        s["bias"] = _randn(gen, (N,), dt, 0.1)
        s["skip"] = _randn(gen, (rows, N), dt) if case["residual"] else None
    elif op == "linear_bwd":
        K, N = case["K"], case["N"]
        s["dy"] = _randn(gen, (rows, N), dt)
        s["w"] = _randn(gen, (N, K), dt, K ** -0.5)
        if case["ckpt"]:
            s["q"], s["scales"] = _make_checkpoint(gen, rows, K, 1.5)
    else:
        C, H = case["C"], case["hidden"]
        s["dy"] = _randn(gen, (rows, C), dt)
        s["gamma"], s["beta"] = params(C)
        s["w1"] = _randn(gen, (H, C), dt, C ** -0.5)
        s["w2"] = _randn(gen, (C, H), dt, H ** -0.5)
        s["q"], s["scales"] = _make_checkpoint(gen, rows, C)
        s["rstd"] = torch.rand((rows,), generator=gen, device="cuda") + 0.5
        s["pre_q"], s["pre_scales"] = _make_checkpoint(gen, rows, H)
    return s


# ---------------------------------------------------------------- the plain form


def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(GELU_A * (v + GELU_B * v * v * v)))
    return v


def _dact(v, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-v))
        return sg * (1.0 + v * (1.0 - sg))
    if act == "gelu":
        t = torch.tanh(GELU_A * (v + GELU_B * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * (GELU_A * (1.0 + 3.0 * GELU_B * v * v))
    return torch.ones_like(v)


def _values(q, scales, C):
    rows = q.shape[0]
    return (q.view(rows, -1, 32).float() * _step(scales)[..., None]).view(rows, -1)[:, :C]


def _norm_bwd(dy, xhat, rstd, gamma):
    """(dx, dgamma, dbeta) of y = xhat * gamma + beta, fp32."""
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _plain(s):
    op, dt = s["op"], s["dt"]
    if op == "layernorm":
        x = s["x"].float()
        mean = x.mean(-1)
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(-1) + EPS)
        return (d * rstd[:, None] * s["gamma"].float() + s["beta"].float()).to(dt), mean, rstd
    if op == "layernorm_bwd":
        if s["ckpt"]:
            xhat = _values(s["q"], s["scales"], s["C"])
        else:
            xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dx, dgamma, dbeta = _norm_bwd(s["dy"].float(), xhat, s["rstd"], s["gamma"].float())
        if s["dskip"] is not None:
            dx = dx + s["dskip"].float()
        return dx.to(dt), dgamma.to(dt), dbeta.to(dt)
    if op == "act8":
        q, scales = _codes(s["x"].float())
        return _values(q, scales, s["C"]).to(dt)
    if op == "act8_unpack":
        v = _values(s["q"], s["scales"], s["C"])
        if s["affine"]:
            v = v * s["gamma"].float() + s["beta"].float()
        return _act(v, s["act"]).to(dt)
    if op == "act8_bwd":
        return (s["dy"].float() * _dact(_values(s["q"], s["scales"], s["C"]), s["act"])).to(dt)
    if op == "linear":
        pre = s["x"].float() @ s["w"].float().t() + s["bias"].float()
        y = _act(pre, s["act"])
        if s["skip"] is not None:
            y = y + s["skip"].float()
        if not s["ckpt"]:
            return y.to(dt)
        q, scales = _codes(pre)
        return y.to(dt), _values(q, scales, s["N"]).to(dt)
    if op == "linear_bwd":
        dx = s["dy"].float() @ s["w"].float()
        if s["ckpt"]:
            dx = dx * _dact(_values(s["q"], s["scales"], s["K"]), s["act"])
        return dx.to(dt)
    # mlp_bwd: y = x + act(norm(x) w1^T + b1) w2^T + b2
    dy, w1, w2 = s["dy"].float(), s["w1"].float(), s["w2"].float()
    pre = _values(s["pre_q"], s["pre_scales"], s["hidden"])
    dw2 = dy.t() @ _act(pre, s["act"])
    dpre = (dy @ w2) * _dact(pre, s["act"])
    xhat = _values(s["q"], s["scales"], s["C"])
    dw1 = dpre.t() @ (xhat * s["gamma"].float() + s["beta"].float())
    dx, dgamma, dbeta = _norm_bwd(dpre @ w1, xhat, s["rstd"], s["gamma"].float())
    grads = (dx + dy, dgamma, dbeta, dw1, dpre.sum(0), dw2, dy.sum(0))
    return tuple(g.to(dt) for g in grads)


def _own(s):
    import video_vae_convolution_implicit_b200 as c3
    op, dt = s["op"], s["dt"]
    act = ACTS[s.get("act", "none")]
    if op == "layernorm":
        return c3.layernorm(s["x"], s["gamma"], s["beta"], EPS, with_stats=True)
    if op == "layernorm_bwd":
        if s["ckpt"]:
            saved, mean = c3.Act8(s["q"], s["scales"], s["C"]), None
        else:
            saved, mean = s["x"], s["mean"]
        return c3.layernorm_bwd(s["dy"], saved, s["rstd"], mean=mean, gamma=s["gamma"], dres=s["dskip"])
    if op == "act8":
        return c3.act8_unpack(c3.act8_pack(s["x"]), dt)
    if op == "act8_unpack":
        return c3.act8_unpack(c3.Act8(s["q"], s["scales"], s["C"]), dt, s["gamma"], s["beta"], act)
    if op == "act8_bwd":
        return c3.act8_bwd(s["dy"], c3.Act8(s["q"], s["scales"], s["C"]), act)
    if op == "linear":
        if not s["ckpt"]:
            return c3.linear(s["x"], s["w"], s["bias"], s["skip"], act)
        y, pre = c3.linear(s["x"], s["w"], s["bias"], s["skip"], act, checkpoint8=True)
        return y, c3.act8_unpack(pre, dt)
    if op == "linear_bwd":
        pre = c3.Act8(s["q"], s["scales"], s["K"]) if s["ckpt"] else None
        return c3.linear_bwd_data(s["dy"], s["w"], pre, act)
    saved = c3.ChannelMlpSaved(c3.Act8(s["q"], s["scales"], s["C"]), s["rstd"],
                               c3.Act8(s["pre_q"], s["pre_scales"], s["hidden"]))
    return c3.channel_mlp_bwd(s["dy"], saved, s["gamma"], s["beta"], s["w1"], s["w2"], act)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """From the definitions, in fp64: layer norm by its moments, the codes by the blocks' exponents, the activations
    and their derivatives through the sigmoid (gelu(v) = v * sigmoid(2 u(v)))."""
    s = prepare(case, seed)
    op = case["op"]
    f = lambda name: s[name].to(torch.float64)  # noqa: E731

    def power2(n):
        return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)

    def decode(q, scales, C):
        steps = power2(scales.to(torch.int64) - 133)
        return (q.to(torch.float64) * steps.repeat_interleave(32, dim=1))[:, :C]

    def through_codes(v):
        rows, C = v.shape
        pad = torch.zeros((rows, -C % 32), dtype=torch.float64, device=v.device)
        b = torch.cat([v, pad], 1).reshape(rows, -1, 32)
        top = b.abs().max(dim=-1).values.clamp_min(2.0 ** -120)
        # (the factor keeps an exact power of two from landing just under its own exponent)
        step = power2(torch.floor(torch.log2(top * (1.0 + 2.0 ** -40))) - 6.0).unsqueeze(-1)
        k = torch.minimum(torch.round((b / step).abs()), torch.full_like(b, 127.0)) * torch.sign(b)
        return (k * step).reshape(rows, -1)[:, :C]

    def act(v, order):
        name = case.get("act", "none")
        if name == "none":
            return v if order == 0 else torch.ones_like(v)
        if name == "silu":
            arg, darg = v, torch.ones_like(v)
        else:
            arg = 2.0 * GELU_A * (v + GELU_B * v ** 3)
            darg = 2.0 * GELU_A * (1.0 + 3.0 * GELU_B * v ** 2)
        sg = torch.sigmoid(arg)
        return v * sg if order == 0 else sg + v * sg * (1.0 - sg) * darg

    def norm_grads(dn, xhat, rstd, gamma):
        C = xhat.shape[1]
        g = dn * gamma
        along = (g * xhat).sum(1, keepdim=True) / C
        dx = (g - g.sum(1, keepdim=True) / C - xhat * along) * rstd.unsqueeze(1)
        return dx, torch.einsum("rc,rc->c", dn, xhat), dn.sum(0)

    if op == "layernorm":
        x = f("x")
        mean = x.sum(1) / x.shape[1]
        var = ((x - mean.unsqueeze(1)) ** 2).sum(1) / x.shape[1]
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(f("beta"), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), f("gamma"))
        return y, mean, rstd
    if op == "layernorm_bwd":
        if case["ckpt"]:
            xhat = decode(s["q"], s["scales"], case["C"])
        else:
            xhat = (f("x") - f("mean").unsqueeze(1)) * f("rstd").unsqueeze(1)
        dx, dgamma, dbeta = norm_grads(f("dy"), xhat, f("rstd"), f("gamma"))
        return (dx + f("dskip") if case["dres"] else dx), dgamma, dbeta
    if op == "act8":
        return through_codes(f("x"))
    if op == "act8_unpack":
        v = decode(s["q"], s["scales"], case["C"])
        return act(torch.addcmul(f("beta"), v, f("gamma")) if case["affine"] else v, 0)
    if op == "act8_bwd":
        return f("dy") * act(decode(s["q"], s["scales"], case["C"]), 1)
    if op == "linear":
        pre = torch.addmm(f("bias"), f("x"), f("w").t())
        y = act(pre, 0)
        if case["residual"]:
            y = y + f("skip")
        return (y, through_codes(pre)) if case["ckpt"] else y
    if op == "linear_bwd":
        dx = torch.mm(f("dy"), f("w"))
        return dx * act(decode(s["q"], s["scales"], case["K"]), 1) if case["ckpt"] else dx
    dy = f("dy")
    pre = decode(s["pre_q"], s["pre_scales"], case["hidden"])
    dw2 = torch.mm(dy.t(), act(pre, 0))
    dpre = torch.mm(dy, f("w2")) * act(pre, 1)
    xhat = decode(s["q"], s["scales"], case["C"])
    dw1 = torch.mm(dpre.t(), torch.addcmul(f("beta"), xhat, f("gamma")))
    dx, dgamma, dbeta = norm_grads(torch.mm(dpre, f("w1")), xhat, f("rstd"), f("gamma"))
    return dx + dy, dgamma, dbeta, dw1, dpre.sum(0), dw2, dy.sum(0)


# ---------------------------------------------------------------- the work that no implementation can do without


def _ckpt_bytes(rows, C):
    return rows * -(-C // 32) * 33


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("linear", "linear_bwd"):
        K, N = case["K"], case["N"]
        b = 2 * (rows * K + rows * N + N * K)
        if op == "linear":
            b += 2 * N + (2 * rows * N if case["residual"] else 0)
            b += _ckpt_bytes(rows, N) + 2 * rows * N if case["ckpt"] else 0   # codes out; their values out
            return {"bytes": b, "flops": 2 * rows * K * N}
        return {"bytes": b + (_ckpt_bytes(rows, K) if case["ckpt"] else 0), "flops": 2 * rows * K * N}
    if op == "mlp_bwd":
        C, H = case["C"], case["hidden"]
        b = 2 * 2 * rows * C + _ckpt_bytes(rows, C) + _ckpt_bytes(rows, H) + 4 * rows
        b += 2 * 4 * C * H + 2 * (2 * C + 2 * C + H + C)
        return {"bytes": b, "flops": 8 * rows * C * H}
    C = case["C"]
    n = rows * C
    if op == "layernorm":
        return {"bytes": 4 * n + 8 * rows + 4 * C, "flops": 8 * n}
    if op == "layernorm_bwd":
        b = 4 * n + (_ckpt_bytes(rows, C) + 4 * rows if case["ckpt"] else 2 * n + 8 * rows)
        return {"bytes": b + (2 * n if case["dres"] else 0) + 6 * C, "flops": 12 * n}
    if op == "act8":
        return {"bytes": 4 * n + _ckpt_bytes(rows, C), "flops": 6 * n}
    if op == "act8_unpack":
        return {"bytes": 2 * n + _ckpt_bytes(rows, C) + (4 * C if case["affine"] else 0), "flops": 8 * n}
    return {"bytes": 4 * n + _ckpt_bytes(rows, C), "flops": 12 * n}
