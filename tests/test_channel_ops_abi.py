"""The channel-wise operators' argument checks: every refusal happens on the host, before any CUDA call (fake,
never dereferenced addresses), and the Python layer's own checks."""
import pytest
import torch

import video_vae_convolution_implicit_b200 as c3
from video_vae_convolution_implicit_b200 import Status

P = [0x100000000 * (i + 1) for i in range(12)]    # widely separated fake device addresses
X, G, B, Y, MEAN, RSTD, Q, E, DY, DX, W, R = P


def ln_fwd(x=X, gamma=G, beta=B, y=Y, mean=None, rstd=None, q=None, e=None, rows=4, C=64, eps=1e-6, dt=c3.BF16):
    return c3.layernorm_fwd_ptr(x, gamma, beta, y, mean, rstd, q, e, rows, C, eps, dt, None)


def ln_bwd(dy=DY, x=X, mean=MEAN, q=None, e=None, rstd=RSTD, gamma=G, dres=None, dx=DX, dg=W, db=R, rows=4, C=64,
           dt=c3.BF16, ws=B, ws_bytes=1 << 20):
    return c3.layernorm_bwd_ptr(dy, x, mean, q, e, rstd, gamma, dres, dx, dg, db, rows, C, dt, ws, ws_bytes, None)


def pack(x=X, q=Q, e=E, rows=4, C=64, dt=c3.BF16):
    return c3.act8_pack_ptr(x, q, e, rows, C, dt, None)


def unpack(q=Q, e=E, gamma=None, beta=None, act=0, y=Y, rows=4, C=64, dt=c3.BF16):
    return c3.act8_unpack_ptr(q, e, gamma, beta, act, y, rows, C, dt, None)


def act_bwd(dy=DY, q=Q, e=E, act=1, dx=DX, rows=4, C=64, dt=c3.BF16):
    return c3.act8_bwd_ptr(dy, q, e, act, dx, rows, C, dt, None)


def lin(x=X, w=W, bias=B, res=R, y=Y, q=None, e=None, rows=4, K=64, N=64, act=0, dt=c3.BF16):
    return c3.linear_fwd_ptr(x, w, bias, res, y, q, e, rows, K, N, act, dt, None)


def lin_bwd(dy=DY, w=W, q=None, e=None, act=0, dx=DX, x=None, rows=4, K=64, N=64, dt=c3.BF16):
    return c3.linear_bwd_data_ptr(dy, w, q, e, act, dx, x, rows, K, N, dt, None)


def lin_dw(x=X, dy=DY, dw=W, db=B, rows=4, K=64, N=64, dt=c3.BF16, ws=R, ws_bytes=1 << 30):
    return c3.linear_bwd_weight_ptr(x, dy, dw, db, rows, K, N, dt, ws, ws_bytes, None)


CALLS = [ln_fwd, ln_bwd, pack, unpack, act_bwd]
PRODUCTS = [lin, lin_bwd, lin_dw]


@pytest.mark.parametrize("call", CALLS + PRODUCTS)
def test_sizes_and_dtype(call):
    assert call(rows=0) == Status.INVALID_ARG
    assert call(rows=-1) == Status.INVALID_ARG
    assert call(dt=7) == Status.INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
def test_channels(call):
    assert call(C=0) == Status.INVALID_ARG
    assert call(C=12) == Status.UNSUPPORTED
    assert "multiple of 8" in c3.last_error()


@pytest.mark.parametrize("call", PRODUCTS)
def test_product_extents(call):
    assert call(K=0) == Status.INVALID_ARG
    assert call(N=-8) == Status.INVALID_ARG
    assert call(K=60) == Status.UNSUPPORTED
    assert call(N=4) == Status.UNSUPPORTED
    assert call(rows=1 << 31) == Status.UNSUPPORTED


@pytest.mark.parametrize("call", PRODUCTS)
def test_product_row_limit(call):
    """A persistent pair's next tile may lie 74 tiles of 256 rows behind the last one: its row stays an int."""
    assert call(rows=2 ** 31 - 65535) == Status.UNSUPPORTED
    assert call(rows=2 ** 31 - 18944) == Status.UNSUPPORTED
    assert c3.linear_bwd_weight_workspace_bytes(2 ** 31 - 65535, 64, 64) == 0


def test_layernorm_channel_limit():
    assert ln_fwd(C=8200) == Status.UNSUPPORTED
    assert ln_bwd(C=8200) == Status.UNSUPPORTED
    assert c3.layernorm_bwd_workspace_bytes(4, 8200) == 0
    assert c3.layernorm_bwd_workspace_bytes(0, 64) == 0
    assert c3.layernorm_bwd_workspace_bytes(1, 64) == 512


def test_nulls():
    for kw in ({"x": None}, {"y": None}, {"q": Q}, {"e": E}, {"eps": -1.0}, {"eps": float("nan")}):
        assert ln_fwd(**kw) == Status.INVALID_ARG, kw
    for kw in ({"dy": None}, {"dx": None}, {"rstd": None}, {"x": None}, {"mean": None}, {"q": Q, "e": E}, {"q": Q},
               {"x": None, "mean": None, "q": Q}, {"x": None, "q": Q, "e": E}):
        assert ln_bwd(**kw) == Status.INVALID_ARG, kw
    for kw in ({"x": None}, {"q": None}, {"e": None}):
        assert pack(**kw) == Status.INVALID_ARG, kw
    for kw in ({"q": None}, {"e": None}, {"y": None}, {"act": 3}, {"act": -1}):
        assert unpack(**kw) == Status.INVALID_ARG, kw
    for kw in ({"dy": None}, {"dx": None}, {"q": None}, {"act": 5}):
        assert act_bwd(**kw) == Status.INVALID_ARG, kw
    for kw in ({"x": None}, {"w": None}, {"y": None}, {"q": Q}, {"e": E}, {"act": 3}):
        assert lin(**kw) == Status.INVALID_ARG, kw
    for kw in ({"dy": None}, {"w": None}, {"dx": None}, {"q": Q}, {"act": 1}, {"act": 9}):
        assert lin_bwd(**kw) == Status.INVALID_ARG, kw


@pytest.mark.parametrize("call,name", [(ln_fwd, n) for n in ("x", "y", "gamma", "beta")] +
                         [(ln_bwd, n) for n in ("dy", "x", "dx", "gamma", "dg", "db")] +
                         [(pack, n) for n in ("x", "q", "e")] + [(unpack, n) for n in ("q", "e", "y")] +
                         [(act_bwd, n) for n in ("dy", "q", "e", "dx")] +
                         [(lin, n) for n in ("x", "w", "bias", "res", "y")] +
                         [(lin_bwd, n) for n in ("dy", "w", "dx")] + [(lin_dw, n) for n in ("x", "dy", "dw", "db")])
def test_alignment(call, name):
    defaults = dict(zip(call.__code__.co_varnames, call.__defaults__))
    assert call(**{name: defaults[name] + 8}) == Status.ALIGNMENT
    assert "aligned" in c3.last_error()


def test_alignment_of_the_optional_buffers():
    assert ln_fwd(mean=MEAN + 2) == Status.ALIGNMENT
    assert ln_fwd(q=Q + 8, e=E) == Status.ALIGNMENT
    assert ln_bwd(rstd=RSTD + 1) == Status.ALIGNMENT
    assert ln_bwd(ws=B + 64) == Status.ALIGNMENT
    assert lin(q=Q, e=E + 4) == Status.ALIGNMENT


def test_workspace():
    need = c3.layernorm_bwd_workspace_bytes(4, 64)
    assert ln_bwd(ws=None) == Status.WORKSPACE
    assert ln_bwd(ws_bytes=need - 1) == Status.WORKSPACE
    assert str(need) in c3.last_error()


def test_weight_gradient_workspace():
    assert c3.linear_bwd_weight_workspace_bytes(4, 64, 64) == 0                 # one row range
    need = c3.linear_bwd_weight_workspace_bytes(100000, 512, 2048)
    assert need > 0 and need % 256 == 0
    big = dict(rows=100000, K=512, N=2048)
    assert lin_dw(**big, ws=None) == Status.WORKSPACE
    assert lin_dw(**big, ws_bytes=need - 1) == Status.WORKSPACE
    assert lin_dw(**big, ws=R + 64) == Status.ALIGNMENT
    assert lin_dw(**big, ws=DY) == Status.INVALID_ARG
    assert c3.linear_bwd_weight_workspace_bytes(0, 64, 64) == 0


def test_layernorm_outputs_overlap_nothing():
    assert ln_fwd(y=G) == Status.INVALID_ARG
    for name in ("mean", "rstd"):
        assert ln_fwd(**{name: G + 64}) == Status.INVALID_ARG
        assert ln_fwd(**{name: B}) == Status.INVALID_ARG
    assert ln_fwd(q=G, e=E) == Status.INVALID_ARG
    assert ln_fwd(q=Q, e=B + 16) == Status.INVALID_ARG


def test_overlaps():
    n = 4 * 64 * 2
    assert lin_dw(dw=X) == Status.INVALID_ARG
    assert lin_dw(dw=DY + 16) == Status.INVALID_ARG
    assert lin_dw(db=W + 16) == Status.INVALID_ARG
    assert lin_dw(x=None) == Status.INVALID_ARG and lin_dw(dw=None) == Status.INVALID_ARG
    assert ln_fwd(y=X + 16) == Status.INVALID_ARG
    assert ln_fwd(y=G) == Status.INVALID_ARG
    assert ln_fwd(q=X, e=E) == Status.INVALID_ARG
    assert ln_fwd(q=Q, e=Q + 16) == Status.INVALID_ARG
    assert ln_fwd(rstd=Y + n - 4) == Status.INVALID_ARG
    assert ln_fwd(mean=RSTD, rstd=RSTD) == Status.INVALID_ARG
    assert ln_bwd(dx=DY + 16) == Status.INVALID_ARG
    assert ln_bwd(dx=X + n - 16) == Status.INVALID_ARG
    assert ln_bwd(dg=W, db=W) == Status.INVALID_ARG
    assert ln_bwd(dg=DY) == Status.INVALID_ARG
    assert ln_bwd(ws=DX) == Status.INVALID_ARG
    assert pack(q=X) == Status.INVALID_ARG
    assert pack(e=Q + 128) == Status.INVALID_ARG
    assert unpack(y=Q) == Status.INVALID_ARG
    assert act_bwd(dx=DY + 16) == Status.INVALID_ARG
    assert act_bwd(dx=E) == Status.INVALID_ARG
    assert lin(y=X) == Status.INVALID_ARG
    assert lin(y=W + 16) == Status.INVALID_ARG
    assert lin(y=R + 16) == Status.INVALID_ARG
    assert lin(q=Y, e=E) == Status.INVALID_ARG
    assert lin(q=R, e=E) == Status.INVALID_ARG
    assert lin_bwd(dx=DY) == Status.INVALID_ARG
    assert lin_bwd(act=1, q=DX, e=E) == Status.INVALID_ARG
    assert lin_bwd(act=1, q=Q, e=E, x=DX) == Status.INVALID_ARG
    assert lin_bwd(act=1, q=Q, e=E, x=DY + 16) == Status.INVALID_ARG
    assert lin_bwd(act=1, q=Q, e=E, x=E) == Status.INVALID_ARG
    assert lin_bwd(act=1, q=Q, e=E, x=X + 8) == Status.ALIGNMENT
    assert lin_bwd(act=0, q=Q, e=E, x=X) == Status.INVALID_ARG


def test_python_checks_need_no_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    a = c3.Act8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), 64)
    for call in (lambda: c3.layernorm(x), lambda: c3.act8_pack(x), lambda: c3.act8_bwd(x, a, 1),
                 lambda: c3.act8_unpack(a, torch.bfloat16), lambda: c3.linear(x, torch.zeros(8, 64)),
                 lambda: c3.linear_bwd_data(x, torch.zeros(64, 64)), lambda: c3.linear_bwd_weight(x, x),
                 lambda: c3.layernorm_bwd(x, x, torch.zeros(4))):
        with pytest.raises((ValueError, TypeError)):
            call()
    empty = c3.Act8.empty((3, 5, 40), "cpu")
    assert tuple(empty.codes.shape) == (3, 5, 64) and tuple(empty.exponents.shape) == (3, 5, 2)


def test_reference_codes_by_hand():
    """The 64-bit code of the tests against values worked out by hand."""
    from channel_ref import codes
    v = torch.zeros(1, 40, dtype=torch.float64)
    v[0, 0], v[0, 1], v[0, 2], v[0, 3] = 1.0, -0.5, 1.0 / 128, 3.0 / 128    # exponent 0: step 2^-6
    v[0, 32] = 1.9999                                                        # 127.99 steps: clamps
    k, e = codes(v)
    assert e.tolist() == [[127, 127]]
    assert k[0, :4].tolist() == [64, -32, 0, 2]                              # 0.5 -> 0, 1.5 -> 2: ties to even
    assert k[0, 32].item() == 127 and k[0, 40:].abs().sum() == 0
    k, e = codes(torch.full((1, 8), 2.0 ** -130, dtype=torch.float64))
    assert e.item() == 7 and k[0, 0].item() == 0
