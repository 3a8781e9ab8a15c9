"""Python binding of libconv3d: implicit-GEMM 3D convolution on B200 (sm_100a).

Argument marshalling only.  Every step of the convolution runs in the CUDA
library ``libconv3d.so`` (built from ``csrc/`` by ``build.py``); torch is used
here for device memory and streams.  There is no fallback: if the library is
missing or fails to load, importing this package raises.

Operation (engineering.drawthings.ai, "Metal conv3d" post; Qwen Image post,
"Video VAE" section): y = conv3d(x, w) + bias + residual with NDHWC
activations, [Cout, kt, kh, kw, Cin] weights, spatial zero padding, strides
and a temporal padding mode (zero, causal replicate-first-frame, causal zero,
or the cached frames of the previous chunk).  Also: the GroupNorm + SiLU pass
in front of a decoder convolution (groupnorm_stats / groupnorm_silu), the
backward pass (conv3d_bwd_data, conv3d_bwd_weight) and a torch.autograd
wrapper over both directions (Conv3dFunction / conv3d_autograd).  Each call has
a raw-pointer twin (``*_ptr``) that returns the library's status code.

Channel-wise operators on [..., C] tensors, a row per pixel or token: layer norm
(layernorm, layernorm_bwd), 8-bit activation checkpoints (Act8, act8_pack,
act8_unpack, act8_bwd), the channel product with its epilogue (linear,
linear_bwd_data, linear_bwd_weight) and the channel MLP block made of them
(channel_mlp, channel_mlp_bwd), each with a torch.autograd wrapper.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

__all__ = [
    "TPAD_ZERO", "TPAD_CAUSAL_REPLICATE", "TPAD_CAUSAL_ZERO", "TPAD_CAUSAL_CACHED", "F16", "BF16",
    "Status", "Conv3dError", "lib_path", "status_string", "last_error", "kernel_launches",
    "conv3d", "conv3d_fwd", "conv3d_fwd_ptr", "conv3d_fwd_ws_ptr", "conv3d_fwd_noalloc_ptr",
    "conv3d_fwd_cached_ptr", "conv3d_gn", "conv3d_gn_ptr", "output_shape", "workspace_bytes",
    "groupnorm_stats", "groupnorm_silu", "groupnorm_stats_ptr", "groupnorm_silu_ptr",
    "conv3d_bwd_data", "conv3d_bwd_data_ptr", "bwd_data_workspace_bytes",
    "conv3d_bwd_weight", "conv3d_bwd_weight_ptr", "bwd_weight_workspace_bytes",
    "conv3d_bwd_data_cached", "conv3d_bwd_weight_cached",
    "Conv3dFunction", "conv3d_autograd",
    "ACT_NONE", "ACT_SILU", "ACT_GELU", "Act8", "act8_pack", "act8_unpack", "act8_bwd",
    "layernorm", "layernorm_bwd", "layernorm_bwd_workspace_bytes", "LayerNormFunction",
    "layernorm_autograd", "linear", "linear_bwd_data", "linear_bwd_weight", "LinearFunction",
    "linear_autograd", "ChannelMlpSaved", "channel_mlp", "channel_mlp_bwd", "ChannelMlpFunction",
    "channel_mlp_autograd", "layernorm_fwd_ptr", "layernorm_bwd_ptr", "act8_pack_ptr",
    "act8_unpack_ptr", "act8_bwd_ptr", "linear_fwd_ptr", "linear_bwd_data_ptr",
    "linear_bwd_weight_ptr", "linear_bwd_weight_workspace_bytes",
    "poll_status", "selftest_wait_timeout", "release", "test_arm_stall",
]

F16 = 0
BF16 = 1
TPAD_ZERO = 0
TPAD_CAUSAL_REPLICATE = 1
TPAD_CAUSAL_ZERO = 2
TPAD_CAUSAL_CACHED = 3
ACT_NONE = 0
ACT_SILU = 1
ACT_GELU = 2


class Status:
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    ALIGNMENT = 3
    CUDA = 4
    TIMEOUT = 5
    DEVICE_CHECK = 6
    WORKSPACE = 7


class Conv3dError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libconv3d status {status}: {message}")
        self.status = status


_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libconv3d.so")

if not os.path.exists(lib_path):
    raise ImportError(f"{lib_path} is missing: build it with "
                      "`python video_vae_convolution_implicit_b200/build.py` (nvcc, sm_100a)")
_lib = ctypes.CDLL(lib_path)


class _NoBinding:
    """Stands in for the native binding where it does not load (not built, or built
    against another torch): the calls that need it say so, the others do without."""

    def __init__(self, cause: ImportError):
        self._cause = cause

    def __getattr__(self, name):
        raise ImportError("the native binding _channel.so is missing or does not load: build it with "
                          "`python video_vae_convolution_implicit_b200/build.py`") from self._cause


try:
    from . import _channel   # the native calls of the channel-wise operators (csrc/binding.cpp)
except ImportError as e:
    _channel = _NoBinding(e)

_i3 = ctypes.c_int * 3
_vp = ctypes.c_void_p
_c = ctypes.c_int

_lib.conv3d_fwd.restype = _c
_lib.conv3d_fwd.argtypes = [_vp] * 5 + [_c] * 6 + [_i3] * 3 + [_c, _c, _vp]
_lib.conv3d_fwd_ws.restype = _c
_lib.conv3d_fwd_ws.argtypes = [_vp] * 5 + [_c] * 6 + [_i3] * 3 + [_c, _c, _vp, ctypes.c_size_t, _vp]
_lib.conv3d_fwd_cached.restype = _c
_lib.conv3d_fwd_cached.argtypes = [_vp] * 6 + [_c] * 6 + [_i3] * 3 + [_c, _vp]
_lib.conv3d_groupnorm_stats.restype = _c
_lib.conv3d_groupnorm_stats.argtypes = [_vp] + [_c] * 7 + [ctypes.c_float, _c, _vp, _vp]
_lib.conv3d_groupnorm_silu.restype = _c
_lib.conv3d_groupnorm_silu.argtypes = [_vp] * 5 + [_c] * 8 + [_c, _vp]
_lib.conv3d_bwd_data.restype = _c
_lib.conv3d_bwd_data.argtypes = [_vp] * 3 + [_c] * 6 + [_i3] * 3 + [_c, _c, _vp, ctypes.c_size_t,
                                                                   _vp]
_lib.conv3d_bwd_data_workspace_bytes.restype = ctypes.c_size_t
_lib.conv3d_bwd_data_workspace_bytes.argtypes = [_c] * 6 + [_i3, _i3, _c]
_lib.conv3d_bwd_weight.restype = _c
_lib.conv3d_bwd_weight.argtypes = [_vp] * 4 + [_c] * 6 + [_i3] * 3 + [_c, _c, _vp,
                                                                     ctypes.c_size_t, _vp]
_lib.conv3d_bwd_data_cached.restype = _c
_lib.conv3d_bwd_data_cached.argtypes = [_vp] * 4 + [_c] * 6 + [_i3] * 3 + [_c, _vp, ctypes.c_size_t,
                                                                          _vp]
_lib.conv3d_bwd_weight_cached.restype = _c
_lib.conv3d_bwd_weight_cached.argtypes = [_vp] * 5 + [_c] * 6 + [_i3] * 3 + [_c, _vp,
                                                                            ctypes.c_size_t, _vp]
_lib.conv3d_bwd_weight_workspace_bytes.restype = ctypes.c_size_t
_lib.conv3d_bwd_weight_workspace_bytes.argtypes = [_c, _c, _i3]
_lib.conv3d_fwd_noalloc.restype = _c
_lib.conv3d_fwd_noalloc.argtypes = [_vp] * 5 + [_c] * 6 + [_i3] * 3 + [_c, _c, _vp]
_lib.conv3d_workspace_bytes.restype = ctypes.c_size_t
_lib.conv3d_workspace_bytes.argtypes = [_c, _c, _i3, _c, _c]
_lib.conv3d_output_shape.restype = _c
_lib.conv3d_output_shape.argtypes = [_c, _c, _c, _i3, _i3, _i3, _c, _i3]
_lib.conv3d_poll_status.restype = _c
_lib.conv3d_poll_status.argtypes = [_vp]
_lib.conv3d_status_string.restype = ctypes.c_char_p
_lib.conv3d_status_string.argtypes = [_c]
_lib.conv3d_last_error.restype = ctypes.c_char_p
_lib.conv3d_last_error.argtypes = []
_lib.conv3d_kernel_launches.restype = ctypes.c_ulonglong
_lib.conv3d_kernel_launches.argtypes = []
_lib.conv3d_release.restype = None
_lib.conv3d_release.argtypes = []
_lib.conv3d_selftest_wait_timeout.restype = _c
_lib.conv3d_selftest_wait_timeout.argtypes = [_c]
_lib.conv3d_fwd_gn.restype = _c
_lib.conv3d_fwd_gn.argtypes = ([_vp, _vp, _vp, _vp, _c, _c, _c] + [_vp] * 4 + [_c] * 6 + [_i3] * 3
                                + [_c, _c, _vp, _c, ctypes.c_float, _vp])
_lib.conv3d_test_arm_stall.restype = _c
_lib.conv3d_test_arm_stall.argtypes = [_c, _c]
_ll = ctypes.c_longlong
_lib.conv3d_layernorm_fwd.restype = _c
_lib.conv3d_layernorm_fwd.argtypes = [_vp] * 8 + [_ll, _c, ctypes.c_float, _c, _vp]
_lib.conv3d_layernorm_bwd.restype = _c
_lib.conv3d_layernorm_bwd.argtypes = [_vp] * 11 + [_ll, _c, _c, _vp, ctypes.c_size_t, _vp]
_lib.conv3d_layernorm_bwd_workspace_bytes.restype = ctypes.c_size_t
_lib.conv3d_layernorm_bwd_workspace_bytes.argtypes = [_ll, _c]
_lib.conv3d_act8_pack.restype = _c
_lib.conv3d_act8_pack.argtypes = [_vp] * 3 + [_ll, _c, _c, _vp]
_lib.conv3d_act8_unpack.restype = _c
_lib.conv3d_act8_unpack.argtypes = [_vp] * 4 + [_c, _vp, _ll, _c, _c, _vp]
_lib.conv3d_act8_bwd.restype = _c
_lib.conv3d_act8_bwd.argtypes = [_vp] * 3 + [_c, _vp, _ll, _c, _c, _vp]
_lib.conv3d_linear_fwd.restype = _c
_lib.conv3d_linear_fwd.argtypes = [_vp] * 7 + [_ll, _c, _c, _c, _c, _vp]
_lib.conv3d_linear_bwd_data.restype = _c
_lib.conv3d_linear_bwd_data.argtypes = [_vp] * 4 + [_c, _vp, _vp, _ll, _c, _c, _c, _vp]
_lib.conv3d_linear_bwd_weight.restype = _c
_lib.conv3d_linear_bwd_weight.argtypes = [_vp] * 4 + [_ll, _c, _c, _c, _vp, ctypes.c_size_t, _vp]
_lib.conv3d_linear_bwd_weight_workspace_bytes.restype = ctypes.c_size_t
_lib.conv3d_linear_bwd_weight_workspace_bytes.argtypes = [_ll, _c, _c]

if not isinstance(_channel, _NoBinding):
    _channel.set_error_class(Conv3dError)


def raw_library() -> ctypes.CDLL:
    """The loaded ctypes handle of libconv3d.so."""
    return _lib


def status_string(status: int) -> str:
    return _lib.conv3d_status_string(status).decode()


def last_error() -> str:
    return _lib.conv3d_last_error().decode()


def kernel_launches() -> int:
    """GPU kernels the library has launched in this process (counted at enqueue)."""
    return int(_lib.conv3d_kernel_launches())


def _check(status: int) -> None:
    if status != Status.OK:
        raise Conv3dError(status, f"{status_string(status)}: {last_error()}")


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float16:
        return F16
    raise TypeError(f"libconv3d computes in bf16 or fp16, got {t}")


def _stream_handle(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class _CallOn:
    """The stream a call is given, current while the call lasts, so that what it allocates
    belongs to the stream its kernels run on and is not handed to another one before they
    have run.  Enters as the stream to run on (None: the current one).

    CUDA's handle 1 is the legacy default stream, torch's 0.  Handle 2 is the calling
    thread's, which torch's allocator cannot keep memory for: the current stream's is used,
    and the two streams wait for each other around the call."""

    def __init__(self, stream):
        self._stream, self._guard, self._lender = stream, None, None

    def __enter__(self):
        if self._stream is None:
            return None
        handle = _stream_handle(self._stream)
        if handle == 2:
            lender = torch.cuda.current_stream()
            torch.cuda.ExternalStream(2).wait_stream(lender)
            self._lender = lender
            return handle
        if handle in (0, 1):
            handle, stream = 0, torch.cuda.default_stream()
        elif isinstance(self._stream, torch.cuda.Stream):
            stream = self._stream
        else:
            stream = torch.cuda.ExternalStream(handle)
        self._guard = torch.cuda.stream(stream)
        self._guard.__enter__()
        return handle

    def __exit__(self, *error):
        if self._lender is not None:
            self._lender.wait_stream(torch.cuda.ExternalStream(2))
        if self._guard is not None:
            self._guard.__exit__(*error)


def output_shape(D, H, W, kernel, stride=(1, 1, 1), pad=(0, 1, 1), tpad=TPAD_CAUSAL_REPLICATE):
    out = _i3()
    _check(_lib.conv3d_output_shape(D, H, W, _i3(*kernel), _i3(*stride), _i3(*pad), tpad, out))
    return tuple(out)


def workspace_bytes(Cin, Cout, kernel, D, tpad) -> int:
    return int(_lib.conv3d_workspace_bytes(Cin, Cout, _i3(*kernel), D, tpad))


def conv3d_fwd_ptr(x, w, bias, residual, y, N, Cin, D, H, W, Cout, kernel, stride, pad, tpad,
                   dtype, stream) -> int:
    """Raw-pointer call of conv3d_fwd; returns the status code (no raise)."""
    return _lib.conv3d_fwd(x, w, bias, residual, y, N, Cin, D, H, W, Cout, _i3(*kernel),
                           _i3(*stride), _i3(*pad), tpad, dtype, stream)


def conv3d_fwd_ws_ptr(x, w, bias, residual, y, N, Cin, D, H, W, Cout, kernel, stride, pad, tpad,
                      dtype, workspace, ws_bytes, stream) -> int:
    """Raw-pointer call of conv3d_fwd_ws; returns the status code (no raise)."""
    return _lib.conv3d_fwd_ws(x, w, bias, residual, y, N, Cin, D, H, W, Cout, _i3(*kernel),
                              _i3(*stride), _i3(*pad), tpad, dtype, workspace, ws_bytes, stream)


def conv3d_fwd_noalloc_ptr(x, w, bias, residual, y, N, Cin, D, H, W, Cout, kernel, stride, pad,
                           tpad, dtype, stream) -> int:
    """Raw-pointer call of conv3d_fwd_noalloc (for callers that cannot allocate
    device memory; its first-frame scratch is a fixed 16 MiB array inside the
    library).  Returns the status code (no raise)."""
    return _lib.conv3d_fwd_noalloc(x, w, bias, residual, y, N, Cin, D, H, W, Cout, _i3(*kernel),
                                   _i3(*stride), _i3(*pad), tpad, dtype, stream)


def conv3d_fwd_cached_ptr(x, prev, w, bias, residual, y, N, Cin, D, H, W, Cout, kernel, stride,
                          pad, dtype, stream) -> int:
    """Raw-pointer call of conv3d_fwd_cached (one chunk of a causal conv whose
    front padding is the previous chunk's last kt-1 frames).  Returns the status."""
    return _lib.conv3d_fwd_cached(x, prev, w, bias, residual, y, N, Cin, D, H, W, Cout,
                                  _i3(*kernel), _i3(*stride), _i3(*pad), dtype, stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _overwritten(*tensors) -> None:
    """Tensors of the caller's that a call writes: autograd is told, as torch's own in-place
    operators tell it, so that a backward pass which saved one of them notices."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def conv3d_fwd(x: torch.Tensor, w: torch.Tensor, bias, residual, y: torch.Tensor,
               stride=(1, 1, 1), pad=(0, 1, 1), tpad=TPAD_CAUSAL_REPLICATE, stream=None,
               workspace: torch.Tensor | None = None, prev: torch.Tensor | None = None
               ) -> torch.Tensor:
    """Enqueue y = conv3d(x, w) + bias + residual on ``stream`` (default: current stream).

    x: [N, D, H, W, Cin]; w: [Cout, kt, kh, kw, Cin]; bias: [Cout] or None;
    residual: y's shape or None; y: [N, Do, Ho, Wo, Cout].  All contiguous CUDA
    tensors of one dtype (bf16 or fp16).  With ``workspace`` (a uint8 CUDA
    tensor) the call goes through conv3d_fwd_ws and never allocates.  With
    tpad=TPAD_CAUSAL_CACHED, ``prev`` ([N, kt-1, H, W, Cin]) holds the frames
    before x and the call goes through conv3d_fwd_cached.
    """
    for name, t in (("x", x), ("w", w), ("y", y), ("bias", bias), ("residual", residual),
                    ("prev", prev)):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != x.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, x has {x.dtype}")
    if x.dim() != 5 or w.dim() != 5:
        raise ValueError("x must be [N,D,H,W,Cin] and w [Cout,kt,kh,kw,Cin]")
    N, D, H, W, Cin = x.shape
    Cout, kt, kh, kw, Cin_w = w.shape
    if Cin_w != Cin:
        raise ValueError("w's last extent must equal Cin")
    out = output_shape(D, H, W, (kt, kh, kw), stride, pad, tpad)
    if tuple(y.shape) != (N, *out, Cout):
        raise ValueError(f"y must be {(N, *out, Cout)}, got {tuple(y.shape)}")
    if residual is not None and tuple(residual.shape) != tuple(y.shape):
        raise ValueError("residual must have y's shape")
    if bias is not None and tuple(bias.shape) != (Cout,):
        raise ValueError("bias must be [Cout]")
    code = _dtype_code(x.dtype)
    s = _stream_handle(stream)
    if tpad == TPAD_CAUSAL_CACHED:
        if prev is not None and tuple(prev.shape) != (N, kt - 1, H, W, Cin):
            raise ValueError(f"prev must be {(N, kt - 1, H, W, Cin)}")
        st = conv3d_fwd_cached_ptr(_ptr(x), _ptr(prev), _ptr(w), _ptr(bias), _ptr(residual),
                                   _ptr(y), N, Cin, D, H, W, Cout, (kt, kh, kw), stride, pad, code,
                                   s)
    elif workspace is None:
        st = conv3d_fwd_ptr(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), N, Cin, D, H,
                            W, Cout, (kt, kh, kw), stride, pad, tpad, code, s)
    else:
        st = conv3d_fwd_ws_ptr(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), N, Cin, D,
                               H, W, Cout, (kt, kh, kw), stride, pad, tpad, code,
                               _ptr(workspace), workspace.numel() * workspace.element_size(), s)
    _check(st)
    _overwritten(y)
    return y


def conv3d(x: torch.Tensor, w: torch.Tensor, bias=None, residual=None, stride=(1, 1, 1),
           pad=(0, 1, 1), tpad=TPAD_CAUSAL_REPLICATE, stream=None, prev=None) -> torch.Tensor:
    """Allocate y (torch) and run :func:`conv3d_fwd`."""
    with _CallOn(stream) as s:
        N, D, H, W, _ = x.shape
        Cout, kt, kh, kw, _ = w.shape
        out = output_shape(D, H, W, (kt, kh, kw), stride, pad, tpad)
        y = torch.empty((N, *out, Cout), dtype=x.dtype, device=x.device)
        return conv3d_fwd(x, w, bias, residual, y, stride, pad, tpad, s, prev=prev)


def conv3d_gn_ptr(x, stats, gamma, beta, groups, per_frame, apply_silu, w, bias, residual, y, N,
                  Cin, D, H, W, Cout, kernel, stride, pad, tpad, dtype, stream, out_stats=None,
                  out_groups=0, out_eps=1e-6) -> int:
    """Raw-pointer call of conv3d_fwd_gn; returns the status code (no raise)."""
    return _lib.conv3d_fwd_gn(x, stats, gamma, beta, groups, int(per_frame), int(apply_silu), w,
                              bias, residual, y, N, Cin, D, H, W, Cout, _i3(*kernel),
                              _i3(*stride), _i3(*pad), tpad, dtype, out_stats, int(out_groups),
                              float(out_eps), stream)


def conv3d_gn(x: torch.Tensor, stats, gamma, beta, w: torch.Tensor, bias=None,
              residual=None, y: torch.Tensor | None = None, groups: int | None = None,
              per_frame: bool = False, apply_silu: bool = True, stride=(1, 1, 1), pad=(0, 1, 1),
              tpad=TPAD_CAUSAL_REPLICATE, out_groups: int = 0, out_eps: float = 1e-6,
              stream=None):
    """y = conv3d(silu(GroupNorm(x)), w) + bias + residual with the GroupNorm + SiLU
    applied as the convolution reads x (``stats`` from groupnorm_stats over x, or
    None for plain x).  With ``out_groups`` > 0 also returns the per-sample
    GroupNorm statistics of y ([N, out_groups, 2] float64): (y, out_stats)."""
    with _CallOn(stream) as s:
        N, D, H, W, Cin = x.shape
        Cout, kt, kh, kw, _ = w.shape
        groups = (stats.shape[1] if stats is not None else 1) if groups is None else groups
        if y is None:
            out = output_shape(D, H, W, (kt, kh, kw), stride, pad, tpad)
            y = torch.empty((N, *out, Cout), dtype=x.dtype, device=x.device)
        for name, t in (("x", x), ("w", w), ("y", y)):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != x.dtype:
                raise ValueError(f"{name} must be a contiguous CUDA tensor of x's dtype")
        if stats is not None and (stats.dtype != torch.float64 or not stats.is_cuda):
            raise ValueError("stats must be a float64 CUDA tensor")
        out_stats = (torch.empty((N, out_groups, 2), dtype=torch.float64, device=x.device)
                     if out_groups > 0 else None)
        _check(conv3d_gn_ptr(x.data_ptr(), _ptr(stats), _ptr(gamma), _ptr(beta), groups,
                             per_frame, apply_silu, w.data_ptr(), _ptr(bias), _ptr(residual),
                             y.data_ptr(), N, Cin, D, H, W, Cout, (kt, kh, kw), stride, pad, tpad,
                             _dtype_code(x.dtype), _stream_handle(s), _ptr(out_stats),
                             out_groups, out_eps))
        _overwritten(y)
        return (y, out_stats) if out_stats is not None else y


def poll_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device status word."""
    return int(_lib.conv3d_poll_status(_stream_handle(stream)))


def selftest_wait_timeout(timeout_ms: int) -> int:
    """Run the bounded-wait self test; returns Status.TIMEOUT when it works."""
    return int(_lib.conv3d_selftest_wait_timeout(timeout_ms))


def release() -> None:
    _lib.conv3d_release()


def test_arm_stall(launches: int, timeout_ms: int = 50) -> None:
    """Failure-detection test hook: the next ``launches`` convolution-kernel
    launches stall on their first pipeline stage and abort after ``timeout_ms``
    (poll_status then returns Status.TIMEOUT).  0 disarms."""
    _check(_lib.conv3d_test_arm_stall(int(launches), int(timeout_ms)))


def groupnorm_stats_ptr(x, N, D, H, W, C, groups, per_frame, eps, dtype, stats, stream) -> int:
    """Raw-pointer call of conv3d_groupnorm_stats; returns the status code."""
    return _lib.conv3d_groupnorm_stats(x, N, D, H, W, C, groups, int(per_frame), eps, dtype, stats,
                                       stream)


def groupnorm_silu_ptr(x, stats, gamma, beta, y, N, D, H, W, C, groups, per_frame, apply_silu,
                       dtype, stream) -> int:
    """Raw-pointer call of conv3d_groupnorm_silu; returns the status code."""
    return _lib.conv3d_groupnorm_silu(x, stats, gamma, beta, y, N, D, H, W, C, groups,
                                      int(per_frame), int(apply_silu), dtype, stream)


def groupnorm_stats(x: torch.Tensor, groups: int, eps: float = 1e-6, per_frame: bool = False,
                    stats: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """{mean, 1/sqrt(var+eps)} per (sample [, frame], group) of an NDHWC tensor, as a
    float64 CUDA tensor [sets, groups, 2] (``stats`` is reused when given)."""
    with _CallOn(stream) as s:
        if not x.is_cuda or not x.is_contiguous() or x.dim() != 5:
            raise ValueError("x must be a contiguous CUDA tensor [N, D, H, W, C]")
        N, D, H, W, C = x.shape
        sets = N * D if per_frame else N
        if stats is None:
            stats = torch.empty((sets, groups, 2), dtype=torch.float64, device=x.device)
        elif tuple(stats.shape) != (sets, groups, 2) or stats.dtype != torch.float64:
            raise ValueError(f"stats must be float64 {(sets, groups, 2)}")
        _check(groupnorm_stats_ptr(x.data_ptr(), N, D, H, W, C, groups, per_frame, eps,
                                   _dtype_code(x.dtype), stats.data_ptr(), _stream_handle(s)))
        _overwritten(stats)
        return stats


def groupnorm_silu(x: torch.Tensor, stats: torch.Tensor, gamma=None, beta=None, y=None,
                   groups: int | None = None, per_frame: bool = False, apply_silu: bool = True,
                   stream=None) -> torch.Tensor:
    """y = silu((x - mean) * rstd * gamma + beta) with ``stats`` from groupnorm_stats.
    ``y`` may be ``x`` (in place); it is allocated when None."""
    with _CallOn(stream) as s:
        if not x.is_cuda or not x.is_contiguous() or x.dim() != 5:
            raise ValueError("x must be a contiguous CUDA tensor [N, D, H, W, C]")
        N, D, H, W, C = x.shape
        groups = stats.shape[1] if groups is None else groups
        if y is None:
            y = torch.empty_like(x)
        for name, t in (("gamma", gamma), ("beta", beta)):
            if t is not None and (tuple(t.shape) != (C,) or t.dtype != x.dtype or not t.is_cuda):
                raise ValueError(f"{name} must be a CUDA [C] tensor of x's dtype")
        _check(groupnorm_silu_ptr(x.data_ptr(), stats.data_ptr(), _ptr(gamma), _ptr(beta),
                                  y.data_ptr(), N, D, H, W, C, groups, per_frame, apply_silu,
                                  _dtype_code(x.dtype), _stream_handle(s)))
        _overwritten(y)
        return y


def conv3d_bwd_data_ptr(dy, w, dx, N, Cin, D, H, W, Cout, kernel, stride, pad, tpad, dtype,
                        workspace, ws_bytes, stream) -> int:
    """Raw-pointer call of conv3d_bwd_data; returns the status code."""
    return _lib.conv3d_bwd_data(dy, w, dx, N, Cin, D, H, W, Cout, _i3(*kernel), _i3(*stride),
                                _i3(*pad), tpad, dtype, workspace, ws_bytes, stream)


def bwd_data_workspace_bytes(N, Cin, D, H, W, Cout, kernel, pad, tpad) -> int:
    return int(_lib.conv3d_bwd_data_workspace_bytes(N, Cin, D, H, W, Cout, _i3(*kernel), _i3(*pad),
                                                    tpad))


def conv3d_bwd_data(dy: torch.Tensor, w: torch.Tensor, x_shape, pad=(0, 1, 1),
                    tpad=TPAD_CAUSAL_REPLICATE, dx: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None,
                    stride=(1, 1, 1)) -> torch.Tensor:
    """dx for the forward problem x [x_shape] -> y (dy has y's shape); temporal
    stride 1, spatial strides up to 8."""
    with _CallOn(stream) as s:
        N, D, H, W, Cin = x_shape
        Cout, kt, kh, kw, _ = w.shape
        if dx is None:
            dx = torch.empty(tuple(x_shape), dtype=dy.dtype, device=dy.device)
        need = bwd_data_workspace_bytes(N, Cin, D, H, W, Cout, (kt, kh, kw), pad, tpad)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dy.device)
        for name, t in (("dy", dy), ("w", w), ("dx", dx)):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != dy.dtype:
                raise ValueError(f"{name} must be a contiguous CUDA tensor of dy's dtype")
        _check(conv3d_bwd_data_ptr(dy.data_ptr(), w.data_ptr(), dx.data_ptr(), N, Cin, D, H, W, Cout,
                                   (kt, kh, kw), tuple(stride), pad, tpad, _dtype_code(dy.dtype),
                                   workspace.data_ptr(), workspace.numel(), _stream_handle(s)))
        _overwritten(dx)
        return dx


def conv3d_bwd_weight_ptr(x, dy, dw, dbias, N, Cin, D, H, W, Cout, kernel, stride, pad, tpad,
                          dtype, workspace, ws_bytes, stream) -> int:
    """Raw-pointer call of conv3d_bwd_weight; returns the status code."""
    return _lib.conv3d_bwd_weight(x, dy, dw, dbias, N, Cin, D, H, W, Cout, _i3(*kernel),
                                  _i3(*stride), _i3(*pad), tpad, dtype, workspace, ws_bytes,
                                  stream)


def bwd_weight_workspace_bytes(Cin, Cout, kernel) -> int:
    return int(_lib.conv3d_bwd_weight_workspace_bytes(Cin, Cout, _i3(*kernel)))


def conv3d_bwd_weight(x: torch.Tensor, dy: torch.Tensor, kernel, stride=(1, 1, 1), pad=(0, 1, 1),
                      tpad=TPAD_CAUSAL_REPLICATE, with_bias: bool = True,
                      workspace: torch.Tensor | None = None, stream=None):
    """(dw, dbias) for the forward problem x -> y with upstream gradient dy."""
    with _CallOn(stream) as s:
        N, D, H, W, Cin = x.shape
        Cout = dy.shape[-1]
        dw = torch.empty((Cout, *kernel, Cin), dtype=x.dtype, device=x.device)
        db = torch.empty((Cout,), dtype=x.dtype, device=x.device) if with_bias else None
        need = bwd_weight_workspace_bytes(Cin, Cout, kernel)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        for name, t in (("x", x), ("dy", dy)):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != x.dtype:
                raise ValueError(f"{name} must be a contiguous CUDA tensor of x's dtype")
        _check(conv3d_bwd_weight_ptr(x.data_ptr(), dy.data_ptr(), dw.data_ptr(), _ptr(db), N, Cin, D,
                                     H, W, Cout, tuple(kernel), stride, pad, tpad,
                                     _dtype_code(x.dtype), workspace.data_ptr(), workspace.numel(),
                                     _stream_handle(s)))
        return dw, db


def conv3d_bwd_data_cached(dy: torch.Tensor, w: torch.Tensor, x_shape, pad=(0, 1, 1),
                           with_prev: bool = True, workspace: torch.Tensor | None = None,
                           stream=None):
    """(dx, dprev) for one chunk of the cached-frames mode (stride 1): dprev is
    the gradient of the kt-1 cached frames (None when with_prev is false)."""
    with _CallOn(stream) as s:
        N, D, H, W, Cin = x_shape
        Cout, kt, kh, kw, _ = w.shape
        dx = torch.empty(tuple(x_shape), dtype=dy.dtype, device=dy.device)
        dprev = (torch.empty((N, kt - 1, H, W, Cin), dtype=dy.dtype, device=dy.device)
                 if with_prev and kt > 1 else None)
        need = bwd_data_workspace_bytes(N, Cin, D, H, W, Cout, (kt, kh, kw), pad, TPAD_CAUSAL_CACHED)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dy.device)
        for name, t in (("dy", dy), ("w", w)):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != dy.dtype:
                raise ValueError(f"{name} must be a contiguous CUDA tensor of dy's dtype")
        _check(_lib.conv3d_bwd_data_cached(dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _ptr(dprev), N,
                                           Cin, D, H, W, Cout, _i3(kt, kh, kw), _i3(1, 1, 1),
                                           _i3(*pad), _dtype_code(dy.dtype), workspace.data_ptr(),
                                           workspace.numel(), _stream_handle(s)))
        return dx, dprev


def conv3d_bwd_weight_cached(x: torch.Tensor, prev: torch.Tensor | None, dy: torch.Tensor, kernel,
                             stride=(1, 1, 1), pad=(0, 1, 1), with_bias: bool = True,
                             workspace: torch.Tensor | None = None, stream=None):
    """(dw, dbias) for one chunk of the cached-frames mode; prev: the cached frames."""
    with _CallOn(stream) as s:
        N, D, H, W, Cin = x.shape
        Cout = dy.shape[-1]
        dw = torch.empty((Cout, *kernel, Cin), dtype=x.dtype, device=x.device)
        db = torch.empty((Cout,), dtype=x.dtype, device=x.device) if with_bias else None
        need = bwd_weight_workspace_bytes(Cin, Cout, kernel)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        for name, t in (("x", x), ("dy", dy), ("prev", prev)):
            if t is not None and (not t.is_cuda or not t.is_contiguous() or t.dtype != x.dtype):
                raise ValueError(f"{name} must be a contiguous CUDA tensor of x's dtype")
        _check(_lib.conv3d_bwd_weight_cached(x.data_ptr(), _ptr(prev), dy.data_ptr(), dw.data_ptr(),
                                             _ptr(db), N, Cin, D, H, W, Cout, _i3(*kernel),
                                             _i3(*stride), _i3(*pad), _dtype_code(x.dtype),
                                             workspace.data_ptr(), workspace.numel(),
                                             _stream_handle(s)))
        return dw, db


class _NoSecondDerivative(torch.autograd.Function):
    """Passes gradients on and refuses to be differentiated."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g if g is None else g.detach() for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("libconv3d's gradients are differentiable once: they carry no graph of their own")


def _differentiable_once(backward):
    """A Function's backward whose results refuse to be differentiated again.  (torch's
    once_differentiable lets them pass as constants where the upstream gradient is one,
    although they depend on the call's inputs too.)"""

    @functools.wraps(backward)
    def wrapped(ctx, dy):
        with torch.no_grad():
            grads = backward(ctx, dy)
        if not torch.is_grad_enabled():          # not within create_graph=True
            return grads
        return _NoSecondDerivative.apply(dy.new_empty(0).requires_grad_(), *grads)
    return wrapped


class Conv3dFunction(torch.autograd.Function):
    """torch.autograd wrapper: forward through conv3d_fwd, backward through
    conv3d_bwd_data (dx; temporal stride 1) and conv3d_bwd_weight (dw, dbias).
    The residual's gradient is dy itself.  With checkpoint8 the input is kept as
    an 8-bit checkpoint (Act8), which only dw reads.  Marshalling only: every
    product runs in the library's kernels, none in torch.  Differentiable once, as
    all of these wrappers are: a second derivative is refused."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, stride, pad, tpad, checkpoint8=False):
        y = conv3d(x, w, bias, residual, stride, pad, tpad)
        if not checkpoint8:
            ctx.save_for_backward(w, x)
        elif ctx.needs_input_grad[1] or (bias is not None and ctx.needs_input_grad[2]):
            a = act8_pack(x)
            ctx.save_for_backward(w, a.codes, a.exponents)
        else:
            ctx.save_for_backward(w)   # nothing will read x
        ctx.conf = (tuple(stride), tuple(pad), tpad, bias is not None, residual is not None)
        ctx.x_shape = tuple(x.shape)
        return y

    @staticmethod
    @_differentiable_once
    def backward(ctx, dy):
        w, *saved = ctx.saved_tensors
        stride, pad, tpad, has_bias, has_res = ctx.conf
        dy = dy.contiguous()
        dx = dw = db = dres = None
        if ctx.needs_input_grad[0]:
            if stride[0] != 1:
                raise NotImplementedError("the input gradient supports temporal stride 1 only")
            dx = conv3d_bwd_data(dy, w, ctx.x_shape, pad, tpad, stride=stride)
        if ctx.needs_input_grad[1] or (has_bias and ctx.needs_input_grad[2]):
            x = saved[0] if len(saved) == 1 else act8_unpack(Act8(*saved, ctx.x_shape[-1]), w.dtype)
            dw, db = conv3d_bwd_weight(x, dy, tuple(w.shape[1:4]), stride, pad, tpad,
                                       with_bias=has_bias)
            if not ctx.needs_input_grad[1]:
                dw = None
        if has_res and ctx.needs_input_grad[3]:
            dres = dy
        return dx, dw, db, dres, None, None, None, None


def conv3d_autograd(x, w, bias=None, residual=None, stride=(1, 1, 1), pad=(0, 1, 1),
                    tpad=TPAD_CAUSAL_REPLICATE, checkpoint8=False):
    """y = conv3d(x, w) + bias + residual with gradients for x, w, bias and residual.
    checkpoint8: keep x for the weight gradient in 8 bits (1.03 bytes a value); where neither
    w nor bias needs a gradient, or none is recorded, nothing is kept of x."""
    return Conv3dFunction.apply(x, w, bias, residual, tuple(stride), tuple(pad), tpad,
                                checkpoint8 and torch.is_grad_enabled())


# ---------------------------------------------------------------- channel-wise operators
#
# Tensors are [..., C], contiguous, bf16 or fp16; every leading extent counts as
# rows.  All tensors of a call live on one CUDA device, which need not be the
# current one; the default stream is that device's current stream.  The calls go
# through the native binding, which checks the operands (ValueError, TypeError),
# allocates the outputs and raises Conv3dError for a status of the library.


def layernorm_fwd_ptr(x, gamma, beta, y, mean, rstd, codes, exponents, rows, C, eps, dtype, stream) -> int:
    """Raw-pointer call of conv3d_layernorm_fwd; returns the status code."""
    return _lib.conv3d_layernorm_fwd(x, gamma, beta, y, mean, rstd, codes, exponents, rows, C, eps, dtype, stream)


def layernorm_bwd_ptr(dy, x, mean, codes, exponents, rstd, gamma, dres, dx, dgamma, dbeta, rows, C, dtype,
                      workspace, ws_bytes, stream) -> int:
    """Raw-pointer call of conv3d_layernorm_bwd; returns the status code."""
    return _lib.conv3d_layernorm_bwd(dy, x, mean, codes, exponents, rstd, gamma, dres, dx, dgamma, dbeta, rows, C,
                                     dtype, workspace, ws_bytes, stream)


def layernorm_bwd_workspace_bytes(rows: int, C: int) -> int:
    return int(_lib.conv3d_layernorm_bwd_workspace_bytes(rows, C))


def act8_pack_ptr(x, codes, exponents, rows, C, dtype, stream) -> int:
    """Raw-pointer call of conv3d_act8_pack; returns the status code."""
    return _lib.conv3d_act8_pack(x, codes, exponents, rows, C, dtype, stream)


def act8_unpack_ptr(codes, exponents, gamma, beta, act, y, rows, C, dtype, stream) -> int:
    """Raw-pointer call of conv3d_act8_unpack; returns the status code."""
    return _lib.conv3d_act8_unpack(codes, exponents, gamma, beta, act, y, rows, C, dtype, stream)


def act8_bwd_ptr(dy, codes, exponents, act, dx, rows, C, dtype, stream) -> int:
    """Raw-pointer call of conv3d_act8_bwd; returns the status code."""
    return _lib.conv3d_act8_bwd(dy, codes, exponents, act, dx, rows, C, dtype, stream)


def linear_fwd_ptr(x, w, bias, residual, y, codes, exponents, rows, K, N, act, dtype, stream) -> int:
    """Raw-pointer call of conv3d_linear_fwd; returns the status code."""
    return _lib.conv3d_linear_fwd(x, w, bias, residual, y, codes, exponents, rows, K, N, act, dtype, stream)


def linear_bwd_data_ptr(dy, w, codes, exponents, act, dx, x, rows, K, N, dtype, stream) -> int:
    """Raw-pointer call of conv3d_linear_bwd_data; returns the status code."""
    return _lib.conv3d_linear_bwd_data(dy, w, codes, exponents, act, dx, x, rows, K, N, dtype, stream)


def linear_bwd_weight_ptr(x, dy, dw, dbias, rows, K, N, dtype, workspace, ws_bytes, stream) -> int:
    """Raw-pointer call of conv3d_linear_bwd_weight; returns the status code."""
    return _lib.conv3d_linear_bwd_weight(x, dy, dw, dbias, rows, K, N, dtype, workspace, ws_bytes, stream)


def linear_bwd_weight_workspace_bytes(rows: int, K: int, N: int) -> int:
    return int(_lib.conv3d_linear_bwd_weight_workspace_bytes(rows, K, N))


class Act8(NamedTuple):
    """An 8-bit activation checkpoint of a [..., C] tensor: int8 codes
    [..., 32 * ceil(C/32)] and uint8 exponents [..., ceil(C/32)] (conv3d.h)."""
    codes: torch.Tensor
    exponents: torch.Tensor
    channels: int

    @staticmethod
    def empty(shape, device) -> "Act8":
        """An uninitialised checkpoint of a tensor of ``shape``."""
        blocks = -(-shape[-1] // 32)
        lead = tuple(shape[:-1])
        return Act8(torch.empty((*lead, blocks * 32), dtype=torch.int8, device=device),
                    torch.empty((*lead, blocks), dtype=torch.uint8, device=device), int(shape[-1]))


def _on(stream):
    """A stream argument for the native binding: None is the device's current stream."""
    return None if stream is None else _stream_handle(stream)


def act8_pack(x: torch.Tensor, stream=None) -> Act8:
    """The 8-bit checkpoint of x [..., C]."""
    codes, exponents = _channel.act8_pack(x, _on(stream))
    return Act8(codes, exponents, x.shape[-1])


def act8_unpack(a: Act8, dtype: torch.dtype, gamma=None, beta=None, act: int = ACT_NONE,
                y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """act(v * gamma + beta) of the checkpoint's values v, as a ``dtype`` tensor."""
    return _channel.act8_unpack(a[0], a[1], a[2], dtype, gamma, beta, act, y, _on(stream))


def act8_bwd(dy: torch.Tensor, a: Act8, act: int, dx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dy * act'(v) of the checkpoint's values v (``dx`` may be ``dy``)."""
    return _channel.act8_bwd(dy, a[0], a[1], a[2], act, dx, _on(stream))


def layernorm(x: torch.Tensor, gamma=None, beta=None, eps: float = 1e-6, with_stats: bool = False,
              checkpoint8: bool = False, y: torch.Tensor | None = None, stream=None):
    """y = (x - mean) * rstd * gamma + beta over the last axis of x [..., C].

    Returns y; with ``with_stats`` (y, mean, rstd), fp32 [...]; with
    ``checkpoint8`` (y, xhat, rstd), xhat the :class:`Act8` of (x - mean) * rstd:
    either is what :func:`layernorm_bwd` needs.  ``y`` may be ``x``.
    """
    out = _channel.layernorm(x, gamma, beta, eps, with_stats, checkpoint8, y, _on(stream))
    return (out[0], Act8(out[1], out[2], x.shape[-1]), out[3]) if checkpoint8 else out


def layernorm_bwd(dy: torch.Tensor, saved, rstd: torch.Tensor, mean: torch.Tensor | None = None, gamma=None,
                  dres=None, with_params: bool = True, dx: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None):
    """(dx, dgamma, dbeta) of :func:`layernorm`; dgamma and dbeta are None without ``with_params``.

    saved: x (then ``mean`` is needed) or the :class:`Act8` of the normalised x.
    dres: added to dx (the gradient of a skip connection around the norm).
    ``dx`` may be ``dy``, ``dres`` or x.
    """
    x, a = (None, saved) if isinstance(saved, Act8) else (saved, (None, None, 0))
    return _channel.layernorm_bwd(dy, x, mean, a[0], a[1], a[2], rstd, gamma, dres, with_params, dx, workspace,
                                  _on(stream))


def linear(x: torch.Tensor, w: torch.Tensor, bias=None, residual=None, act: int = ACT_NONE,
           checkpoint8: bool = False, y: torch.Tensor | None = None, stream=None):
    """y = act(x w^T + bias) + residual for x [..., K], w [N, K] (or [N, 1, 1, 1, K]).

    With ``checkpoint8`` returns (y, pre): pre is the :class:`Act8` of x w^T + bias.
    ``y`` may be ``residual``.
    """
    out = _channel.linear(x, w, bias, residual, act, checkpoint8, y, _on(stream))
    return (out[0], Act8(out[1], out[2], w.shape[0])) if checkpoint8 else out


def linear_bwd_data(dy: torch.Tensor, w: torch.Tensor, pre: Act8 | None = None, act: int = ACT_NONE,
                    dx: torch.Tensor | None = None, with_x: bool = False, stream=None):
    """dx = (dy w) * act'(pre) for dy [..., N], w [N, K]: the gradient of x, or, with the
    checkpoint ``pre`` of what ``act`` was applied to (x = act(pre)), of that argument.
    ``with_x`` returns (dx, x): act8_unpack's x, for the weight gradient, in the same pass."""
    a = pre if pre is not None else (None, None, 0)
    dx, x = _channel.linear_bwd_data(dy, w, a[0], a[1], a[2], act, dx, with_x, _on(stream))
    return (dx, x) if with_x else dx


def linear_bwd_weight(x: torch.Tensor, dy: torch.Tensor, with_bias: bool = True,
                      workspace: torch.Tensor | None = None, stream=None):
    """(dw [N, K], dbias [N]) of :func:`linear` without activation (dbias is None without
    ``with_bias``): fp32 sums in a fixed order, so the same inputs give the same bits."""
    return _channel.linear_bwd_weight(x, dy, with_bias, workspace, _on(stream))


class ChannelMlpSaved(NamedTuple):
    """What :func:`channel_mlp` keeps for its backward pass, beside the weights:
    the checkpoints of the normalised input and of the pre-activation."""
    xhat: Act8
    rstd: torch.Tensor
    pre: Act8


def channel_mlp(x: torch.Tensor, gamma, beta, w1: torch.Tensor, b1, w2: torch.Tensor, b2, act: int = ACT_GELU,
                eps: float = 1e-6, save: bool = False, stream=None):
    """y = x + act(layernorm(x) w1^T + b1) w2^T + b2 over the channels of x [..., C];
    w1 [H, C], w2 [C, H].  With ``save`` returns (y, :class:`ChannelMlpSaved`): about
    1.03 (C + H) bytes a row in place of the 16-bit activations (2 (2C + 2H))."""
    if not save:
        n = layernorm(x, gamma, beta, eps, stream=stream)
        return linear(linear(n, w1, b1, None, act, stream=stream), w2, b2, x, stream=stream)
    n, xhat, rstd = layernorm(x, gamma, beta, eps, checkpoint8=True, stream=stream)
    h, pre = linear(n, w1, b1, None, act, checkpoint8=True, stream=stream)
    return linear(h, w2, b2, x, stream=stream), ChannelMlpSaved(xhat, rstd, pre)


def channel_mlp_bwd(dy: torch.Tensor, saved: ChannelMlpSaved, gamma, beta, w1: torch.Tensor, w2: torch.Tensor,
                    act: int = ACT_GELU, stream=None):
    """(dx, dgamma, dbeta, dw1, db1, dw2, db2) of :func:`channel_mlp` from its checkpoints.

    The two inputs that the weight gradients need are recomputed from the
    checkpoints: the activation by the product dy w2, whose epilogue reads them for
    act' (:func:`linear_bwd_data`), the normalised input by a pass of its own.  The
    skip connection's gradient rides in the layer norm's.
    While the call runs it holds the activation and its gradient, 4 H bytes a row, then the
    gradient and the normalised input, whose place dx takes, 2 H + 2 C: at most max(4 H, 2 H +
    2 C) bytes a row, the weight gradients, and a workspace of :func:`linear_bwd_weight`
    (linear_bwd_weight_workspace_bytes).

    What goes into the products is rounded to 16 bits: the two recomputed inputs, the hidden
    activation's gradient and the normalised input's.  From the same checkpoints the bf16
    results are off by about 0.003 of their norm, their own rounding being 0.0017 of it.
    """
    x, pre = saved.xhat, saved.pre
    return _channel.channel_mlp_bwd(dy, x[0], x[1], x[2], saved.rstd, pre[0], pre[1], pre[2], gamma, beta, w1, w2, act,
                                    _on(stream))


class LayerNormFunction(torch.autograd.Function):
    """torch.autograd wrapper of layernorm; with checkpoint8 it keeps the 8-bit
    normalised input instead of x."""

    @staticmethod
    def forward(ctx, x, gamma, beta, eps, checkpoint8):
        if checkpoint8:
            y, a, rstd = layernorm(x, gamma, beta, eps, checkpoint8=True)
            ctx.save_for_backward(gamma, rstd, a.codes, a.exponents)
        else:
            y, mean, rstd = layernorm(x, gamma, beta, eps, with_stats=True)
            ctx.save_for_backward(gamma, rstd, x, mean)
        ctx.conf = (checkpoint8, x.shape[-1])
        return y

    @staticmethod
    @_differentiable_once
    def backward(ctx, dy):
        gamma, rstd, s0, s1 = ctx.saved_tensors
        checkpoint8, C = ctx.conf
        saved, mean = (Act8(s0, s1, C), None) if checkpoint8 else (s0, s1)
        need = ctx.needs_input_grad
        dx, dgamma, dbeta = layernorm_bwd(dy.contiguous(), saved, rstd, mean, gamma, with_params=need[1] or need[2])
        return dx if need[0] else None, dgamma if need[1] else None, dbeta if need[2] else None, None, None


def layernorm_autograd(x, gamma=None, beta=None, eps: float = 1e-6, checkpoint8: bool = False):
    """layernorm with gradients for x, gamma and beta."""
    return LayerNormFunction.apply(x, gamma, beta, eps, checkpoint8)


class LinearFunction(torch.autograd.Function):
    """torch.autograd wrapper of linear.  With an activation the pre-activation
    is kept as an 8-bit checkpoint."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, act):
        if act != ACT_NONE:
            y, a = linear(x, w, bias, residual, act, checkpoint8=True)
            ctx.save_for_backward(x, w, a.codes, a.exponents)
        else:
            y = linear(x, w, bias, residual, act)
            ctx.save_for_backward(x, w)
        ctx.conf = (act, bias is not None, residual is not None)
        return y

    @staticmethod
    @_differentiable_once
    def backward(ctx, dy):
        x, w, *a = ctx.saved_tensors
        act, has_bias, has_res = ctx.conf
        dy = dy.contiguous()
        need = ctx.needs_input_grad
        dx = dw = db = None
        if need[0] or need[1] or (has_bias and need[2]):
            dpre = act8_bwd(dy, Act8(a[0], a[1], w.shape[0]), act) if act != ACT_NONE else dy
            if need[0]:
                dx = linear_bwd_data(dpre, w)
            if need[1] or (has_bias and need[2]):
                dw, db = linear_bwd_weight(x, dpre, with_bias=has_bias)
                dw = dw.view(w.shape) if need[1] else None
        return dx, dw, db if has_bias and need[2] else None, dy if has_res and need[3] else None, None


def linear_autograd(x, w, bias=None, residual=None, act: int = ACT_NONE):
    """y = act(x w^T + bias) + residual with gradients for x, w, bias and residual.
    With an activation act' is taken at the 8-bit checkpoint of x w^T + bias (off by at most
    1/64 of the largest magnitude in its block of 32 channels), which is what is kept of it."""
    return LinearFunction.apply(x, w, bias, residual, act)


class ChannelMlpFunction(torch.autograd.Function):
    """torch.autograd wrapper of channel_mlp: between forward and backward it keeps
    the two checkpoints, rstd and the weights, no 16-bit activation."""

    @staticmethod
    def forward(ctx, x, gamma, beta, w1, b1, w2, b2, act, eps):
        y, s = channel_mlp(x, gamma, beta, w1, b1, w2, b2, act, eps, save=True)
        ctx.save_for_backward(gamma, beta, w1, w2, s.xhat.codes, s.xhat.exponents, s.rstd, s.pre.codes,
                              s.pre.exponents)
        ctx.conf = (act, x.shape[-1], w1.shape[0], b1 is not None, b2 is not None)
        return y

    @staticmethod
    @_differentiable_once
    def backward(ctx, dy):
        gamma, beta, w1, w2, qc, qe, rstd, pc, pe = ctx.saved_tensors
        act, C, H, has_b1, has_b2 = ctx.conf
        dx, dg, dbt, dw1, db1, dw2, db2 = channel_mlp_bwd(
            dy.contiguous(), ChannelMlpSaved(Act8(qc, qe, C), rstd, Act8(pc, pe, H)), gamma, beta, w1, w2, act)
        grads = (dx, dg if gamma is not None else None, dbt if beta is not None else None, dw1.view(w1.shape),
                 db1 if has_b1 else None, dw2.view(w2.shape), db2 if has_b2 else None)
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad)) + (None, None)


def channel_mlp_autograd(x, gamma, beta, w1, b1, w2, b2, act: int = ACT_GELU, eps: float = 1e-6):
    """channel_mlp with gradients for x, gamma, beta, w1, b1, w2 and b2, taken at the 8-bit
    checkpoints of the normalised input and the pre-activation (each value off by at most 1/64
    of the largest magnitude in its block of 32 channels): see :func:`channel_mlp_bwd`."""
    return ChannelMlpFunction.apply(x, gamma, beta, w1, b1, w2, b2, act, eps)
