"""Which CUDA context a call leaves current in its thread.

A call binds the device's primary context only in a thread that has none: one
that left its context is bound again, and a context that the thread has made
current stays current.  Each case runs in a process of its own.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import ctypes, threading
import torch
import video_vae_convolution_implicit_b200 as c3
cu = ctypes.CDLL("libcuda.so.1")
def current():
    c = ctypes.c_void_p()
    assert cu.cuCtxGetCurrent(ctypes.byref(c)) == 0
    return c.value
x = torch.randn(64, 64, device="cuda").bfloat16()
w = torch.randn(64, 64, device="cuda").bfloat16()
y = torch.zeros(64, 64, device="cuda").bfloat16()
want = c3.linear(x, w)
torch.cuda.synchronize()
primary = current()
def call():
    return c3.linear_fwd_ptr(x.data_ptr(), w.data_ptr(), None, None, y.data_ptr(), None, None, 64, 64, 64,
                             c3.ACT_NONE, c3.BF16, 0)
failed = []
def run(work):
    def guarded():
        try:
            work()
        except BaseException as e:
            failed.append(repr(e))
    t = threading.Thread(target=guarded)
    t.start()
    t.join()
    assert not failed, failed
"""

LEFT = PRELUDE + """
def work():
    assert call() == 0, c3.last_error()
    assert current() == primary
    assert cu.cuCtxSetCurrent(None) == 0 and current() is None
    assert call() == 0, c3.last_error()
    assert current() == primary
run(work)
torch.cuda.synchronize()
assert torch.equal(y, want)
"""

# The call of the own context's thread is one that the host refuses after it has
# looked at the device (more tiles than the kernel can count): nothing is
# launched, and its addresses are not read.
OWN = PRELUDE + """
def work():
    own = ctypes.c_void_p()
    assert cu.cuCtxCreate_v2(ctypes.byref(own), 0, 0) == 0
    assert current() == own.value != primary
    st = c3.linear_fwd_ptr(1 << 40, 1 << 44, None, None, 1 << 54, None, None, 2 ** 31 - 65600, 8, 2 ** 21,
                           c3.ACT_NONE, c3.BF16, 0)
    assert st == c3.Status.UNSUPPORTED and "tile indexing" in c3.last_error(), (st, c3.last_error())
    kept = current()
    assert cu.cuCtxDestroy_v2(own) == 0
    assert kept == own.value, (kept, own.value, primary)
run(work)
assert call() == 0
torch.cuda.synchronize()
assert torch.equal(y, want)
"""


@pytest.mark.parametrize("script", [LEFT, OWN], ids=["left", "own"])
def test_current_context(script):
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-500:] + r.stderr[-2000:]
