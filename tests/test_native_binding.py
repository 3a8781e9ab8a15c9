"""The package where the native binding of the channel-wise operators does not load,
and when the binding is built again."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
class Refuse:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._channel"):
            raise ImportError("built against another torch")
sys.meta_path.insert(0, Refuse())
import torch
import video_vae_convolution_implicit_b200 as c3
# the convolution's calls are there, down to the library
assert c3.output_shape(9, 16, 16, (3, 3, 3)) == (9, 16, 16)
assert c3.kernel_launches() == 0 and callable(c3.conv3d) and callable(c3.conv3d_autograd)
x = torch.zeros(4, 64, dtype=torch.bfloat16)
for call in (lambda: c3.layernorm(x), lambda: c3.act8_pack(x), lambda: c3.linear(x, x),
             lambda: c3.linear_bwd_weight(x, x), lambda: c3.channel_mlp(x, None, None, x, None, x.T, None)):
    try:
        call()
    except ImportError as e:
        assert "_channel.so" in str(e) and "another torch" in str(e.__cause__), (e, e.__cause__)
    else:
        raise AssertionError("no error without the binding")
"""


def test_convolution_works_without_the_binding():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.fixture
def builder(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location(
        "_builder", os.path.join(ROOT, "video_vae_convolution_implicit_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / "_channel.so"))
    monkeypatch.setattr(mod, "BUILT_FOR", str(tmp_path / "built_for"))
    return mod


def test_binding_is_stale_for_another_torch(builder):
    assert builder.binding_stale()                  # no binding
    open(builder.BINDING, "w").close()
    assert builder.binding_stale()                  # one of unknown origin
    with open(builder.BUILT_FOR, "w") as f:
        f.write(builder.binding_target())
    assert not builder.binding_stale()
    with open(builder.BUILT_FOR, "w") as f:
        f.write("torch 1.0, Python 3.12.3\n")
    assert builder.binding_stale()
