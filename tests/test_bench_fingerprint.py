"""The fingerprint that bench.py's DRAM figures are keyed to covers the whole kernel."""
import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "video_vae_convolution_implicit_b200", "csrc")


def test_fingerprint_covers_every_header_of_the_kernel():
    found, todo = set(), ["conv3d_kernel.cuh"]
    while todo:
        name = todo.pop()
        if name in found:
            continue
        found.add(name)
        with open(os.path.join(CSRC, name)) as f:
            included = re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M)
        todo += [i for i in included if os.path.exists(os.path.join(CSRC, i))]
    assert "pipeline.cuh" in found and set(bench.KERNEL_SOURCES) == found


def test_fingerprint_changes_with_each_header(tmp_path, monkeypatch):
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    folder = tmp_path / "video_vae_convolution_implicit_b200" / "csrc"
    folder.mkdir(parents=True)
    for name in bench.KERNEL_SOURCES:
        (folder / name).write_text(name)
    seen = {bench.kernel_source_hash()}
    for name in bench.KERNEL_SOURCES:
        (folder / name).write_text(name + " changed")
        seen.add(bench.kernel_source_hash())
    assert len(seen) == 1 + len(bench.KERNEL_SOURCES)
