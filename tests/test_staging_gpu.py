"""Output staging of the convolution's epilogues across tiles.

An epilogue warp stages its 32-column chunks in two buffers in turn while the
TMA store of the chunk before may still read the other.  The turn has to go on
from tile to tile: where a warp has an odd number of chunks in a tile (32 or 96
output channels, one or three; two chunks split over eight epilogue warps; a
transposed tile clipped at its frame's end), a turn that began anew would hand
the next tile's first chunk the buffer of the store just issued.  Pointwise
layers with few input channels follow their tiles fastest; every persistent
block here walks at least four, and every element is compared.

Tolerance: the output's one rounding, eps / 2 of the value, and the fp32 sums:
Cin products, the bias and the residual, one rounding of at most 2^-24 of the
sum of their magnitudes each.
"""
import pytest
import torch

import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CASES = [
    # swap, epi8, (D, H, W, Cin, Cout, dtype, residual)
    ("0", "0", (4, 128, 160, 64, 32, "bf16", False)),    # one chunk a tile
    ("0", "0", (4, 128, 160, 64, 96, "bf16", True)),     # three
    ("0", "1", (4, 128, 160, 64, 64, "bf16", True)),     # two, one for each warp of a pair
    ("0", "1", (4, 128, 160, 64, 32, "f16", False)),     # one for the first, none for the second
    ("0", "1", (4, 128, 160, 32, 160, "bf16", False)),   # three and two
    ("1", "0", (640, 8, 12, 64, 128, "bf16", True)),     # transposed, frames of three pixel chunks
    ("1", "1", (640, 8, 12, 64, 128, "f16", False)),     # two and one
    ("1", "0", (640, 4, 8, 64, 128, "bf16", False)),     # one
]


@pytest.mark.parametrize("swap,epi8,case", CASES, ids=lambda c: c if isinstance(c, str) else "x".join(map(str, c)))
def test_odd_chunks_over_many_tiles(swap, epi8, case, monkeypatch):
    monkeypatch.setenv("CONV3D_SWAP", swap)
    monkeypatch.setenv("CONV3D_EPI8", epi8)
    monkeypatch.setenv("CONV3D_SPLIT", "0")
    monkeypatch.setenv("CONV3D_CTA_PAIR", "0")
    D, H, W, Cin, Cout, dt, res = case
    dtype = TYPES[dt]
    x = si.tensor((1, D, H, W, Cin), 71, 0, 1.0, dtype, "cuda")
    w = si.tensor((Cout, 1, 1, 1, Cin), 71, 1, Cin ** -0.5, dtype, "cuda")
    b = si.tensor((Cout,), 71, 2, 1.0, dtype, "cuda")
    r = si.tensor((1, D, H, W, Cout), 71, 3, 1.0, dtype, "cuda") if res else None
    y = torch.empty((1, D, H, W, Cout), dtype=dtype, device="cuda")
    wd = w.double().view(Cout, Cin)
    ref = x.double() @ wd.T + b.double()
    size = x.double().abs() @ wd.abs().T + b.double().abs()
    if res:
        ref += r.double()
        size += r.double().abs()
    bound = ref.abs() * (torch.finfo(dtype).eps / 2) + size * ((Cin + 2) * 2.0 ** -24) * 1.01
    for _ in range(4):
        y.fill_(float("nan"))
        c3.conv3d_fwd(x, w, b, r, y, (1, 1, 1), (0, 0, 0), c3.TPAD_ZERO)
        assert c3.poll_status() == c3.Status.OK
        wrong = ~((y.double() - ref).abs() <= bound)
        assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:4].tolist())
