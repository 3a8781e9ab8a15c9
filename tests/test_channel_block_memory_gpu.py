"""The channel MLP block with more channels than hidden ones, and what its backward
pass holds while it runs."""
import pytest
import torch

import video_vae_convolution_implicit_b200 as c3
from test_channel_block_gpu import (block, rand, test_block_autograd_against_the_formula_and_differences,
                                    test_block_backward_from_given_checkpoints, test_block_forward)

pytestmark = pytest.mark.gpu

NARROW = [(1, 128, 64), (41, 200, 72), (700, 512, 256)]
_forward, _backward, _autograd = (test_block_forward, test_block_backward_from_given_checkpoints,
                                  test_block_autograd_against_the_formula_and_differences)
del test_block_forward, test_block_backward_from_given_checkpoints, test_block_autograd_against_the_formula_and_differences


@pytest.mark.parametrize("rows,C,H", NARROW)
def test_narrow_block(rows, C, H):
    for act in (c3.ACT_SILU, c3.ACT_GELU):
        _forward(rows, C, H, act)
        _backward(rows, C, H, act)
    _autograd(rows, C, H)


@pytest.mark.parametrize("rows,C,H", [(20000, 1024, 256), (20000, 256, 1024), (20000, 512, 512)])
def test_memory_of_the_backward_pass(rows, C, H):
    p = block(rows, C, H, 31)
    _, saved = c3.channel_mlp(**p, save=True)
    dy = rand((rows, C), 31, 7)

    def run():
        return c3.channel_mlp_bwd(dy, saved, p["gamma"], p["beta"], p["w1"], p["w2"])
    run()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = run()
    torch.cuda.synchronize()
    peak = torch.cuda.max_memory_allocated() - before
    held = rows * max(4 * H, 2 * H + 2 * C)
    workspace = max(c3.linear_bwd_weight_workspace_bytes(rows, H, C), c3.linear_bwd_weight_workspace_bytes(rows, C, H),
                    c3.layernorm_bwd_workspace_bytes(rows, C))
    weights = sum(t.numel() * 2 for t in out[1:])
    # torch's allocator may give a large request up to 1 MiB more than it asked for
    assert held < peak <= held + workspace + weights + len(out) * 2 ** 20, (peak, held, workspace, weights)
