"""Memory of the convolution and GroupNorm calls on a stream that is not the current one.

The workspaces of the gradients go back to torch's allocator when the call returns, and
its outputs come from it: both have to belong to the stream the kernels run on, or the
current stream's next tensors share their memory while the kernels are still to run.
"""
import pytest
import torch

import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SHAPE = (1, 3, 32, 32, 64)
K = (3, 3, 3)


def rand(shape, k, scale=1.0):
    return si.tensor(shape, 61, k, scale, BF, "cuda")


def _calls():
    """name: (bytes of a workspace or output, call(stream) -> tensors that repeat exactly)"""
    x, w, dy, b = rand(SHAPE, 0), rand((64, *K, 64), 1, 0.025), rand(SHAPE, 2), rand((64,), 3)
    prev, first = rand((1, 2, 32, 32, 64), 4), rand((1, 1, 32, 32, 64), 5)
    stats = c3.groupnorm_stats(x, 8)
    pad = (0, 1, 1)
    act = x.numel() * 2
    return {
        "conv3d": (act, lambda s: c3.conv3d(x, w, b, stream=s)),
        "conv3d_gn": (act, lambda s: c3.conv3d_gn(x, stats, None, None, w, b, stream=s)),
        "groupnorm_silu": (act, lambda s: c3.groupnorm_silu(x, stats, stream=s)),
        "conv3d_bwd_data": (c3.bwd_data_workspace_bytes(1, 64, 3, 32, 32, 64, K, pad, c3.TPAD_CAUSAL_REPLICATE),
                            lambda s: c3.conv3d_bwd_data(dy, w, SHAPE, stream=s)),
        "conv3d_bwd_weight": (c3.bwd_weight_workspace_bytes(64, 64, K),
                              lambda s: c3.conv3d_bwd_weight(x, dy, K, stream=s)[0]),
        "conv3d_bwd_data_cached": (act, lambda s: c3.conv3d_bwd_data_cached(dy, w, SHAPE, stream=s)[0]),
        "conv3d_bwd_weight_cached": (c3.bwd_weight_workspace_bytes(64, 64, K),
                                     lambda s: c3.conv3d_bwd_weight_cached(x, prev, dy, K, stream=s)[0]),
        "first frame": (first.numel() * 2, lambda s: c3.conv3d(first, w, b, stream=s)),
    }


NAMES = ["conv3d", "conv3d_gn", "groupnorm_silu", "conv3d_bwd_data", "conv3d_bwd_weight", "conv3d_bwd_data_cached",
         "conv3d_bwd_weight_cached", "first frame"]


@pytest.mark.parametrize("where", ["stream", "handle", 0, 1, 2])
@pytest.mark.parametrize("name", NAMES)
def test_freed_memory_is_not_lent_early(name, where):
    need, call = _calls()[name]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    busy = other if where in ("stream", "handle") else torch.cuda.default_stream()
    stream = other if where == "stream" else other.cuda_stream if where == "handle" else where
    with torch.cuda.stream(side):
        expected = call(stream)
        torch.cuda.synchronize()
        del expected                                # the pools hold blocks of these sizes from here on
        expected = call(stream)
        torch.cuda.synchronize()
        for _ in range(2):
            with torch.cuda.stream(busy):
                torch.cuda._sleep(20_000_000)       # about 10 ms (both default streams wait for it)
            got = call(stream)
            # the side stream does not wait for the sleep: what it gets now, it fills now
            mine = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
            torch.cuda.synchronize()
            assert all(bool((t == 7).all()) for t in mine)
            if "weight" in name:                    # fp32 atomics: the order of the sums varies
                torch.testing.assert_close(got, expected, rtol=2.0 ** -6, atol=2e-2)
            else:
                assert torch.equal(got, expected)
            del mine, got
    assert c3.poll_status() == c3.Status.OK
