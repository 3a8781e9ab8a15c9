"""Memory of the channel-wise calls on CUDA's handles of the default streams.

Handle 1 is the legacy default stream (torch's 0) and handle 2 the calling
thread's.  Torch's other streams are not ordered against either, so what a call
allocates and frees must not be handed to the current stream while the call's
kernels are still to run.
"""
import pytest
import torch

import seeded_inputs as si
import video_vae_convolution_implicit_b200 as c3

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(shape, k, scale=1.0):
    return si.tensor(shape, 81, k, scale, BF, "cuda")


def _weight_gradient(handle):
    x, dy = rand((4096, 256), 0), rand((4096, 256), 1)
    need = c3.linear_bwd_weight_workspace_bytes(4096, 256, 256)
    return need, lambda: c3.linear_bwd_weight(x, dy, stream=handle)


def _layer_norm_gradient(handle):
    x, dy, g = rand((4096, 512), 2), rand((4096, 512), 3), rand((512,), 4)
    _, mean, rstd = c3.layernorm(x, g, None, with_stats=True)
    need = c3.layernorm_bwd_workspace_bytes(4096, 512)
    return need, lambda: c3.layernorm_bwd(dy, x, rstd, mean, g, stream=handle)


def _block(handle):
    x, dy = rand((4096, 256), 5), rand((4096, 256), 6)
    g, b = rand((256,), 7), rand((256,), 8)
    w1, w2 = rand((512, 256), 9, 0.06), rand((256, 512), 10, 0.04)
    _, saved = c3.channel_mlp(x, g, b, w1, None, w2, None, save=True)
    return 4096 * 512 * 2, lambda: c3.channel_mlp_bwd(dy, saved, g, b, w1, w2, stream=handle)


@pytest.mark.parametrize("handle", [0, 1, 2])
@pytest.mark.parametrize("make", [_weight_gradient, _layer_norm_gradient, _block])
def test_freed_memory_is_not_lent_early(make, handle):
    need, call = make(handle)
    assert need > 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        expected = call()                       # the pools hold blocks of these sizes from here on
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(torch.cuda.default_stream()):
                torch.cuda._sleep(20_000_000)   # about 10 ms; both default streams wait for it
            got = call()
            # the side stream does not wait for the sleep: what it gets now, it fills now
            mine = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
            torch.cuda.synchronize()
            assert all(bool((t == 7).all()) for t in mine)
            assert all(torch.equal(a, b) for a, b in zip(expected, got))
            del mine, got
    assert c3.poll_status() == c3.Status.OK


def test_thread_stream_follows_and_is_followed():
    """Handle 2: the call waits for the current stream's work, whose memory it uses, and
    the current stream's next work waits for the call."""
    x, w = rand((2048, 256), 11), rand((256, 256), 12, 0.06)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = c3.linear(x, w)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        x2 = x * 2                              # runs after the sleep
        z = c3.linear(x2, w, stream=2)
        total = (z == y * 2).all()              # on the side stream, without a synchronisation
        side.synchronize()
        assert bool(total)
    assert c3.poll_status() == c3.Status.OK
