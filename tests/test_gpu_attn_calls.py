"""Calls of the attention step on the GPU that its documentation allows and
that test_gpu_attn.py does not make; its cases and bounds are used here."""
import pytest
import torch

from gpu_harness import torch_dev
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("q_len", [1, 90])
def test_stream_without_buffers(q_len, raw):
    """A call on a stream of the caller's that makes its own result and workspace, while the current stream is busy and
    goes on to allocate and overwrite blocks of the same sizes."""
    dev = torch_dev()
    c = Case([(q_len, 3000), (q_len, 257), (1, 5000)], 16, 2, 128, 64, rope=(128, "half", "none", 1.0), seed=31)
    want = c.run()
    turned = c.rope.apply(c.q, c.positions)
    size = c.cache.attention_workspace(16).numel()
    side = torch.cuda.Stream(dev)
    busy = torch.randn((4096, 4096), device=dev)
    torch.cuda.synchronize()
    for _ in range(10):
        for _ in range(4):
            busy @ busy  # the current stream is behind the calls on the other one
        with torch.cuda.stream(side):
            busy @ busy  # and that one behind the host
        stream = side.cuda_stream if raw else side
        got = c.run(stream=stream)
        rows = c.rope.apply(c.q, c.positions, stream=stream)
        for _ in range(3):  # blocks that were free, or have just been given back
            torch.empty(size, dtype=torch.uint8, device=dev).fill_(0xFF)
            torch.empty_like(want).fill_(float("nan"))
        side.synchronize()
        assert same_bits(got, want)
        assert same_bits(rows, turned)
        torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 5, 70])
@pytest.mark.parametrize("window", [1, 21, 150])
def test_garbage_in_front_of_the_window(D, q_len, window):
    """Positions in front of the first query's window may hold anything: not-a-number and infinite scales on the page
    and in the tile where the window begins never count."""
    c = Case([(q_len, 333), (q_len, 100 + q_len), (q_len, 512)], 8, 2, D, 16, window=window, seed=D + window)
    live = torch.zeros((c.cache.n_pages, c.page), dtype=torch.bool, device=torch_dev())
    for b, L in enumerate(c.lens.tolist()):
        for j in range(max(L - q_len - window + 1, 0), L):
            live[int(c.table[b, j // c.page]), j % c.page] = True
    assert not bool(live.all())
    for i, poison in ((1, float("nan")), (3, float("inf"))):
        t = c.cache.tensors[i]
        t.copy_(torch.where(live[:, None, :, None], t, torch.full_like(t, poison)))
    c.cache.tensors[3][..., 0].masked_fill_(~live[:, None], float("nan"))
    c.check()
