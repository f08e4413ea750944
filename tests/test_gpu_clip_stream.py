"""Clipping queued on a busy stream that is not current, with one launch and with two."""
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("sizes", [(1000, 70), (300000, 70001)])
def test_clipping_behind_a_busy_stream_that_is_not_current(sizes, as_handle):
    """The gradients are written on the side stream behind 6 ms of products: a launch anywhere
    else would read and scale what they were before."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    real = [torch.randn(n, generator=gen, device="cuda").to(t) for n, t in zip(sizes, (BF, F32))]
    want = [torch.empty_like(g) for g in real]
    norm = gmm.clip_grads(real, 0.5, out=want)
    grads, out = [torch.full_like(g, 3.0) for g in real], [torch.zeros_like(g) for g in real]
    busy = torch.zeros((2, 8192, 8192), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):
            torch.mm(busy[0], busy[0], out=busy[1])
        for g, r in zip(grads, real):
            g.copy_(r)
    got = gmm.clip_grads(grads, 0.5, out=out, stream=side.cuda_stream if as_handle else side)
    # what the current stream takes and writes now must not be the call's memory
    junk = [torch.full((1 << i,), 0xFF, dtype=torch.uint8, device="cuda") for i in range(9, 20) for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert _same(got, norm)
    for a, b in zip(out, want, strict=True):
        assert _same(a, b)
    assert all(bool((j == 0xFF).all()) for j in junk)
