"""The operators around the experts with scratch of exactly the bytes that the library asks
for, between guard bands.  Bounds of clipping as in test_gpu_clip."""
import array

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _scratch(nbytes):
    assert nbytes > 0
    return Guarded((nbytes,), torch.uint8)


# 4 and 16 ids a thread, tables summed by every CTA and by a scan, bins with and without a word each
@pytest.mark.parametrize("N,G", [(65537, 1), (65537, 4096), (131072, 257), (131073, 1024), (524288, 1025), (524289, 3),
                                 (524289, 4096), (700001, 300)])
def test_sort(N, G):
    gen = torch.Generator(device="cuda").manual_seed(N)
    ids = torch.randint(-1, G + 1, (N,), device="cuda", dtype=I32, generator=gen)
    nbytes = gmm.gmm_sort_rows_scratch_bytes(N, G)
    scratch, rows, sizes = _scratch(nbytes), Guarded((N,), I32), Guarded((G,), I32)
    assert gmm.gmm_sort_rows(ids, N, G, rows.t, sizes.t, scratch.t, nbytes) == 0
    for g in (scratch, rows, sizes):
        g.check()
    group = torch.where((ids >= 0) & (ids < G), ids, G)
    order = torch.sort(group, stable=True).indices
    want = torch.empty_like(rows.t)
    want[order] = torch.arange(N, device="cuda", dtype=I32)
    assert torch.equal(rows.t, torch.where(group < G, want, -1 - want))
    assert torch.equal(sizes.t.long(), torch.bincount(group.long(), minlength=G + 1)[:G])
    assert gmm.gmm_sort_rows(ids, N, G, rows.t, sizes.t, scratch.t, nbytes - 1) == 8


# teams of rows and single rows a CTA, more CTAs than rows and fewer, the wide rows' shared memory
@pytest.mark.parametrize("T,K", [(65, 2048), (513, 256), (5000, 8), (2000, 1000), (65, 4096), (330, 2304), (1, 4104),
                                 (310, 8184), (155, 8192)])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("full", [False, True])
def test_norm_backward(T, K, stream, full):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s, dt=F32: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    dout, dn, out, b = rnd(T, K, dt=stream), rnd(T, K, dt=BF), rnd(T, K, dt=stream), rnd(T, K, dt=BF)
    w_post, w_next, gate = rnd(K), rnd(K), rnd(T, K, dt=BF) if full else rnd(K)
    want = gmm.norm_join_bwd(dout, dn, out, b, w_post, gate, w_next)
    nbytes = gmm.gmm_norm_join_bwd_scratch_bytes(T, K)
    scratch = _scratch(nbytes)
    got = [Guarded((T, K), stream), Guarded((T, K), BF), Guarded((K,), F32),
           Guarded((T, K), BF) if full else Guarded((K,), F32), Guarded((K,), F32)]
    args = (dout, dn, out, int(stream == F32), b, w_post, gate, full, w_next, T, K, 1.0, 1.0, 1e-6,
            *(g.t for g in got), scratch.t)
    assert gmm.gmm_norm_join_bwd(*args, nbytes) == 0
    scratch.check("scratch")
    for g, w in zip(got, want, strict=True):
        g.check()
        assert _same(g.t, w)
    assert gmm.gmm_norm_join_bwd(*args, nbytes - 1) == 8


# one table and several, of fewer tensors than are given
@pytest.mark.parametrize("counts", [[300000] + [1] * 63, [300000] + [1] * 64, [0] * 5 + [300000] + [3] * 60, [7] * 65,
                                    [0] * 3 + [4097] * 2000, [3] * 1001, [1] * 1000 + [0], [3000000]],
                         ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("in_place", [False, True])
def test_clipping(counts, in_place):
    gen = torch.Generator(device="cuda").manual_seed(len(counts))
    flat = torch.randn(sum(counts), generator=gen, device="cuda")
    grads = [g.to(BF if i % 3 else F32) for i, g in enumerate(flat.split(counts))]
    want = [g.double() for g in grads]
    norm = torch.cat(want).norm().item()
    out = [Guarded(g.shape, g.dtype) for g in grads]
    if in_place:
        for o, g in zip(out, grads):
            o.t.copy_(g)
    n, total = len(grads), sum(counts)
    nbytes = gmm.gmm_clip_grads_scratch_bytes(n, total)
    scratch, got = _scratch(nbytes), Guarded((1,), F32)
    src = array.array("Q", [t.data_ptr() for t in ((o.t for o in out) if in_place else grads)])
    dst = array.array("Q", [o.t.data_ptr() for o in out])
    count = array.array("q", counts)
    types = array.array("i", [int(g.dtype == F32) for g in grads])
    at = lambda a: a.buffer_info()[0]  # noqa: E731
    args = (at(src), None if in_place else at(dst), at(count), at(types), n, 0.5, got.t, scratch.t)
    assert gmm.gmm_clip_grads(*args, nbytes - 1) == 8
    assert gmm.gmm_clip_grads(*args, nbytes) == 0
    scratch.check("scratch")
    got.check("norm")
    assert abs(got.t.item() - norm) <= R.F32 * norm
    for i in list(range(min(n, 70))) + list(range(max(0, n - 70), n)):
        out[i].check(f"gradient {i}")
    for o, w in zip(out, want, strict=True):
        half = R.U if o.t.dtype == F32 else R.BF16
        R.assert_within(o.t, w * (0.5 / norm), (half + R.F32) * w.abs() * (0.5 / norm), "scaled")
