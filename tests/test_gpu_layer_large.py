"""Sizes past 32-bit indices of what surrounds the experts, on rows that lie anywhere in them."""
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _spots(n, device="cuda"):
    return torch.tensor([0, 1, n // 3, n // 2 - 1, n // 2, n - 2, n - 1], device=device)


def test_gather_and_combine_with_64_bit_thread_indices():
    """T K / 8 = 2^31 threads."""
    T, K = 2 ** 21, 8192
    ids = (torch.arange(T, device="cuda") % 3).int().view(T, 1)
    rows, sizes = gmm.sort_rows(ids, 2)  # every third token is nobody's
    live = int(sizes.sum())
    assert sizes.tolist() == [(T + 2) // 3, (T + 1) // 3]
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    at = _spots(T)
    x[at] = torch.randn((len(at), K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)
    out = gmm.gather_rows(x, rows)
    place = rows[at, 0].long()
    for t, p in zip(at.tolist(), place.tolist()):
        if p >= 0:
            assert p < live and torch.equal(out[p], x[t])
        else:
            assert -1 - p >= live and not bool(out[-1 - p].any())
    back = gmm.combine_rows(out, rows)
    assert torch.equal(back[at], torch.where((place >= 0)[:, None], x[at], 0))


def test_gather_quantize_with_64_bit_thread_indices():
    """T K / 128 = 2^28 blocks of 8 threads."""
    T, K = 2 ** 22, 8192
    rows = torch.arange(T, device="cuda", dtype=I32).flip(0).view(T, 1)
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    at = _spots(T)
    x[at] = torch.randn((len(at), K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(BF)
    xq, xs = gmm.gather_quantize(x, rows)
    wq, ws = gmm.quantize_lhs(x[at])
    p = rows[at, 0].long()
    assert torch.equal(xq[p], wq) and torch.equal(xs[:, p], ws)
    del xq, xs
    xq, xs = gmm.gather_mx4_quantize(x, rows)
    wq, ws = gmm.mx4_quantize_lhs(x[at])
    assert torch.equal(xq[p], wq) and torch.equal(xs[:, p], ws)


def test_combine_gradient_past_32_bits():
    T, k, K = 2 ** 17 + 3, 4, 8192
    rows, _ = gmm.sort_rows((torch.arange(T * k, device="cuda") % 7).int().view(T, k), 6)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dout, y = torch.zeros((T, K), dtype=BF, device="cuda"), torch.zeros((T * k, K), dtype=BF, device="cuda")
    at = _spots(T)
    dout[at] = torch.randn((len(at), K), device="cuda", generator=gen).to(BF)
    place = torch.where(rows[at] >= 0, rows[at], -1 - rows[at]).long()
    y[place.flatten()] = torch.randn((len(at) * k, K), device="cuda", generator=gen).to(BF)
    w = torch.rand((T, k), device="cuda", generator=gen)
    assert y.numel() > 2 ** 31
    dy, dw = gmm.combine_rows_bwd(dout, y, rows, w)
    live = (rows[at] >= 0)[:, :, None]
    want = torch.where(live, w[at].double()[:, :, None] * dout[at].double()[:, None, :], 0.0)
    R.assert_within(dy[place], want, (R.BF16 + 2 * R.U) * want.abs(), "dy")
    terms = torch.where(live, dout[at].double()[:, None, :] * y[place].double(), 0.0)
    R.assert_within(dw[at], terms.sum(2), (K / 32 + 24) * R.U * terms.abs().sum(2), "dweights")


@pytest.mark.parametrize("N,E", [(50_000_000, 300), (70_001, 2000)])
def test_sort_of_many(N, E):
    ids = torch.randint(-1, E + 1, (N,), device="cuda", dtype=I32, generator=torch.Generator(device="cuda").manual_seed(4))
    rows, sizes = gmm.sort_rows(ids, E)
    group = torch.where((ids >= 0) & (ids < E), ids, E)
    order = torch.sort(group, stable=True).indices
    want = torch.empty_like(rows)
    want[order] = torch.arange(N, device="cuda", dtype=I32)
    assert torch.equal(rows, torch.where(group < E, want, -1 - want))
    assert torch.equal(sizes.long(), torch.bincount(group.long(), minlength=E + 1)[:E])


def test_route_past_32_bits():
    T, E, k = 2 ** 23 + 3, 512, 2
    l = torch.zeros((T, E), dtype=BF, device="cuda")
    at = _spots(T)
    l[at] = torch.randn((len(at), E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF)
    ids, w = gmm.route(l, k)
    assert torch.equal(ids[at].cpu(), torch.from_numpy(R.chosen(l[at], None, k)))
    ref = R.route_weights(l[at].double(), ids[at], "softmax", False, 1.0)
    R.assert_within(w[at], ref, 4 * R.F32 * ref, "weights")
    assert ids[5].tolist() == [0, 1]
    dw = torch.ones_like(w)
    dl = gmm.route_bwd(dw, l, ids)
    want, mag = R.route_bwd(dw[at], l[at], ids[at], "softmax", False, 1.0)
    R.assert_within(dl[at], want, R.BF16 * want.abs() + 12 * R.F32 * mag, "dlogits")


def test_norms_past_32_bits():
    T, K = 2 ** 18 + 5, 8192
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, b = (torch.ones((T, K), dtype=BF, device="cuda") for _ in range(2))
    at = _spots(T)
    x[at] = torch.randn((len(at), K), device="cuda", generator=gen).to(BF)
    b[at] = torch.randn((len(at), K), device="cuda", generator=gen).to(BF)
    w = torch.rand(K, device="cuda", generator=gen) + 0.5
    out, n = gmm.norm_join(x, b, w, w, w)
    want, wn, mag = R.norm_join(x[at].double(), b[at].double(), w.double(), w.double(), w.double(), 1.0, 1.0, 1e-6)
    R.assert_within(out[at], want, R.BF16 * want.abs() + R.F32 * mag, "out")
    R.assert_within(n[at], wn, R.BF16 * wn.abs() + 8 * R.F32 * (wn.abs() + mag), "n")
    del n
    dx, db, *_ = gmm.norm_join_bwd(x, b, out, b, w, w, w)
    ref, mags = R.norm_join_bwd(x[at].double(), b[at].double(), out[at].double(), b[at].double(), w.double(), w.double(),
                                w.double(), 1.0, 1.0, 1e-6)
    R.assert_within(dx[at], ref[0], R.BF16 * ref[0].abs() + 2 * R.F32 * mags[0], "dx")
    R.assert_within(db[at], ref[1], R.BF16 * ref[1].abs() + 2 * R.F32 * mags[1], "db")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_clipping_of_one_tensor_past_32_bits(dtype):
    n = 2 ** 31 + 70001
    g = torch.zeros(n, dtype=dtype, device="cuda")
    at = _spots(n)
    g[at] = torch.tensor([3.0, -4.0, 1.0, 2.0, -2.0, 5.0, 7.0], device="cuda").to(dtype)
    norm = gmm.clip_grads([g], 1.0).item()
    want = 108.0 ** 0.5
    assert abs(norm - want) <= R.F32 * want
    half = R.U if dtype == F32 else R.BF16
    ref = torch.tensor([3.0, -4.0, 1.0, 2.0, -2.0, 5.0, 7.0], device="cuda").double() / want
    R.assert_within(g[at], ref, (half + R.F32) * ref.abs(), "scaled")
    assert int(torch.count_nonzero(g[:1000])) == 2
