"""Rows sorted by expert and joined again: places and moved rows are equal to the plain
implementation's, sums and gradients within the bounds of layer_ref (a sum of k terms; a
product of K terms in chains of K / 32 and fewer)."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _ids(T, k, E, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":  # every choice on one expert
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    if kind == "zipf":
        p = np.arange(1.0, E + 1) ** -1.1
        ids = rng.choice(E, (T, k), p=p / p.sum())
    else:
        ids = rng.integers(0, E, (T, k))
    if kind == "ragged":  # choices of no group: padding, experts of other shards, both ends of int32
        odd = rng.random((T, k))
        ids = np.where(odd < 0.2, -1, np.where(odd < 0.4, E + rng.integers(0, 9, (T, k)), ids))
        ids.ravel()[:2] = (-2 ** 31, 2 ** 31 - 1)[:ids.size]
    return ids.astype(np.int32)


SORTS = [(1, 1, 1, "even"), (1, 8, 4, "even"), (3, 2, 5, "ragged"), (64, 8, 32, "even"), (65, 8, 256, "zipf"),
         (511, 1, 7, "ragged"), (513, 4, 64, "ragged"), (1024, 8, 4096, "even"), (1024, 8, 8, "one"), (1025, 8, 33, "zipf"),
         (8192, 8, 256, "zipf"), (8192, 8, 1, "one"), (5000, 7, 4096, "ragged"), (20000, 8, 257, "ragged"),
         (70000, 8, 100, "zipf"), (40000, 8, 3, "none"), (300000, 8, 4096, "even")]


@pytest.mark.parametrize("T,k,E,kind", SORTS)
def test_sort_rows(T, k, E, kind):
    ids = _ids(T, k, E, kind, T + E)
    rows, sizes = Guarded((T, k), torch.int32), Guarded((E,), torch.int32)
    gmm.sort_rows(torch.from_numpy(ids).cuda(), E, out=(rows.t, sizes.t))
    rows.check("rows")
    sizes.check("group_sizes")
    want, n = R.places(ids, E)
    assert np.array_equal(sizes.t.cpu().numpy(), n)
    assert np.array_equal(rows.t.cpu().numpy(), want)


def test_sort_of_nothing():
    rows, sizes = gmm.sort_rows(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 300)
    assert rows.shape == (0, 4) and sizes.tolist() == [0] * 300


def test_sort_of_a_vector():
    ids = torch.tensor([3, 1, -1, 1], dtype=torch.int32, device="cuda")
    rows, sizes = gmm.sort_rows(ids, 4)
    assert rows.tolist() == [2, 0, -4, 1] and sizes.tolist() == [0, 2, 0, 1]


MOVES = [(1, 1, 1, 128, "even"), (1, 8, 8, 2048, "even"), (5, 3, 4, 384, "ragged"), (33, 8, 32, 1152, "zipf"),
         (257, 2, 9, 640, "ragged"), (100, 6, 3, 128, "none"), (64, 32, 40, 256, "ragged"), (1500, 8, 64, 2048, "zipf"),
         (40, 9, 5, 8192, "ragged")]


def _case(T, k, E, K, kind):
    gen = torch.Generator(device="cuda").manual_seed(T * 31 + K)
    rows, sizes = gmm.sort_rows(torch.from_numpy(_ids(T, k, E, kind, T)).cuda(), E)
    x = torch.randn((T, K), generator=gen, device="cuda", dtype=BF)
    y = torch.randn((T * k, K), generator=gen, device="cuda", dtype=BF)
    w = torch.randn((T, k), generator=gen, device="cuda")
    return rows, int(sizes.sum()), x, y, w


def _moved(x, rows):
    token, _, live = R.tokens_of(rows.cpu().numpy())
    out = x[torch.from_numpy(token).cuda()]
    out[~torch.from_numpy(live).cuda()] = 0
    return out


@pytest.mark.parametrize("T,k,E,K,kind", MOVES)
def test_gather_rows(T, k, E, K, kind):
    rows, S, x, _, _ = _case(T, k, E, K, kind)
    x[0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 1e-40])
    out = Guarded((T * k, K), BF)
    gmm.gather_rows(x, rows, out=out.t)
    out.check("rows")
    assert torch.equal(out.t.view(torch.int16), _moved(x, rows).view(torch.int16))


@pytest.mark.parametrize("K", [8, 24, 1000, 2056])
def test_gather_and_combine_of_odd_columns(K):
    rows, _, x, _, _ = _case(130, 4, 9, K, "ragged")
    out = Guarded((130 * 4, K), BF)
    gmm.gather_rows(x, rows, out=out.t)
    out.check("rows")
    assert torch.equal(out.t, _moved(x, rows))
    back = Guarded((130, K), BF)
    gmm.combine_rows(out.t, rows, out=back.t)
    back.check("sums")
    n = (rows >= 0).sum(1, keepdim=True)
    R.assert_within(back.t, n * x.double(), R.BF16 * (n * x.double()).abs(), "sums")


@pytest.mark.parametrize("T,k,E,K,kind", MOVES)
def test_gather_quantize_is_the_quantisation_of_the_gathered_rows(T, k, E, K, kind):
    rows, S, x, _, _ = _case(T, k, E, K, kind)
    x[T - 1] = 0
    x[0, :128] *= 1e-30
    xq, xs = Guarded((T * k, K), torch.uint8), Guarded((K // 128, T * k), torch.float32)
    gmm.gather_quantize(x, rows, out=(xq.t, xs.t))
    xq.check("codes")
    xs.check("scales")
    wq, ws = gmm.quantize_lhs(_moved(x, rows))
    assert torch.equal(xq.t, wq)
    assert torch.equal(xs.t.view(torch.int32), ws.view(torch.int32))


@pytest.mark.parametrize("T,k,E,K,kind", MOVES)
def test_gather_mx4_quantize_is_the_quantisation_of_the_gathered_rows(T, k, E, K, kind):
    rows, S, x, _, _ = _case(T, k, E, K, kind)
    x[T - 1] = 0
    x[0, :32] *= 1e-30
    x[0, 40], x[0, 80] = float("inf"), -0.0
    xq, xs = Guarded((T * k, K // 2), torch.uint8), Guarded((K // 128, T * k, 4), torch.uint8)
    gmm.gather_mx4_quantize(x, rows, out=(xq.t, xs.t))
    xq.check("codes")
    xs.check("scales")
    wq, ws = gmm.mx4_quantize_lhs(_moved(x, rows))
    assert torch.equal(xq.t, wq) and torch.equal(xs.t, ws)
    got = gmm.gather_mx4_quantize(x, rows)
    assert torch.equal(got[0], wq) and torch.equal(got[1], ws)


@pytest.mark.parametrize("T,k,E,K,kind", MOVES)
@pytest.mark.parametrize("weighted", [False, True])
def test_combine_rows(T, k, E, K, kind, weighted):
    rows, S, _, y, w = _case(T, k, E, K, kind)
    y[S:] = float("nan")  # what lies behind the groups is nobody's
    w[rows < 0] = float("inf")
    out = Guarded((T, K), BF)
    gmm.combine_rows(y, rows, w if weighted else None, out=out.t)
    out.check("sums")
    want, mag = R.combine(y, rows, w if weighted else None)
    R.assert_within(out.t, want, R.BF16 * want.abs() + (k + 1) * R.U * mag, "sums")


@pytest.mark.parametrize("T,k,E,K,kind", MOVES + [(9, 4, 5, 8, "ragged"), (130, 3, 5, 1000, "ragged")])
def test_combine_rows_bwd(T, k, E, K, kind):
    rows, S, dout, y, w = _case(T, k, E, K, kind)
    y[S:] = float("nan")
    w[rows < 0] = float("inf")
    dy, dw = Guarded((T * k, K), BF), Guarded((T, k), torch.float32)
    gmm.combine_rows_bwd(dout, y, rows, w, out=(dy.t, dw.t))
    dy.check("dy")
    dw.check("dweights")
    token, choice, live = (torch.from_numpy(a).cuda() for a in R.tokens_of(rows.cpu().numpy()))
    want = torch.where(live[:, None], w[token, choice].double()[:, None] * dout[token].double(), 0.0)
    R.assert_within(dy.t, want, (R.BF16 + 2 * R.U) * want.abs(), "dy")
    terms = torch.where(live[:, None], dout[token].double() * y.double(), 0.0)
    at = torch.where(rows >= 0, rows, -1 - rows).long()
    R.assert_within(dw.t, terms.sum(1)[at], (K / 32 + 24) * R.U * terms.abs().sum(1)[at], "dweights")


def test_rows_that_name_no_row_are_skipped():
    """Values that no sort gives touch nothing: checked against guard bands, and rows left as they were."""
    T, k, K = 6, 2, 256
    M = T * k
    rows, _, x, y, w = _case(T, k, 4, K, "even")
    for i, v in enumerate((M, -1 - M, 2 ** 31 - 1, -2 ** 31)):
        rows[i, 1] = v
    kept = {r if r >= 0 else -1 - r for r in rows.ravel().tolist()}
    out, q, s = Guarded((M, K), BF), Guarded((M, K), torch.uint8), Guarded((K // 128, M), torch.float32)
    gmm.gather_rows(x, rows, out=out.t)
    gmm.gather_quantize(x, rows, out=(q.t, s.t))
    dy, dw = Guarded((M, K), BF), Guarded((T, k), torch.float32)
    gmm.combine_rows_bwd(x, y, rows, w, out=(dy.t, dw.t))
    for g in (out, q, s, dy, dw):
        g.check()
    left = [r for r in range(M) if r not in kept]
    assert len(left) == 4
    assert bool(out.t[left].isnan().all()) and bool(dy.t[left].isnan().all()) and bool((q.t[left] == 0xEE).all())
    got = gmm.combine_rows(y, rows, w)
    ok = (rows >= 0) & (rows < M)
    want, mag = R.combine(y, torch.where(ok, rows, -1), w)
    R.assert_within(got, want, R.BF16 * want.abs() + 4 * R.U * mag, "sums")


def test_the_same_row_twice_in_combine():
    y = torch.randn((4, 128), device="cuda", dtype=BF)
    rows = torch.tensor([[1, 1], [3, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.25, 0.5], [1.0, 2.0]], device="cuda")
    want, mag = R.combine(y, rows, w)
    R.assert_within(gmm.combine_rows(y, rows, w), want, R.BF16 * want.abs() + 3 * R.U * mag, "sums")


def test_no_tokens():
    rows = torch.empty((0, 8), dtype=torch.int32, device="cuda")
    x, w = torch.empty((0, 256), dtype=BF, device="cuda"), torch.empty((0, 8), device="cuda")
    assert gmm.gather_rows(x, rows).shape == (0, 256)
    assert gmm.gather_quantize(x, rows)[0].shape == (0, 256)
    assert gmm.gather_mx4_quantize(x, rows)[1].shape == (2, 0, 4)
    assert gmm.combine_rows(x, rows, w).shape == (0, 256)
    assert gmm.combine_rows_bwd(x, x, rows, w)[1].shape == (0, 8)


def test_offsets_past_32_bits():
    """2^31 + elements of sorted rows: the last rows land where they belong."""
    T, k, K = 34000, 8, 8192
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) % 5
    rows, sizes = gmm.sort_rows(ids, 5)
    x = torch.randn((T, K), device="cuda", dtype=BF, generator=torch.Generator(device="cuda").manual_seed(0))
    out = gmm.gather_rows(x, rows)
    assert out.numel() > 2 ** 31
    place, pick = rows.view(-1).long(), torch.tensor([0, 1, 7, T * k // 2, T * k - 9, T * k - 1], device="cuda")
    assert torch.equal(out[place[pick]], x[pick // k])
    assert torch.equal(out[-1], x[(place == T * k - 1).nonzero()[0, 0] // k])
    back = gmm.combine_rows(out, rows)
    assert torch.equal(back, (x.float() * k).to(BF))
    w = torch.full((T, k), 0.5, device="cuda")
    dy, dw = gmm.combine_rows_bwd(x, out, rows, w)
    assert torch.equal(dy[place[pick]], (x.float() * 0.5).to(BF)[pick // k])
    t = pick // k
    want = x[t].double().square().sum(1)
    R.assert_within(dw.view(-1)[pick], want, (K / 32 + 24) * R.U * want, "dweights")
