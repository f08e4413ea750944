"""Host-side checks of the entry points around the experts (no GPU needed): refusals,
all made before any launch, and the plain implementations that the GPU tests compare
with, against autograd, differences and values worked out by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import layer_ref as R

FAKE = 1 << 20  # an aligned non-null pointer value; never dereferenced on the host
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    from fp8_blockwise_quantized_gb300 import build as b
    b.build()
    import fp8_blockwise_quantized_gb300 as g
    return g.load()


def _call(fn, spec, kw):
    names, values = zip(*spec)
    a = dict(zip(names, values))
    assert set(kw) <= set(names)
    a.update(kw)
    return fn(*[a[n] for n in names])


ROUTE = [("logits", FAKE), ("type", 1), ("bias", FAKE), ("T", 8), ("E", 16), ("k", 4), ("score", 0), ("renorm", 0),
         ("scale", 1.0), ("ids", FAKE), ("weights", FAKE), ("stream", None)]
ROUTE_BWD = [("dw", FAKE), ("logits", FAKE), ("type", 1), ("ids", FAKE), ("T", 8), ("E", 16), ("k", 4), ("score", 0),
             ("renorm", 0), ("scale", 1.0), ("dlogits", FAKE), ("stream", None)]
CHOICES = [(dict(T=-1), 2), (dict(k=0), 2), (dict(k=33, E=64), 2), (dict(E=0), 2), (dict(E=4097), 2), (dict(k=17), 2),
           (dict(T=1 << 31), 2), (dict(T=1 << 30), 2), (dict(type=2), 4), (dict(type=-1), 4), (dict(score=2), 4)]


@pytest.mark.parametrize("kw,code", CHOICES + [
    (dict(logits=None), 1), (dict(ids=None), 1), (dict(weights=None), 1), (dict(logits=FAKE + 4), 3),
    (dict(bias=FAKE + 4), 3), (dict(ids=FAKE + 8), 3), (dict(T=0, logits=None, ids=None, weights=None), 0)])
def test_route_refusals(lib, kw, code):
    assert _call(lib.gmm_route, ROUTE, kw) == code


@pytest.mark.parametrize("kw,code", CHOICES + [
    (dict(dw=None), 1), (dict(logits=None), 1), (dict(ids=None), 1), (dict(dlogits=None), 1), (dict(dw=FAKE + 4), 3),
    (dict(dlogits=FAKE + 2), 3), (dict(T=0, dw=None, logits=None, ids=None, dlogits=None), 0)])
def test_route_bwd_refusals(lib, kw, code):
    assert _call(lib.gmm_route_bwd, ROUTE_BWD, kw) == code


SORT = [("ids", FAKE), ("N", 100000), ("G", 16), ("rows", FAKE), ("sizes", FAKE), ("scratch", FAKE), ("sbytes", 1 << 20),
        ("stream", None)]


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 2), (dict(N=1 << 31), 2), (dict(G=0), 2), (dict(G=4097), 2), (dict(ids=None), 1), (dict(rows=None), 1),
    (dict(sizes=None), 1), (dict(N=0, sizes=None), 1), (dict(ids=FAKE + 4), 3), (dict(scratch=FAKE + 4), 3),
    (dict(scratch=None), 8), (dict(sbytes=64), 8)])
def test_sort_refusals(lib, kw, code):
    assert _call(lib.gmm_sort_rows, SORT, kw) == code


def test_sort_scratch(lib):
    need = lib.gmm_sort_rows_scratch_bytes
    assert need(0, 4) == 0 and need(65536, 4096) == 0 and need(-1, 4) == 0 and need(10, 0) == 0
    for n, g in ((65537, 1), (1 << 18, 256), (1 << 20, 4096), (2 ** 31 - 1, 4096)):
        assert 0 < need(n, g) < 5 * 2 ** 32


ROWS = {
    "gmm_gather_rows": ("x rows | out", 8),
    "gmm_gather_quantize": ("x rows | xq xs", 128),
    "gmm_gather_mx4_quantize": ("x rows | xq xs", 128),
    "gmm_combine_rows": ("y rows weights | out", 8),
    "gmm_combine_rows_bwd": ("dout y rows weights | dy dweights", 8),
}


@pytest.mark.parametrize("name", ROWS)
def test_row_refusals(lib, name):
    spec, unit = ROWS[name]
    before, after = (s.split() for s in spec.split("|"))
    full = [(n, FAKE) for n in before] + [("T", 8), ("k", 4), ("K", 256)] + [(n, FAKE) for n in after] + [("stream", None)]
    fn = getattr(lib, name)
    for kw, code in [(dict(T=-1), 2), (dict(k=0), 2), (dict(k=33), 2), (dict(T=1 << 31), 2), (dict(T=1 << 30, k=2), 2),
                     (dict(K=0), 2), (dict(K=256 + unit // 2), 2), (dict(K=-256), 2), (dict(K=1 << 25), 2)]:
        assert _call(fn, full, kw) == code, kw
    for n in before + after:
        if not (name == "gmm_combine_rows" and n == "weights"):
            assert _call(fn, full, {n: None}) == 1, n
        assert _call(fn, full, {n: FAKE + 8}) == 3, n
    assert _call(fn, full, dict({n: None for n in before + after}, T=0)) == 0


JOIN = [("x", FAKE), ("type", 1), ("b", FAKE), ("w_post", FAKE), ("gate", FAKE), ("gate_rows", 0), ("w_next", FAKE),
        ("T", 8), ("K", 256), ("alpha", 1.0), ("beta", 1.0), ("eps", 1e-6), ("out", FAKE), ("n", FAKE), ("stream", None)]
JOIN_BWD = [("dout", FAKE), ("dn", FAKE), ("out", FAKE), ("type", 1), ("b", FAKE), ("w_post", FAKE), ("gate", FAKE),
            ("gate_rows", 0), ("w_next", FAKE), ("T", 8), ("K", 256), ("alpha", 1.0), ("beta", 1.0), ("eps", 1e-6),
            ("dx", FAKE), ("db", FAKE), ("dw_post", FAKE), ("dgate", FAKE), ("dw_next", FAKE), ("scratch", FAKE),
            ("sbytes", 1 << 30), ("stream", None)]
SHARED = [(dict(T=-1), 2), (dict(T=1 << 31), 2), (dict(K=0), 2), (dict(K=260), 2), (dict(K=8200), 2), (dict(type=2), 4),
          (dict(eps=-1.0), 4), (dict(eps=math.nan), 4)]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(x=None), 1), (dict(out=None), 1), (dict(n=None), 1), (dict(b=None), 1), (dict(b=None, w_post=None), 1),
    (dict(b=None, w_post=None, gate=None, w_next=None), 1), (dict(x=FAKE + 8), 3), (dict(gate=FAKE + 4), 3),
    (dict(T=0, x=None, out=None, n=None), 0)])
def test_join_refusals(lib, kw, code):
    assert _call(lib.gmm_norm_join, JOIN, kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(b=None), 1), (dict(w_post=None), 1), (dict(gate=None), 1), (dict(w_next=None), 1),
    (dict(w_next=None, dw_next=None), 1), (dict(out=None), 1), (dict(db=None), 1), (dict(gate_rows=1, dgate=None), 1),
    (dict(dout=FAKE + 8), 3), (dict(dw_next=FAKE + 4), 3), (dict(scratch=FAKE + 4), 3)])
def test_join_bwd_refusals(lib, kw, code):
    assert _call(lib.gmm_norm_join_bwd, JOIN_BWD, kw) == code


def _clip(lib, kw):
    n = kw.pop("n", 2)
    ptrs = kw.pop("grads", [FAKE, FAKE + 64])
    outs = kw.pop("out", None)
    counts, types = kw.pop("counts", [5, 7]), kw.pop("types", [1, 0])
    arr = lambda t, v: None if v is None else (t * max(1, len(v)))(*v)  # noqa: E731
    a = dict(max_norm=1.0, norm=FAKE, scratch=FAKE, sbytes=1 << 20)
    a.update(kw)
    return lib.gmm_clip_grads(arr(ctypes.c_void_p, ptrs), arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, counts),
                              arr(ctypes.c_int32, types), n, a["max_norm"], a["norm"], a["scratch"], a["sbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 2), (dict(max_norm=-1.0), 4), (dict(max_norm=math.nan), 4), (dict(norm=None), 1), (dict(grads=None), 1),
    (dict(counts=None), 1), (dict(types=None), 1), (dict(types=[1, 2]), 4), (dict(counts=[5, -1]), 2),
    (dict(counts=[1 << 42, 1]), 2), (dict(grads=[None, FAKE]), 1), (dict(out=[FAKE, None]), 1),
    (dict(grads=[FAKE + 2, FAKE + 64]), 3), (dict(grads=[FAKE, FAKE + 65]), 3), (dict(out=[FAKE, FAKE + 65]), 3),
    (dict(norm=FAKE + 4), 3), (dict(scratch=FAKE + 8), 3),
    # 5 fp32 values (20 bytes) and 7 bf16 values (14 bytes) that share memory
    (dict(grads=[FAKE, FAKE]), 4), (dict(grads=[FAKE, FAKE + 18]), 4), (dict(grads=[FAKE + 12, FAKE]), 4),
    (dict(out=[FAKE, FAKE + 4]), 4), (dict(grads=[FAKE, FAKE + 64], out=[FAKE + 4, FAKE + 64]), 4),
    (dict(grads=[FAKE, FAKE + 64], out=[FAKE + 64, FAKE]), 4),
    (dict(grads=[FAKE, FAKE + 64], out=[FAKE + 128, FAKE + 4]), 4)])
def test_clip_refusals(lib, kw, code):
    assert _clip(lib, dict(kw)) == code


def test_python_entry_points_refuse_what_kernels_cannot_take(lib):
    """Tensors on the host, of another type, size or stride are refused before anything reads them."""
    import fp8_blockwise_quantized_gb300 as g
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    rows, w = z(4, 2, dt=I32), z(4, 2, dt=F32)
    for call in (lambda: g.route(z(4, 8), 2), lambda: g.route_bwd(w, z(4, 8), rows), lambda: g.sort_rows(rows, 8),
                 lambda: g.gather_rows(z(4, 128), rows), lambda: g.gather_quantize(z(4, 128), rows),
                 lambda: g.gather_mx4_quantize(z(4, 128), rows),
                 lambda: g.combine_rows(z(8, 128), rows, w), lambda: g.combine_rows_bwd(z(4, 128), z(8, 128), rows, w),
                 lambda: g.norm_join(z(4, 128), w_next=z(128, dt=F32)),
                 lambda: g.norm_join_bwd(z(4, 128), None, z(4, 128)), lambda: g.clip_grads([z(4)], 1.0)):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        g.route(z(4, 8, dt=torch.float16), 2)
    with pytest.raises(ValueError, match="score"):
        g.route(z(4, 8), 2, score="relu")
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        g.clip_grads([z(4, dt=torch.float16)], 1.0)
    with pytest.raises(ValueError, match="out"):
        g.clip_grads([z(4)], 1.0, out=[])


# ---- the plain implementations -------------------------------------------------

def test_places_by_hand():
    rows, sizes = R.places(np.array([[2, 0], [5, 2], [-1, 0]]), 3)
    assert sizes.tolist() == [2, 0, 2]
    assert rows.tolist() == [[2, 0], [-1 - 4, 3], [-1 - 5, 1]]
    token, choice, live = R.tokens_of(rows)
    assert token.tolist() == [0, 2, 0, 1, 1, 2] and choice.tolist() == [1, 1, 0, 1, 0, 0]
    assert live.tolist() == [True] * 4 + [False] * 2


def test_chosen_by_hand():
    l = torch.tensor([[1.0, 3.0, 3.0, -math.inf], [math.nan, -math.inf, 0.0, -0.0], [-math.inf] * 4])
    assert R.chosen(l, None, 3).tolist() == [[1, 2, 0], [2, 3, -1], [-1, -1, -1]]
    bias = torch.tensor([2.5, 0.0, 0.0, math.inf])
    assert R.chosen(l, bias, 2).tolist() == [[0, 1], [3, 2], [-1, -1]]
    w = R.route_weights(l.double(), torch.from_numpy(R.chosen(l, None, 3)), "softmax", True, 2.0)
    assert torch.allclose(w[0], 2 * torch.softmax(torch.tensor([3.0, 3.0, 1.0]).double(), 0))
    assert torch.equal(w[2], torch.zeros(3).double())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_of_the_formula_and_by_differences(score, renorm):
    gen = torch.Generator().manual_seed(3)
    T, E, k = 4, 7, 3
    l = torch.randn((T, E), generator=gen, dtype=torch.float64).requires_grad_()
    ids = torch.from_numpy(R.chosen(l.detach(), None, k))
    ids[1, 2], ids[2, 1], ids[3] = -1, ids[2, 0], 9  # one without an expert, one named twice, none in range
    dw = torch.randn((T, k), generator=gen, dtype=torch.float64)
    loss = lambda v: (dw * R.route_weights(v, ids, score, renorm, 1.7)).sum()  # noqa: E731
    want, = torch.autograd.grad(loss(l), l)
    got, mag = R.route_bwd(dw, l.detach(), ids, score, renorm, 1.7)
    assert torch.allclose(got, want, atol=1e-14) and bool((mag >= got.abs() - 1e-15).all())
    for t in range(T):
        for e in range(E):
            h = torch.zeros_like(l)
            h[t, e] = 1e-6
            d = (loss(l.detach() + h) - loss(l.detach() - h)) / 2e-6
            assert abs(d - got[t, e]) < 1e-8


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "column", "full"])
def test_join_gradient_of_the_formula_and_by_differences(post, gate):
    gen = torch.Generator().manual_seed(5)
    T, K, a, c, eps = 3, 8, 0.9, 0.7, 1e-3
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, b, w_next = rnd(T, K), rnd(T, K), rnd(K)
    w_post = rnd(K) if post else None
    g = {None: None, "column": rnd(K), "full": rnd(T, K)}[gate]
    dout, dn = rnd(T, K).detach(), rnd(T, K).detach()

    def loss(x, b, w_post, g, w_next):
        out, n, _ = R.norm_join(x, b, w_post, g, w_next, a, c, eps)
        return (dout * out).sum() + (dn * n).sum()

    leaves = [x, b, w_post, g, w_next]
    got, mags = R.norm_join_bwd(dout, dn, R.norm_join(x, b, w_post, g, w_next, a, c, eps)[0].detach(), b.detach(),
                                *(None if t is None else t.detach() for t in (w_post, g, w_next)), a, c, eps)
    for i, leaf in enumerate(leaves):
        if leaf is None:
            assert got[i] is None
            continue
        want, = torch.autograd.grad(loss(*leaves), leaf)
        assert torch.allclose(got[i], want, atol=1e-13), i
        assert bool((mags[i] >= got[i].abs() - 1e-13).all())
        h = torch.zeros_like(leaf)
        h.view(-1)[3] = 1e-6
        up, down = ([t if j != i else t + s * h for j, t in enumerate(leaves)] for s in (1, -1))
        assert abs((loss(*up) - loss(*down)) / 2e-6 - got[i].reshape(-1)[3]) < 1e-7


def test_norm_in_front_of_a_first_block():
    x = torch.randn((2, 8), dtype=torch.float64).requires_grad_()
    w, dn = torch.randn(8, dtype=torch.float64), torch.randn((2, 8), dtype=torch.float64)
    out, n, _ = R.norm_join(x, None, None, None, w, 1.0, 1.0, 1e-6)
    want, = torch.autograd.grad((dn * n).sum(), x)
    got, _ = R.norm_join_bwd(None, dn, x.detach(), None, None, None, w, 1.0, 1.0, 1e-6)
    assert torch.allclose(got[0], want, atol=1e-13) and got[1] is None
