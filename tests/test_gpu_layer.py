"""The operators around the experts together, as a layer uses them (examples/moe_layer.py),
against the same layer in 64 bits by autograd; on streams and devices; captured and replayed.

Bound of the layer's outputs and gradients, as a share of their norms: what is held in bf16
is rounded by 2^-8 of itself at most.  Forward: n, gate | up, h, y, b, out or n.  Backward
besides: dx, db, dy, dgu, h again, the experts' gradients, dxs, its sum by token, dn, dx:
17 in all.  Norms, weighted sums and products with weights of variance 1 / K do not make
such errors grow, so 17 of them stay below 17 * 2^-8; the norm's and the softmax's
gradients subtract a mean, which at most doubles a share: 34 * 2^-8 = 0.133.  The weights'
and norms' parameters lose nothing more.  (A layer wired wrongly is off by its whole norm.)"""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FORWARD, BACKWARD = 6 * R.BF16, 34 * R.BF16


def _exact(layer, x, ids, absent, dout, dn):
    """(out, n, {name: gradient}, dx) in 64 bits, the choice taken as given."""
    p = {k: v.double().requires_grad_() for k, v in layer.params.items()}
    # the products take the weights' bf16 copies
    w, w2 = (p[n] + (p[n].detach().to(BF).double() - p[n].detach()) for n in ("w", "w2"))
    x = x.double().requires_grad_()
    eps = 1e-6
    n = R.unit(x, eps)[0] * p["w_pre"]
    weights = R.route_weights(n @ p["w_router"].t(), ids, layer.score, True, 1.0)
    b = torch.zeros_like(x)
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = n[t] @ w[e]
        N = gu.shape[1] // 2
        y = (torch.nn.functional.silu(gu[:, :N]) * gu[:, N:]) @ w2[e]
        b = b.index_add(0, t, weights[t, j, None] * y)
    out, nn, _ = R.norm_join(x, b, p["w_post"], p["gate"], p["w_next"], 1.0, 1.0, eps)
    loss = (nn * dn.double()).sum() + (0.0 if dout is None else (out * dout.double()).sum())
    loss.backward()
    return out.detach(), nn.detach(), {k: v.grad for k, v in p.items()}, x.grad


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("E,k,T,score", [(8, 2, 300, "softmax"), (16, 4, 1, "sigmoid"), (5, 1, 257, "sigmoid"),
                                         (32, 8, 128, "softmax")])
def test_layer_forward_and_gradients(E, k, T, score):
    from examples.moe_layer import MoELayer
    K, N = 384, 256
    layer = MoELayer(E, K, N, k, T, seed=E, score=score)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dout, dn = (torch.randn((T, K), generator=gen, device="cuda").to(BF) for _ in range(3))
    absent = torch.arange(T, device="cuda") >= max(1, T - T // 5)
    out, n = layer.forward(x, absent)
    logits, ids = layer.kept[2], layer.kept[3]
    assert torch.equal(ids.cpu(), torch.from_numpy(R.chosen(logits, layer.bias, k)))
    assert bool((ids[absent] == -1).all())
    dx, grads = layer.backward(dout, dn)
    assert layer.workspace.status() == 0
    w_out, w_n, w_grads, w_dx = _exact(layer, x, ids, absent, dout, dn)
    assert _off(out, w_out) < FORWARD and _off(n, w_n) < FORWARD
    assert _off(dx, w_dx) < BACKWARD
    for name, g in grads.items():
        if name == "w_router" and k == 1:  # renormed, one choice weighs 1 whatever the logits
            assert not bool(g.any())
            continue
        assert _off(g, w_grads[name]) < BACKWARD, name


@pytest.mark.parametrize("E,k,T", [(8, 2, 300), (16, 4, 1), (5, 1, 257)])
def test_layer_served_in_4_bits(E, k, T):
    """Bit for bit the layer that gathers in bf16 and quantises the sorted rows."""
    from examples.moe_layer import EPS, MoELayer
    K, N = 384, 256
    layer = MoELayer(E, K, N, k, T, seed=E)
    p, ws = layer.params, layer.workspace
    x = torch.randn((T, K), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(BF)
    got = layer.serve()(x)
    _, n = gmm.norm_join(x, w_next=p["w_pre"], eps=EPS)
    ids, weights = gmm.route(n.float() @ p["w_router"].t(), k, bias=layer.bias, score=layer.score, renorm=True)
    rows, sizes = gmm.sort_rows(ids, E)
    xq, xs = gmm.mx4_quantize_lhs(gmm.gather_rows(n, rows))
    _, hq, hs = gmm.mx4_fwd_swiglu_quant(xq, xs, *gmm.mx4_quantize_rhs(p["w"].to(BF)), sizes, workspace=ws)
    y = gmm.mx4_fwd(hq, hs, *gmm.mx4_quantize_rhs(p["w2"].to(BF)), sizes, workspace=ws)
    want = gmm.norm_join(x, gmm.combine_rows(y, rows, weights), p["w_post"], p["gate"], p["w_next"], eps=EPS)
    assert ws.status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_example_runs():
    from examples.moe_layer import main
    losses = main(["--steps", "3", "--tokens", "200"])
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


# ---- streams, graphs, calls in flight together ------------------------------------

@pytest.fixture(scope="module")
def data():
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, E, k, K = 700, 48, 4, 512
    rnd = lambda *s, dt=BF: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    d = dict(T=T, E=E, k=k, logits=rnd(T, E, dt=F32), bias=rnd(E, dt=F32), x=rnd(T, K), b=rnd(T, K), xf=rnd(T, K, dt=F32),
             y=rnd(T * k, K), col=rnd(K, dt=F32), dw=rnd(T, k, dt=F32),
             long_ids=torch.randint(-1, E, (90000,), generator=gen, device="cuda", dtype=I32),
             grads=[rnd(30000), rnd(7, 11, dt=F32), rnd(1)])
    d["ids"], d["weights"] = gmm.route(d["logits"], k)
    d["rows"], _ = gmm.sort_rows(d["ids"], E)
    torch.cuda.synchronize()
    return d


def _clip(d, **kw):
    out = [torch.zeros_like(g) for g in d["grads"]]
    return (gmm.clip_grads(d["grads"], 0.5, out=out, **kw), *out)


CALLS = {
    "route": lambda d, **k: gmm.route(d["logits"], d["k"], bias=d["bias"], renorm=True, **k),
    "route_bwd": lambda d, **k: gmm.route_bwd(d["dw"], d["logits"], d["ids"], **k),
    "sort_rows": lambda d, **k: gmm.sort_rows(d["ids"], d["E"], **k),
    "sort_rows long": lambda d, **k: gmm.sort_rows(d["long_ids"], d["E"], **k),
    "gather_rows": lambda d, **k: gmm.gather_rows(d["x"], d["rows"], **k),
    "gather_quantize": lambda d, **k: gmm.gather_quantize(d["x"], d["rows"], **k),
    "gather_mx4_quantize": lambda d, **k: gmm.gather_mx4_quantize(d["x"], d["rows"], **k),
    "combine_rows": lambda d, **k: gmm.combine_rows(d["y"], d["rows"], d["weights"], **k),
    "combine_rows_bwd": lambda d, **k: gmm.combine_rows_bwd(d["x"], d["y"], d["rows"], d["weights"], **k),
    "norm_join": lambda d, **k: gmm.norm_join(d["xf"], d["b"], d["col"], d["col"], d["col"], **k),
    "norm_join_bwd": lambda d, **k: gmm.norm_join_bwd(d["x"], d["b"], d["x"], d["b"], d["col"], d["b"], d["col"], **k),
    "clip_grads": _clip,
}


def _flat(out):
    return [t for o in out for t in _flat(o)] if isinstance(out, tuple) else [out]


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", [n for n in CALLS if n != "clip_grads"])
def test_a_busy_stream_that_is_not_current(data, name, as_handle):
    want = [t.clone() for t in _flat(CALLS[name](data))]
    busy = torch.zeros((2, 8192, 8192), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):  # 6 ms: the call below is queued behind it
            torch.mm(busy[0], busy[0], out=busy[1])
    got = _flat(CALLS[name](data, stream=side.cuda_stream if as_handle else side))
    # what the current stream takes and writes now must not be the call's memory
    junk = [torch.full((1 << i,), 0xFF, dtype=torch.uint8, device="cuda") for i in range(9, 24) for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    for a, b in zip(want, got, strict=True):
        assert _same(a, b)
    assert all(bool((j == 0xFF).all()) for j in junk)


def test_clipping_on_a_stream_that_is_not_current(data):
    want = [t.clone() for t in _clip(data)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = [torch.zeros_like(g) for g in data["grads"]]
    norm = gmm.clip_grads(data["grads"], 0.5, out=out, stream=side)
    side.synchronize()
    for a, b in zip(want, [norm, *out], strict=True):
        assert _same(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed_beside_another_graph(data, name):
    """Two graphs of one call on different streams, replayed together, with the inputs changed in between."""
    d = dict(data)
    moved = {k: v.clone() for k, v in d.items() if isinstance(v, torch.Tensor)}
    d.update(moved, grads=[g.clone() for g in d["grads"]])
    CALLS[name](d)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_flat(CALLS[name](d)))
        graphs.append(g)
    for i in range(3):
        for key in ("logits", "x", "b", "xf", "y"):
            d[key].copy_(data[key].roll(i, 0))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = _flat(CALLS[name](d))
        for got in outs:
            for a, b in zip(want, got, strict=True):
                assert _same(a, b)


def test_calls_on_many_streams_at_once(data):
    want = {n: [t.clone() for t in _flat(c(data))] for n, c in CALLS.items()}
    torch.cuda.synchronize()
    got = []
    for i in range(4):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got += [(n, _flat(c(data))) for n, c in CALLS.items()]
    torch.cuda.synchronize()
    for n, outs in got:
        for a, b in zip(want[n], outs, strict=True):
            assert _same(a, b), n


def test_outputs_given_are_written_in_place(data):
    d = data
    T, k, E, K = d["T"], d["k"], d["E"], d["x"].shape[1]
    G = lambda *s, dt=BF: Guarded(s, dt)  # noqa: E731
    cases = [("route", (G(T, k, dt=I32), G(T, k, dt=F32))), ("sort_rows", (G(T, k, dt=I32), G(E, dt=I32))),
             ("gather_quantize", (G(T * k, K, dt=torch.uint8), G(K // 128, T * k, dt=F32))),
             ("combine_rows_bwd", (G(T * k, K), G(T, k, dt=F32))), ("norm_join", (G(T, K, dt=F32), G(T, K)))]
    for name, outs in cases:
        want = CALLS[name](d)
        got = CALLS[name](d, out=tuple(o.t for o in outs))
        for a, b, o in zip(want, got, outs):
            o.check(name)
            assert b.data_ptr() == o.t.data_ptr() and _same(a, b)
    for name, o in (("route_bwd", G(T, E, dt=F32)), ("gather_rows", G(T * k, K)), ("combine_rows", G(T, K))):
        got = CALLS[name](d, out=o.t)
        o.check(name)
        assert got is o.t and _same(got, CALLS[name](d))


def test_refusals_of_layouts_on_the_gpu(data):
    d = data
    T, k = d["T"], d["k"]
    strided = torch.empty((T, 2 * d["x"].shape[1]), dtype=BF, device="cuda")[:, ::2]
    for call in (lambda: gmm.gather_rows(strided, d["rows"]), lambda: gmm.gather_rows(d["x"], d["rows"].t()),
                 lambda: gmm.gather_rows(d["x"][1:], d["rows"]), lambda: gmm.gather_rows(d["xf"], d["rows"]),
                 lambda: gmm.combine_rows(d["y"][1:], d["rows"]), lambda: gmm.combine_rows(d["y"], d["rows"].long()),
                 lambda: gmm.route(d["logits"].t(), k), lambda: gmm.route(d["logits"], k, bias=d["bias"][1:]),
                 lambda: gmm.route_bwd(d["dw"][:, 1:], d["logits"], d["ids"]),
                 lambda: gmm.sort_rows(d["ids"].t(), 4), lambda: gmm.norm_join(d["xf"], d["b"].t()),
                 lambda: gmm.norm_join(d["x"], d["b"], w_next=d["col"].bfloat16()),
                 lambda: gmm.norm_join_bwd(d["xf"], d["b"], d["x"], d["b"], w_next=d["col"]),
                 lambda: gmm.clip_grads([strided], 1.0), lambda: gmm.clip_grads([d["x"], d["x"].cpu()], 1.0)):
        with pytest.raises(ValueError, match="expected a contiguous CUDA tensor"):
            call()
    for call in (lambda: gmm.norm_join(d["x"]), lambda: gmm.norm_join(d["x"], w_post=d["col"], w_next=d["col"]),
                 lambda: gmm.norm_join_bwd(d["x"], d["b"], d["x"], d["b"]), lambda: gmm.route(d["logits"], 0),
                 lambda: gmm.sort_rows(d["ids"], 0), lambda: gmm.clip_grads([d["x"]], 1.0, out=[d["x"][1:]])):
        with pytest.raises(ValueError):
            call()
    odd = torch.empty(T * 512 + 1, dtype=BF, device="cuda")[1:].view(T, 512)  # 2 bytes behind a 16-byte boundary
    for call in (lambda: gmm.gather_rows(odd, d["rows"]), lambda: gmm.norm_join(odd, d["b"], w_next=d["col"]),
                 lambda: gmm.gather_quantize(d["x"][:, :200].contiguous(), d["rows"]),
                 lambda: gmm.clip_grads([d["x"]], -1.0), lambda: gmm.clip_grads([d["x"]], math.nan),
                 lambda: gmm.norm_join(d["x"], d["b"], eps=-1.0), lambda: gmm.sort_rows(d["ids"], 5000)):
        with pytest.raises(gmm.GmmError):
            call()
