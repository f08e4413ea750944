"""The norms before and after a block with its gate and the residual stream, and their
gradient, against the plain 64-bit implementation.  A value is off by at most F32 of the
magnitudes it is made of (a dozen fp32 operations and a sum of K squares in chains of 8 +
10 + 5) and one rounding where it is bf16; a column's sum over T rows adds its chain."""
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
SIZES = [(1, 8), (64, 2048), (65, 2048), (512, 256), (513, 256), (64, 4096), (31, 2304), (2, 264), (16, 2048), (5, 4096), (3, 4104), (4, 8192), (7, 72), (1031, 1000), (2100, 256), (400, 5120)]


def _case(T, K, stream, post, gate, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T * 7 + K)
    rnd = lambda *s, dt=F32, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(dt)  # noqa: E731
    c = dict(x=rnd(T, K, dt=stream, std=3.0), b=rnd(T, K, dt=BF), w_post=rnd(K) if post else None,
             gate={None: None, "column": rnd(K), "full": rnd(T, K, dt=BF)}[gate], w_next=rnd(K))
    c["b"][:, ::17] *= 50
    c["b"][-1] = 0          # a row of nothing: eps alone under the root
    if T > 2:
        c["x"][1] *= 1e-3
    return c, rnd(T, K, dt=stream), rnd(T, K, dt=BF)


def _ref(c, *names):
    return [None if c[n] is None else c[n].double() for n in names]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("post,gate", [(True, None), (False, "column"), (True, "column"), (True, "full"), (False, None)])
def test_forward(T, K, stream, post, gate):
    c, _, _ = _case(T, K, stream, post, gate)
    out, n = Guarded((T, K), stream), Guarded((T, K), BF)
    gmm.norm_join(**c, residual_scale=0.8, block_scale=1.3, eps=EPS, out=(out.t, n.t))
    out.check("out")
    n.check("n")
    want, wn, mag = R.norm_join(*_ref(c, "x", "b", "w_post", "gate", "w_next"), 0.8, 1.3, EPS)
    r = R.unit(want, EPS)[1]
    half = R.BF16 if stream == BF else 0.0
    R.assert_within(out.t, want, half * want.abs() + R.F32 * mag, "out")
    R.assert_within(n.t, wn, R.BF16 * wn.abs() + 2 * R.F32 * r * mag * c["w_next"].abs() + R.F32 * wn.abs(), "n")


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
def test_the_norm_in_front_of_a_first_block(T, K, stream):
    c, dout, dn = _case(T, K, stream, False, None)
    x, n = gmm.norm_join(c["x"], w_next=c["w_next"], eps=EPS)
    assert x is c["x"]
    _, want, _ = R.norm_join(*_ref(c, "x"), None, None, None, *_ref(c, "w_next"), 1.0, 1.0, EPS)
    R.assert_within(n, want, (R.BF16 + 2 * R.F32) * want.abs(), "n")
    for d in (dout, None):
        got = gmm.norm_join_bwd(d, dn, c["x"], w_next=c["w_next"], residual_scale=7.0, eps=EPS)
        assert got[1] is None and got[2] is None and got[3] is None
        ref, mag = R.norm_join_bwd(None if d is None else d.double(), dn.double(), *_ref(c, "x"), None, None, None,
                                   *_ref(c, "w_next"), 1.0, 1.0, EPS)
        half = R.BF16 if stream == BF else 0.0
        R.assert_within(got[0], ref[0], half * ref[0].abs() + R.F32 * mag[0], "dx")
        R.assert_within(got[4], ref[4], (T * R.U + R.F32) * mag[4], "dw_next")


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("post,gate", [(True, None), (False, "column"), (True, "column"), (True, "full"), (False, None),
                                       (False, "full")])
def test_backward(T, K, stream, post, gate):
    c, dout, dn = _case(T, K, stream, post, gate, 5)
    out, _ = gmm.norm_join(**c, residual_scale=0.8, block_scale=1.3, eps=EPS)
    dx, db = Guarded((T, K), stream), Guarded((T, K), BF)
    rest = {k: c[k] for k in ("b", "w_post", "gate", "w_next")}
    got = gmm.norm_join_bwd(dout, dn, out, **rest, residual_scale=0.8, block_scale=1.3, eps=EPS, into=(dx.t, db.t))
    dx.check("dx")
    db.check("db")
    ref, mag = R.norm_join_bwd(dout.double(), dn.double(), out.double(), *_ref(c, "b", "w_post", "gate", "w_next"), 0.8,
                               1.3, EPS)
    for i, name in enumerate(("dx", "db", "dw_post", "dgate", "dw_next")):
        if ref[i] is None:
            assert got[i] is None
            continue
        summed = ref[i].dim() == 1
        half = R.BF16 if got[i].dtype == BF else 0.0
        R.assert_within(got[i], ref[i], half * ref[i].abs() + (2 * R.F32 + (T * R.U if summed else 0.0)) * mag[i], name)


@pytest.mark.parametrize("stream", [BF, F32])
def test_backward_without_one_of_the_gradients(stream):
    c, dout, dn = _case(50, 512, stream, True, "column", 9)
    rest = {k: c[k] for k in ("b", "w_post", "gate", "w_next")}
    zero = torch.zeros_like
    full = gmm.norm_join_bwd(dout, zero(dn), c["x"], **rest)
    less = gmm.norm_join_bwd(dout, None, c["x"], **rest)
    for a, b in zip(full, less):
        assert torch.equal(a, b)
    assert not bool(less[4].any())
    full = gmm.norm_join_bwd(zero(dout), dn, c["x"], **rest)
    for a, b in zip(full, gmm.norm_join_bwd(None, dn, c["x"], **rest)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="dout and dn"):
        gmm.norm_join_bwd(None, None, c["x"], **rest)


def test_without_a_next_norm():
    c, dout, _ = _case(33, 256, BF, True, "full", 1)
    c["w_next"] = None
    out, n = gmm.norm_join(**c, eps=EPS)
    assert n is None
    c["w_next"] = torch.ones(256, device="cuda")
    assert torch.equal(out, gmm.norm_join(**c, eps=EPS)[0])
    got = gmm.norm_join_bwd(dout, None, out, c["b"], c["w_post"], c["gate"], eps=EPS)
    assert got[4] is None
    want = gmm.norm_join_bwd(dout, None, out, c["b"], c["w_post"], c["gate"], c["w_next"], eps=EPS)
    for a, b in zip(got[:4], want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,K", [(460, 4104), (310, 8184), (155, 8192)])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("gate", [None, "column", "full"])
def test_backward_of_wide_rows_a_cta_has_several_of(T, K, stream, gate):
    c, dout, dn = _case(T, K, stream, True, gate, 3)
    rest = {k: c[k] for k in ("b", "w_post", "gate", "w_next")}
    out, _ = gmm.norm_join(**c, eps=EPS)
    for d, e in ((dout, dn), (None, dn), (dout, None)):
        got = gmm.norm_join_bwd(d, e, out, **rest, eps=EPS)
        ref, mag = R.norm_join_bwd(None if d is None else d.double(), (torch.zeros_like(dn) if e is None else e).double(),
                                   out.double(), *_ref(c, "b", "w_post", "gate", "w_next"), 1.0, 1.0, EPS)
        for i, name in enumerate(("dx", "db", "dw_post", "dgate", "dw_next")):
            if ref[i] is None:
                continue
            half = R.BF16 if got[i].dtype == BF else 0.0
            off = (2 * R.F32 + (T * R.U if ref[i].dim() == 1 else 0.0)) * mag[i]
            R.assert_within(got[i], ref[i], half * ref[i].abs() + off, name)
    d, b = dout.clone(), c["b"].clone()  # in place
    want = gmm.norm_join_bwd(dout, dn, out, **rest, eps=EPS)
    for u, v in zip(gmm.norm_join_bwd(d, dn, out, b, c["w_post"], c["gate"], c["w_next"], eps=EPS, into=(d, b)), want):
        assert (u is None and v is None) or torch.equal(u, v)


@pytest.mark.parametrize("stream", [BF, F32])
def test_in_place(stream):
    c, dout, dn = _case(700, 1024, stream, True, "column", 2)
    rest = {k: c[k] for k in ("b", "w_post", "gate", "w_next")}
    out, n = gmm.norm_join(**c)
    x, b = c["x"].clone(), c["b"].clone()
    gmm.norm_join(x, b, c["w_post"], c["gate"], c["w_next"], out=(x, b))
    assert torch.equal(x, out) and torch.equal(b, n)
    want = gmm.norm_join_bwd(dout, dn, out, **rest)
    for which in ("dn", "b"):
        d, e, b = dout.clone(), dn.clone(), c["b"].clone()
        got = gmm.norm_join_bwd(d, e, out, b, c["w_post"], c["gate"], c["w_next"], into=(d, e if which == "dn" else b))
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_no_tokens():
    x, b = torch.empty((0, 256), device="cuda"), torch.empty((0, 256), dtype=BF, device="cuda")
    w = torch.ones(256, device="cuda")
    out, n = gmm.norm_join(x, b, w, w, w)
    assert out.shape == n.shape == (0, 256)
    got = gmm.norm_join_bwd(x, b, out, b, w, w, w)
    assert got[0].shape == (0, 256)
    for g in got[2:]:
        assert g.tolist() == [0.0] * 256


def test_runs_repeat_bit_for_bit():
    c, dout, dn = _case(3000, 512, F32, True, "column", 4)
    rest = {k: c[k] for k in ("b", "w_post", "gate", "w_next")}
    first = gmm.norm_join_bwd(dout, dn, c["x"], **rest)
    for _ in range(3):
        for a, b in zip(first, gmm.norm_join_bwd(dout, dn, c["x"], **rest)):
            assert torch.equal(a, b)
