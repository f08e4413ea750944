"""The norms at the ends of fp32's range and beside values that are not finite, against the
plain 64-bit implementation, with the bounds of test_gpu_norm_join."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# one cluster's rows, several rows a CTA, one row a CTA, rows of over 4096 columns
SIZES = [(9, 264), (700, 1024), (200, 2304), (330, 4104)]
NAMES = ("dx", "db", "dw_post", "dgate", "dw_next")


def _rnd(gen, *s, dt=F32, std=1.0):
    return (torch.randn(s, generator=gen, device="cuda") * std).to(dt)


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("gate", [None, "column", "full"])
@pytest.mark.parametrize("next_norm", [False, True])
def test_the_blocks_gradient_without_its_norm_does_not_read_the_block(T, K, stream, gate, next_norm):
    """Without w_post, out is linear in b: db = block_scale * gate * D whatever b holds.  (A
    gate's gradient does contain b.)"""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dout, b, dn = (_rnd(gen, T, K, dt=t) for t in (stream, stream, BF, BF))
    g = {None: None, "column": _rnd(gen, K), "full": _rnd(gen, T, K, dt=BF)}[gate]
    how = dict(gate=g, w_next=_rnd(gen, K) if next_norm else None, residual_scale=0.8, block_scale=1.3)
    dn = dn if next_norm else None
    want = gmm.norm_join_bwd(dout, dn, x, b, **how)
    bad = b.clone()
    bad[0, 0], bad[T // 2, 1::7], bad[T - 1, K - 1] = math.inf, math.nan, -math.inf
    got = gmm.norm_join_bwd(dout, dn, x, bad, **how)
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1], want[1])
    if next_norm:
        assert torch.equal(got[4], want[4])
    ref, mag = R.norm_join_bwd(*(None if v is None else v.double() for v in (dout, dn, x, b, None, g, how["w_next"])),
                               0.8, 1.3, 1e-6)
    R.assert_within(got[1], ref[1], R.BF16 * ref[1].abs() + 2 * R.F32 * mag[1], "db")


# root mean squares of a row's out and b; their squares are normal numbers of fp32, and sum to less than 3.4e38
SCALES = [(1.0, 1.0), (4e-19, 1.0), (1.0, 4e-19), (1e-16, 1e-16), (1e17, 1.0), (1.0, 1e17), (1e17, 1e17), (4e-19, 1e17),
          (1e17, 4e-19)]


def _scaled(gen, T, K, stream):
    s = torch.tensor(SCALES, device="cuda")[torch.arange(T, device="cuda") % len(SCALES)]
    x, b = _rnd(gen, T, K) * s[:, :1], _rnd(gen, T, K) * s[:, 1:]
    return x.to(stream), b.to(BF)


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("post,gate", [(True, None), (True, "column"), (True, "full"), (False, "column")])
def test_gradients_of_tiny_and_huge_rows_without_eps(T, K, stream, post, gate):
    """The reciprocal roots are 2.5e18 there, and their cubes past fp32's range; the gradients are not."""
    gen = torch.Generator(device="cuda").manual_seed(T + 1)
    out, b = _scaled(gen, T, K, stream)
    w = dict(w_post=_rnd(gen, K) if post else None, w_next=_rnd(gen, K),
             gate={None: None, "column": _rnd(gen, K), "full": _rnd(gen, T, K, dt=BF)}[gate])
    # in part along the rows, so that their products' means do not vanish
    along = b.sign()
    for v in (w["w_post"], w["gate"]):
        along = along if v is None else along * v.sign()
    dout, dn = (_rnd(gen, T, K) + along).to(stream), (_rnd(gen, T, K) + out.sign() * w["w_next"].sign()).to(BF)
    got = gmm.norm_join_bwd(dout, dn, out, b, **w, residual_scale=0.8, block_scale=1.3, eps=0.0)
    ref, mag = R.norm_join_bwd(dout.double(), dn.double(), out.double(), b.double(),
                               *(None if w[n] is None else w[n].double() for n in ("w_post", "gate", "w_next")), 0.8, 1.3,
                               0.0)
    for i, name in enumerate(NAMES):
        if ref[i] is None:
            assert got[i] is None
            continue
        assert bool(ref[i].abs().max() < torch.finfo(F32).max), name  # it has a value in fp32
        half = R.BF16 if got[i].dtype == BF else 0.0
        chain = T * R.U if ref[i].dim() == 1 else 0.0
        R.assert_within(got[i], ref[i], half * ref[i].abs() + (2 * R.F32 + chain) * mag[i], name)


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("stream", [BF, F32])
def test_norms_of_tiny_and_huge_rows_without_eps(T, K, stream):
    gen = torch.Generator(device="cuda").manual_seed(T + 2)
    x, b = _scaled(gen, T, K, stream)
    w_post, w_next = _rnd(gen, K), _rnd(gen, K)
    out, n = gmm.norm_join(x, b, w_post, None, w_next, residual_scale=0.8, block_scale=1.3, eps=0.0)
    want, wn, mag = R.norm_join(x.double(), b.double(), w_post.double(), None, w_next.double(), 0.8, 1.3, 0.0)
    r = R.unit(want, 0.0)[1]
    half = R.BF16 if stream == BF else 0.0
    R.assert_within(out, want, half * want.abs() + R.F32 * mag, "out")
    R.assert_within(n, wn, R.BF16 * wn.abs() + 2 * R.F32 * r * mag * w_next.abs() + R.F32 * wn.abs(), "n")
    _, n = gmm.norm_join(x, w_next=w_next, eps=0.0)
    wn = R.unit(x.double(), 0.0)[0] * w_next.double()
    R.assert_within(n, wn, (R.BF16 + 2 * R.F32) * wn.abs(), "n in front of a first block")
