"""The norms beside values that are not finite, against the plain 64-bit implementation, with
the bounds of test_gpu_norm_join."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# one cluster's rows, several rows a CTA, one row a CTA, rows of over 4096 columns
SIZES = [(9, 264), (700, 1024), (200, 2304), (330, 4104)]


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
    x, dout, b, dn = _rnd(gen, T, K, dt=stream), _rnd(gen, T, K, dt=stream), _rnd(gen, T, K, dt=BF), _rnd(gen, T, K, dt=BF)
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
    ref, mag = R.norm_join_bwd(dout.double(), None if dn is None else dn.double(), x.double(), b.double(), None,
                               None if g is None else g.double(), how["w_next"].double() if next_norm else None, 0.8, 1.3,
                               1e-6)
    R.assert_within(got[1], ref[1], R.BF16 * ref[1].abs() + 2 * R.F32 * mag[1], "db")
