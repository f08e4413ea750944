"""The router and its gradient against the plain 64-bit implementation: ids equal, and
weights within the bounds of layer_ref (a weight is one exp of a rounded difference over
a sum of E of them)."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 2, 2), (3, 31, 4), (5, 32, 32), (7, 33, 8), (16, 256, 8), (9, 255, 6), (33, 384, 1), (6, 513, 8),
         (4, 1024, 16), (3, 2047, 8), (2, 4096, 32), (1027, 64, 6)]


def _logits(T, E, dtype, seed, masked=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=gen, device="cuda") * 2
    l = (l * 8).round() / 8  # many ties
    if masked and T > 2:
        l[0] = -math.inf  # a token without experts
        l[1, 1:] = -math.inf
        l[2, ::2] = math.nan
        l[-1, 0] = 0.0
        l[-1, E // 2] = -0.0
        if T > 4:
            l[3] = torch.finfo(torch.bfloat16).min  # a mask of the type's lowest value
            l[4] *= 40  # far apart
    return l.to(dtype)


def _rel(l):
    """Bound of a weight: the sum's chain, a handful of roundings, and that of l - m."""
    far = torch.where(torch.isfinite(l), l, 0.0).abs().amax(1, keepdim=True).double().clamp(max=200.0)
    return R.U * (l.shape[1] / 32 + 5 + 2 * far) + R.F32


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route(T, E, k, dtype, score, renorm):
    l = _logits(T, E, dtype, T + E)
    bias = None
    if k % 2 == 0:
        bias = torch.randn(E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.25
        if E > 40:
            bias[7], bias[9] = -math.inf, math.nan
    gi, gw = Guarded((T, k), torch.int32), Guarded((T, k), torch.float32)
    gmm.route(l, k, bias=bias, score=score, renorm=renorm, scale=1.5, out=(gi.t, gw.t))
    gi.check("ids")
    gw.check("weights")
    want = torch.from_numpy(R.chosen(l, bias, k))
    assert torch.equal(gi.t.cpu(), want)
    ref = R.route_weights(l.double(), gi.t, score, renorm, 1.5)
    R.assert_within(gw.t, ref, _rel(l) * ref.abs(), "weights")


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_bwd(T, E, k, dtype, score, renorm):
    l = _logits(T, E, dtype, 3 * T + E)
    ids = torch.from_numpy(R.chosen(l, None, k)).cuda()
    if T > 4 and k > 1:
        ids[2] = ids[2].roll(1)
        ids[4, 1], ids[4, 0] = ids[4, 0].item(), E  # one out of range
        ids[3, 1] = ids[3, 0].item()                # one named twice
        ids[T - 1, 0] = -7
    dw = torch.randn((T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    out = Guarded((T, E), dtype)
    gmm.route_bwd(dw, l, ids, score=score, renorm=renorm, scale=0.5, out=out.t)
    out.check("dlogits")
    ref, mag = R.route_bwd(dw, l, ids, score, renorm, 0.5)
    rounding = R.BF16 * ref.abs() if dtype == torch.bfloat16 else 0.0
    R.assert_within(out.t, ref, _rel(l) * 3 * mag + rounding, "dlogits")


def test_route_of_nothing():
    ids, w = gmm.route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert gmm.route_bwd(w, torch.empty((0, 8), device="cuda"), ids).shape == (0, 8)


def test_more_choices_than_experts_are_refused():
    with pytest.raises(gmm.GmmError):
        gmm.route(torch.zeros((2, 4), device="cuda"), 5)


def test_sigmoid_weights_of_far_logits_keep_their_ratio():
    """Sigmoids below the smallest float: renorm's weights are still the softmax of their logarithms."""
    l = torch.tensor([[-200.0, -201.0, -300.0]], device="cuda")
    _, w = gmm.route(l, 2, score="sigmoid", renorm=True)
    want = torch.softmax(torch.tensor([[-200.0, -201.0]], device="cuda").double(), 1)
    R.assert_within(w, want, 2 * R.F32 * want, "weights")


def test_an_infinite_logit_takes_the_sigmoid_of_one_and_poisons_the_softmax():
    l = torch.tensor([[math.inf, 1.0, 0.0]], device="cuda")
    ids, w = gmm.route(l, 2, score="sigmoid")
    assert ids.tolist() == [[0, 1]] and w[0, 0].item() == 1.0
    _, w = gmm.route(l, 2, score="softmax")
    assert math.isnan(w[0, 0].item())
