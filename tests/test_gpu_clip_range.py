"""Clipping where max_norm / norm leaves the normal numbers of fp32: the scaled gradients
are still half a step of their type and a few roundings of fp32 (F32) from the formula's."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# largest value, max_norm: the factor is 1e-37 (normal), subnormal, or 0 in fp32
RANGES = [(1e30, 1e-7), (2e38, 1e-3), (1e38, 1e-5), (1e38, 1e-8), (2e38, 1e-20), (1e30, 1e-30), (1e-2, 1e-40)]
# zeros in front of the values: one launch for few, two for many; odd: off a 16-byte boundary
LAYOUTS = [(0, False), (0, True), (70000, False), (400000, False), (400001, True)]


@pytest.mark.parametrize("value,max_norm", RANGES)
@pytest.mark.parametrize("zeros,odd", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_factor_below_the_normal_numbers(value, max_norm, zeros, odd, dtype, in_place):
    gen = torch.Generator(device="cuda").manual_seed(zeros)
    flat = torch.zeros(zeros + 1001, dtype=dtype, device="cuda")
    v = torch.rand(1000, generator=gen, device="cuda", dtype=torch.float64) * 2 - 1
    v *= 0.01  # small beside the largest
    v[0], v[1] = 1.0, -0.5
    flat[zeros + 1:] = (v * value).to(dtype)
    grads = [flat[1:] if odd else flat[1:].clone(), flat[zeros + 1:zeros + 8].clone().view(7, 1)]
    want = [g.double() for g in grads]
    norm = torch.cat([w.flatten() for w in want]).norm().item()
    assert norm < torch.finfo(F32).max
    out = None if in_place else [torch.full_like(g, math.nan) for g in grads]
    got = gmm.clip_grads(grads, max_norm, out=out).item()
    assert abs(got - norm) <= 2 * R.F32 * norm
    held = torch.tensor(max_norm, dtype=F32).double().item()  # the C entry point takes fp32
    half = R.U if dtype == F32 else R.BF16
    step = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # of the subnormal numbers
    for g, w in zip(out or grads, want):
        w = w * (held / norm)
        off = (g.double() - w).abs()
        assert bool((off <= (half + 2 * R.F32) * w.abs() + step).all()), off.max().item()


def test_a_largest_norm_of_zero_gives_zeros_whatever_the_norm():
    for value in (1e-40, 1.0, 3e38):
        g = torch.full((1,), value, device="cuda")
        gmm.clip_grads([g], 0.0)
        assert g.item() == 0.0
