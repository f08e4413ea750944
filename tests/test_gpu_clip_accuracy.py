"""Clipping's norm and factor rounded once.  The gradients are 0, 1 and -1, so that a thread's
sums are whole numbers that fp32 holds, whatever their order; what is left are the roundings
of the norm (half a step, U, of itself) and of the factor, which the scaled values are (U).
Sums of sums and the root held in twice fp32's bits add 2^-40 of them at most: 1.01 U."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

F32 = torch.float32
ONCE = 1.01 * R.U


@pytest.mark.parametrize("counts", [[3], [7, 11], [1000], [100003], [262144], [262145], [3000001, 77], [33333333, 5],
                                    [4097] * 300, [257] * 2003, [123456789, 98765432]],
                         ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("share", [0.31, 0.7, 1e-3])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_and_factor_are_rounded_once(counts, share, in_place):
    gen = torch.Generator(device="cuda").manual_seed(sum(counts))
    grads = [torch.randint(-1, 2, (c,), generator=gen, device="cuda", dtype=torch.int8).to(F32) for c in counts]
    grads[0][0] = 1.0
    signs = [g.to(torch.int8) for g in grads]
    norm = math.sqrt(sum(int(g.count_nonzero()) for g in signs))
    max_norm = torch.tensor(share * norm, dtype=F32).item()
    out = None if in_place else [torch.empty_like(g) for g in grads]
    got = gmm.clip_grads(grads, max_norm, out=out).item()
    assert abs(got - norm) <= ONCE * norm, (got - norm) / norm / R.U
    by = (out or grads)[0][0].item()
    assert abs(by - max_norm / norm) <= ONCE * max_norm / norm, (by - max_norm / norm) / (max_norm / norm) / R.U
    for o, sign in zip(out or grads, signs, strict=True):
        assert torch.equal(o, by * sign)
