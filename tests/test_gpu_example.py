"""The example's training and serving runs: the loss falls at every step, and the
block served in 4 bits gives what its formats say, worked out in 64 bits from the
trained weights (ffn_ref).

Bound on the served output, as a share of its norm: one bf16 rounding (2^-9) on
the way out; h is rounded to bf16 before its quantisation, and an h whose fp32 sum
(2^-18 off at most) crosses a bf16 rounding boundary (one in 2^-18 / 2^-9 = 1/512
at most) moves by 2^-8 and, at worst, its code by half of its value: sqrt(1/512) / 2
= 0.022 of h's norm; 0.03 covers both."""
import numpy as np
import pytest

from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32
from tests import ffn_ref as R
from tests.gpu_util import bf16_to_np64

pytestmark = pytest.mark.gpu


def _bits(t):
    import torch
    return t.bfloat16().view(torch.int16).cpu().numpy().view(np.uint16)


def _rounded(bits):
    """What rows of bf16 stand for in MXFP4."""
    return R.mx4_values(*R.mx4_quantize(bits))


def test_example_trains_and_serves():
    from examples.moe_block import main
    losses, block, x, sizes, served = main(["--steps", "8"])
    assert losses[-1] < 0.9 * losses[0]
    assert all(b < a for a, b in zip(losses, losses[1:]))
    n = sizes.cpu().numpy()
    w = _rounded(np.ascontiguousarray(_bits(block.w).transpose(0, 2, 1))).transpose(0, 2, 1)
    w2 = _rounded(np.ascontiguousarray(_bits(block.w2).transpose(0, 2, 1))).transpose(0, 2, 1)
    h, _, _, _ = R.swiglu_fwd(_rounded(_bits(x)), w, n)
    hb = (R.bf16_round(h).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    y, _ = R.grouped(_rounded(hb), w2, n)
    off = np.linalg.norm(bf16_to_np64(served) - y) / np.linalg.norm(y)
    assert off < 0.03, off
    assert np.array_equal(bf16_bits_to_f32(hb).astype(np.float64), R.bf16_round(h))
