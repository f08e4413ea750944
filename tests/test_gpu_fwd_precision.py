"""How exact the gated forward's fp32 sums are where they are returned in fp32, the scales of
the 8-bit checkpoint, for any K.

Bound.  The tensor core adds 16 terms a step to its fp32 accumulator and truncates: half an
ulp a step on average.  An ulp is 0.72 * 2^-23 of a value on average, and the sums that give a
scale, the largest of 128, grow about linearly, so that their partial sums are half of them on
average: 0.5 * 0.72 * 2^-23 * 0.5 * steps = 2.1e-8 * steps of the sum.  The kernel adds up at
most 512 terms so, 32 steps, 6.9e-7, and joins these in fp32 with rounding (some 2^-24 each,
of both signs).  1e-6 leaves room for a spread of the sums' shapes; 4096 terms in one
accumulator would be 5e-6 off, 2048 terms 2.7e-6."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32, normal_bf16
from tests import ffn_ref as R
from tests.gpu_util import bf16_to_np64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [128, 512, 640, 1024, 2048, 4096])
def test_scales_of_the_checkpoint(K):
    rng = np.random.default_rng(K)
    sizes, M, N = [200, 0, 130], 330, 256
    x, w = normal_bf16((M, K), 1.0, rng, outlier_p=0.01), normal_bf16((3, K, 2 * N), K ** -0.5, rng)
    st = to_dev(np.array(sizes, np.int32))
    h, (_, scales) = gmm.swiglu_fwd(to_dev_bf16(x), to_dev_bf16(w), st, keep="e4m3")
    x64, w64 = (bf16_bits_to_f32(v).astype(np.float64) for v in (x, w))
    gu, _ = R.grouped(x64, w64, sizes)
    want = np.abs(gu).reshape(M, -1, 128).max(2).T / 448
    got = scales.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= 1e-6 * np.linalg.norm(want)
    # h does not depend on the form that is kept
    h2, _ = gmm.swiglu_fwd(to_dev_bf16(x), to_dev_bf16(w), st, keep="bf16")
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    assert np.all(np.isfinite(bf16_to_np64(h)))
