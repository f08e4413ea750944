"""The weight gradient from 8-bit checkpoints against the product of what the codes stand
for, without the kernel's rounding of each expanded value, and its split rows with reused
metadata.

Bound.  bf16 keeps 8 bits, so rounding a value of [1, 2) errs by up to 2^-8, with an rms of
2^-7 / sqrt(12), 2.26e-3 / value; over values whose mantissas are spread as those of products
are, 1.66e-3 of the value.  The kernel rounds each code times its scale so, and its result
once more; with terms of random signs the errors add up as squares, sqrt(2) 1.66e-3 = 2.3e-3
of the result's norm.  1.05 sqrt(2) 2^-9 = 2.9e-3 leaves a quarter for the sampling of a few
thousand elements and the mantissas of e4m3 codes."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32, normal_bf16
from tests import ffn_ref as R
from tests.gpu_util import bf16_to_np64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

SPLIT = [([5000], 5000, 128, 128), ([4097], 4100, 256, 384), ([0, 9000, 70, 1], 9100, 384, 256),
         ([600, 2500], 3100, 512, 256)]
WHOLE = [([1], 1, 128, 128), ([1, 127, 128, 129, 0, 2], 400, 256, 384), ([1000, 3, 700, 0, 0, 297], 2000, 1152, 512)]


def _inputs(sizes, M, K, N):
    rng = np.random.default_rng(3 * M + K + N)
    xq, xs = gmm.quantize_lhs(to_dev_bf16(normal_bf16((M, K), 1.0, rng)))
    dy = normal_bf16((M, N), 1.0, rng)
    return xq, xs, to_dev_bf16(dy), bf16_bits_to_f32(dy).astype(np.float64), to_dev(np.array(sizes, np.int32))


@pytest.mark.parametrize("sizes,M,K,N", SPLIT + WHOLE)
def test_against_the_unrounded_product(sizes, M, K, N):
    xq, xs, dy, dy64, st = _inputs(sizes, M, K, N)
    got = bf16_to_np64(gmm.tgmm_ckpt(xq, xs, dy, st))
    assert np.all(np.isfinite(got))
    x = R.dequant_e4m3(xq.cpu().numpy(), xs.cpu().numpy())
    off = R.offsets(sizes)
    for g, n in enumerate(sizes):
        r = slice(off[g], off[g + 1])
        if n >= 100:
            dw = x[r].T @ dy64[r]
            assert np.linalg.norm(got[g] - dw) <= 1.05 * np.sqrt(2) * 2.0 ** -9 * np.linalg.norm(dw)


@pytest.mark.parametrize("sizes,M,K,N", SPLIT + WHOLE)
def test_reused_metadata(sizes, M, K, N):
    """Order and offsets from the workspace instead of group_sizes: the same bits, rows split or not."""
    G = len(sizes)
    assert (gmm.tgmm_fp8_ckpt_scratch_bytes(G, M, K, N) > 0) == ((sizes, M, K, N) in SPLIT)
    xq, xs, dy, _, st = _inputs(sizes, M, K, N)
    work = gmm.Workspace(G, M)
    want = gmm.tgmm_ckpt(xq, xs, dy, st, workspace=work)
    got = gmm.tgmm_ckpt(xq, xs, dy, None, workspace=work)
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    alone = gmm.group_metadata(st, M)  # by the metadata pass
    got = gmm.tgmm_ckpt(xq, xs, dy, None, workspace=alone)
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    assert work.status() == alone.status() == 0
