"""Randomized sweep of the feed-forward block's operators over shapes and routings, against
the plain 64-bit implementations and bounds of ffn_ref.  Each case draws G (past 256 groups
too, where a metadata pass runs), M, K, N and a routing, and checks every operator, its
zeros in the rows of no group and, with the metadata reused, the same bits again."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32, normal_bf16
from tests import ffn_ref as R
from tests.gpu_util import bf16_to_np64, to_dev, to_dev_bf16
from tests.test_gpu_random_sweep import _sizes

pytestmark = pytest.mark.gpu


def _f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def _same(a, b):
    for x, y in zip(a, b, strict=True):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def _draw(rng):
    while True:
        G = int(rng.choice([1, 2, 5, 17, 64, 256, 257, 600]))
        M = int(np.exp(rng.uniform(0, np.log(2500))))
        K, N = (128 * int(v) for v in rng.integers(1, 8, 2))
        if G * K * N <= 6e6:
            return G, M, K, N


@pytest.mark.parametrize("seed", range(201, 217))
def test_random_sweep(seed):
    rng = np.random.default_rng(seed)
    G, M, K, N = _draw(rng)
    sizes = _sizes(rng, G, M)
    S, what = int(sizes.sum()), f"G {G} M {M} K {K} N {N} sizes {sizes.tolist()[:20]}"
    st, work = to_dev(sizes), gmm.Workspace(G, M)
    x, dy = normal_bf16((M, K), 1.0, rng, outlier_p=0.01), normal_bf16((M, K), 1.0, rng)
    w, w2 = normal_bf16((G, K, 2 * N), K ** -0.5, rng), normal_bf16((G, N, K), N ** -0.5, rng)
    xd, dyd, wd, w2d = (to_dev_bf16(v) for v in (x, dy, w, w2))

    # gated forward, both forms of what is kept
    h, gu = gmm.swiglu_fwd(xd, wd, st, workspace=work)
    _same((h, gu), gmm.swiglu_fwd(xd, wd, None, workspace=work))
    rh, rh_err, rgu, err = R.swiglu_fwd(_f64(x), _f64(w), sizes)
    R.check(bf16_to_np64(h), rh, rh_err, "h: " + what)
    R.check(bf16_to_np64(gu), rgu, R.BF16 * np.abs(rgu) + err + R.TINY, "gate | up: " + what)
    h8, kept = gmm.swiglu_fwd(xd, wd, st, keep="e4m3", workspace=work)
    _same((h,), (h8,))
    codes, scales = (t.cpu().numpy() for t in kept)
    step = np.repeat(scales.T.astype(np.float64), 128, axis=1) * 2.0 ** -10
    R.check(R.dequant_e4m3(codes, scales), rgu, 2.0 ** -4 * np.abs(rgu) * 1.0001 + step + 2 * err + R.TINY,
            "codes: " + what)

    # backward from both forms
    for k, v in ((gu, bf16_to_np64(gu)), (kept, R.dequant_e4m3(codes, scales))):
        dgu, hb = gmm.swiglu_bwd(dyd, w2d, k, st, workspace=work)
        _same((dgu, hb), gmm.swiglu_bwd(dyd, w2d, k, None, workspace=work))
        rd, rd_err, rhb, rhb_err = R.swiglu_bwd(_f64(dy), _f64(w2), v, sizes)
        R.check(bf16_to_np64(dgu), rd, rd_err, "dgu: " + what)
        R.check(bf16_to_np64(hb), rhb, rhb_err, "h again: " + what)
        assert not torch.any(dgu[S:].view(torch.int16)) and not torch.any(hb[S:].view(torch.int16))

    # weight gradient from x's codes
    xq, xs = gmm.quantize_lhs(xd)
    dw = gmm.tgmm_ckpt(xq, xs, dgu, st, workspace=work)
    _same((dw,), (gmm.tgmm_ckpt(xq, xs, dgu, None, workspace=work),))
    ref, err = R.wgrad(xq.cpu().numpy(), xs.cpu().numpy(), bf16_to_np64(dgu), sizes)
    R.check(bf16_to_np64(dw), ref, err, "dw: " + what)

    # MXFP4: quantisers bit for bit, plain and fused products
    c, b = R.mx4_quantize(x)
    q4, w4 = gmm.mx4_quantize_lhs(xd), gmm.mx4_quantize_rhs(wd)
    assert np.array_equal(R.unpack4(q4[0].cpu().numpy()), c) and np.array_equal(R.mx4_lhs_scales(q4[1].cpu().numpy()), b)
    cw, bw = R.mx4_quantize(np.ascontiguousarray(w.transpose(0, 2, 1)))
    assert np.array_equal(R.unpack4(w4[0].cpu().numpy()), cw) and np.array_equal(R.mx4_rhs_scales(w4[1].cpu().numpy()), bw)
    x4, w44 = R.mx4_values(c, b), R.mx4_values(cw, bw).transpose(0, 2, 1)
    out = gmm.mx4_fwd(*q4, *w4, st, workspace=work)
    _same((out,), (gmm.mx4_fwd(*q4, *w4, None, workspace=work),))
    ref, mag = R.grouped(x4, w44, sizes)
    R.check(bf16_to_np64(out), ref, R.BF16 * np.abs(ref) + R.SUM * mag + R.TINY, "MXFP4 product: " + what)
    h4, hq, hs = gmm.mx4_fwd_swiglu_quant(*q4, *w4, st, workspace=work)
    ref, err, _, _ = R.swiglu_fwd(x4, w44, sizes)
    R.check(bf16_to_np64(h4), ref, err, "MXFP4 gate/up: " + what)
    _same((hq, hs), gmm.mx4_quantize_lhs(h4))
    _same((h4,), (gmm.mx4_fwd(*q4, *w4, st, fuse=True, workspace=work),))
    assert not torch.any(out[S:].view(torch.int16)) and not torch.any(h4[S:].view(torch.int16))
    assert work.status() == 0
