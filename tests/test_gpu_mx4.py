"""MXFP4: the quantisers bit for bit, the grouped product and its fused forms
against a plain 64-bit implementation (ffn_ref), ragged and empty groups, both
unit widths, NaN blocks, other streams."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import normal_bf16
from tests import ffn_ref as R
from tests.gpu_util import Guarded, bf16_to_np64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def _awkward(shape, rng):
    """Values on and around the ties of E2M1, zero blocks, subnormals, the largest and smallest exponents."""
    v = normal_bf16(shape, 1.0, rng, outlier_p=0.02)
    flat = v.reshape(-1, 32)
    for i in range(0, len(flat), 7):
        kind = (i // 7) % 6
        if kind == 0:
            flat[i] = 0
        elif kind == 1:  # subnormal bf16
            flat[i] = rng.integers(0, 128, 32) | (rng.integers(0, 2, 32) << 15)
        elif kind == 2:  # the largest finite exponent
            flat[i] = (254 << 7) | rng.integers(0, 128, 32)
        elif kind == 3:  # every tie of the grid in a block of scale 1, both signs
            t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4, np.float32)
            t[16:] *= -1
            flat[i] = (t.view(np.uint32) >> 16).astype(np.uint16)
        elif kind == 4:  # negative zeros
            flat[i] = 0x8000
        else:  # the smallest normal exponents
            flat[i] = (rng.integers(1, 4, 32) << 7) | rng.integers(0, 128, 32)
    return v


@pytest.mark.parametrize("M,K", [(1, 128), (7, 256), (8, 128), (65, 384), (300, 1152)])
def test_quantize_lhs_bit_exact(M, K):
    rng = np.random.default_rng(M + K)
    x = _awkward((M, K), rng)
    xq, xs = Guarded((M, K // 2), torch.uint8), Guarded((K // 128, M, 4), torch.uint8)
    gmm.mx4_quantize_lhs(to_dev_bf16(x), out=(xq.t, xs.t))
    xq.check("codes")
    xs.check("scales")
    codes, byte = R.mx4_quantize(x)
    assert np.array_equal(R.unpack4(xq.t.cpu().numpy()), codes)
    assert np.array_equal(R.mx4_lhs_scales(xs.t.cpu().numpy()), byte)


@pytest.mark.parametrize("G,K,N", [(1, 128, 128), (3, 384, 256), (2, 256, 640)])
def test_quantize_rhs_bit_exact(G, K, N):
    rng = np.random.default_rng(G + K + N)
    wt = _awkward((G, N, K), rng)  # awkward along K
    wq, ws = gmm.mx4_quantize_rhs(to_dev_bf16(np.ascontiguousarray(wt.transpose(0, 2, 1))))
    codes, byte = R.mx4_quantize(wt)
    assert np.array_equal(R.unpack4(wq.cpu().numpy()), codes)
    assert np.array_equal(R.mx4_rhs_scales(ws.cpu().numpy()), byte)


def test_quantize_marks_infinite_blocks():
    x = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    x[0, 40], x[1, 200] = float("inf"), float("nan")
    _, xs = gmm.mx4_quantize_lhs(x)
    byte = R.mx4_lhs_scales(xs.cpu().numpy())
    want = np.full((2, 8), 125)  # 1.0: exponent 127 - 2
    want[0, 1] = want[1, 6] = 255
    assert np.array_equal(byte, want)


EDGE = [
    ([512], 512, 256, 256),
    ([1], 1, 128, 128),
    ([0, 300, 0, 212], 512, 384, 256),
    ([1, 127, 128, 129, 0, 2], 400, 256, 384),
    ([5, 0, 0, 9], 20, 128, 640),
    ([130, 0, 150], 300, 640, 128),
    ([0, 0, 0], 64, 256, 256),
    ([1000, 3, 700, 0, 0, 297], 2100, 1152, 512),
    # enough units for the wide ones: 43 row tiles x 4 column blocks
    ([2500, 31, 0, 2900], 5500, 512, 1024),
    # an odd number of K blocks over many units
    ([2500, 31, 0, 1500, 1400], 5500, 640, 2048),
]


def _case(sizes, M, K, cols, seed):
    rng = np.random.default_rng(seed)
    x = normal_bf16((M, K), 1.0, rng, outlier_p=0.01)
    w = normal_bf16((len(sizes), K, cols), 1.0 / np.sqrt(K), rng)
    xq, xs = gmm.mx4_quantize_lhs(to_dev_bf16(x))
    wq, ws = gmm.mx4_quantize_rhs(to_dev_bf16(w))
    x64 = R.mx4_values(R.unpack4(xq.cpu().numpy()), R.mx4_lhs_scales(xs.cpu().numpy()))
    w64 = R.mx4_values(R.unpack4(wq.cpu().numpy()), R.mx4_rhs_scales(ws.cpu().numpy())).transpose(0, 2, 1)
    return (xq, xs, wq, ws, to_dev(np.array(sizes, np.int32))), x64, w64


@pytest.mark.parametrize("sizes,M,K,N", EDGE)
def test_product(sizes, M, K, N):
    args, x64, w64 = _case(sizes, M, K, N, M + K + N)
    out = Guarded((M, N), torch.bfloat16)
    work = gmm.Workspace(len(sizes), M)
    gmm.mx4_fwd(*args, out=out.t, workspace=work)
    torch.cuda.synchronize()
    assert work.status() == 0
    out.check("out")
    ref, mag = R.grouped(x64, w64, sizes)
    R.check(bf16_to_np64(out.t), ref, R.BF16 * np.abs(ref) + R.SUM * mag + R.TINY, "out")
    assert torch.all(out.t[sum(sizes):] == 0)


@pytest.mark.parametrize("sizes,M,K,N", EDGE)
def test_fused_product_and_its_quantised_output(sizes, M, K, N):
    args, x64, w64 = _case(sizes, M, K, 2 * N, M + K + 2 * N)
    h, hq, hs = (Guarded(s, d) for s, d in (((M, N), torch.bfloat16), ((M, N // 2), torch.uint8),
                                            ((N // 128, M, 4), torch.uint8)))
    work = gmm.Workspace(len(sizes), M)
    gmm.mx4_fwd_swiglu_quant(*args, workspace=work, out=(h.t, hq.t, hs.t))
    fused = gmm.mx4_fwd(*args, fuse=True)
    _, q_only, s_only = gmm.mx4_fwd_swiglu_quant(*args, with_h=False)
    torch.cuda.synchronize()
    assert work.status() == 0
    for t in (h, hq, hs):
        t.check("fused output")
    ref, err, _, _ = R.swiglu_fwd(x64, w64, sizes)
    R.check(bf16_to_np64(h.t), ref, err, "h")
    assert torch.all(h.t[sum(sizes):] == 0)
    assert torch.equal(fused.view(torch.int16), h.t.view(torch.int16))
    # exactly the quantisation of the kernel's own h
    rq, rs = gmm.mx4_quantize_lhs(h.t)
    assert torch.equal(hq.t, rq) and torch.equal(hs.t, rs)
    assert torch.equal(q_only, rq) and torch.equal(s_only, rs)


def test_each_scale_byte_and_code_counts():
    """One row against weights whose blocks carry distinct scales: every block's scale is
    applied to its own 32 products, for every column and row of a tile."""
    K, N, M = 512, 256, 128
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    x *= torch.exp2((torch.arange(M, device="cuda") % 7).float() - 3)[:, None].bfloat16()
    x[:, 32:64] *= 4
    k = torch.arange(K, device="cuda") // 32
    n = torch.arange(N, device="cuda")
    w = torch.exp2(((k[:, None] * 5 + n[None, :] * 3) % 11).float() - 5).bfloat16()[None].contiguous()
    args = (*gmm.mx4_quantize_lhs(x), *gmm.mx4_quantize_rhs(w))
    got = bf16_to_np64(gmm.mx4_fwd(*args, torch.tensor([M], dtype=torch.int32, device="cuda")))
    ref = bf16_to_np64(x) @ bf16_to_np64(w[0])  # powers of two: quantised without error
    R.check(got, ref, R.BF16 * np.abs(ref), "out")


def test_nan_blocks_reach_their_rows_only():
    sizes, M, K, N = [100, 60], 200, 256, 256
    rng = np.random.default_rng(8)
    x = to_dev_bf16(normal_bf16((M, K), 1.0, rng))
    x[3, 7] = float("inf")
    x[120, 200] = float("nan")
    x[160:] = float("nan")  # rows of no group
    wq, ws = gmm.mx4_quantize_rhs(to_dev_bf16(normal_bf16((2, K, N), 0.06, rng)))
    out = gmm.mx4_fwd(*gmm.mx4_quantize_lhs(x), wq, ws, to_dev(np.array(sizes, np.int32)))
    bad = torch.isnan(out.float()).any(1).cpu().numpy()
    assert np.array_equal(np.flatnonzero(bad), [3, 120])
    assert torch.isnan(out[3].float()).all() and torch.isnan(out[120].float()).all()
    assert torch.all(out[160:] == 0)


def test_other_stream_reused_metadata_and_repeat():
    sizes, M, K, N = [300, 1, 211], 600, 256, 256
    args, _, _ = _case(sizes, M, K, 2 * N, 4)
    work = gmm.Workspace(3, M)
    first = gmm.mx4_fwd_swiglu_quant(*args, workspace=work)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = gmm.mx4_fwd_swiglu_quant(*args[:4], None, workspace=work, stream=side)
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert work.status() == 0
    assert work.buf[16:24].view(torch.int32).tolist() == [0, 0]


def test_offsets_past_32_bits():
    """x and the output of more than 2^31 elements: rows on each side of element 2^31 and the last."""
    K, N = 128, 4096
    M = 2 ** 31 // N + 300
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    wq, ws = gmm.mx4_quantize_rhs(torch.randn((1, K, N), generator=g, device="cuda", dtype=torch.bfloat16) / 8)
    st = torch.tensor([M - 5], dtype=torch.int32, device="cuda")
    rows = torch.tensor([1, 2 ** 31 // N - 1, 2 ** 31 // N, M - 6], device="cuda")
    xq, xs = gmm.mx4_quantize_lhs(x)
    out = gmm.mx4_fwd(xq, xs, wq, ws, st)
    x64 = R.mx4_values(*R.mx4_quantize(x[rows].view(torch.int16).cpu().numpy().view(np.uint16)))
    w64 = R.mx4_values(R.unpack4(wq.cpu().numpy()), R.mx4_rhs_scales(ws.cpu().numpy())).transpose(0, 2, 1)
    ref, mag = R.grouped(x64, w64, [len(rows)])
    R.check(bf16_to_np64(out[rows]), ref, R.BF16 * np.abs(ref) + R.SUM * mag + R.TINY, "out")
    assert torch.all(out[M - 5:] == 0)
    # and the quantiser: a wide x
    wide = torch.randn((2 ** 31 // 8192 + 9, 8192), generator=g, device="cuda", dtype=torch.bfloat16)
    q, s = gmm.mx4_quantize_lhs(wide)
    for r in (0, 2 ** 31 // 8192, len(wide) - 1):
        codes, byte = R.mx4_quantize(wide[r:r + 1].view(torch.int16).cpu().numpy().view(np.uint16))
        assert np.array_equal(R.unpack4(q[r:r + 1].cpu().numpy()), codes)
        assert np.array_equal(s[:, r].reshape(1, -1).cpu().numpy(), byte)


def test_no_rows():
    wq, ws = gmm.mx4_quantize_rhs(torch.zeros((2, 128, 128), dtype=torch.bfloat16, device="cuda"))
    xq, xs = gmm.mx4_quantize_lhs(torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda"))
    out = gmm.mx4_fwd(xq, xs, wq, ws, torch.zeros(2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert out.shape == (0, 128)
