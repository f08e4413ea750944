"""The gated feed-forward block's forward and backward and the weight gradient
from 8-bit checkpoints against plain 64-bit implementations (ffn_ref): ragged,
empty and one-row groups, rows of no group, NaN and infinities in rows that a
group must not see, gradients against differences, other streams, reused
metadata and refusals."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32, normal_bf16
from tests import ffn_ref as R
from tests.gpu_util import Guarded, bf16_to_np64, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

# sizes, M, K (model dimension), N (expert dimension)
EDGE = [
    ([512], 512, 256, 256),
    ([1], 1, 128, 128),
    ([0, 300, 0, 212], 512, 384, 128),
    ([1, 127, 128, 129, 0, 2], 400, 256, 384),
    ([5, 0, 0, 9], 20, 128, 640),
    ([15, 16, 17, 33, 63, 64, 65], 300, 640, 256),
    ([0, 0, 0], 64, 256, 128),
    ([1000, 3, 700, 0, 0, 297], 2000, 1152, 512),
    # more units than SMs: rounds of wide ones and a rest cut in two (43 row tiles)
    ([2500, 31, 0, 2900], 5500, 128, 1024),
]


def _f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def _guard(shape, dtype):
    return Guarded(shape, dtype)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,M,K,N", EDGE)
def test_forward(sizes, M, K, N, keep):
    rng = np.random.default_rng(M + 3 * K + N)
    G, S = len(sizes), sum(sizes)
    x = normal_bf16((M, K), 1.0, rng, outlier_p=0.01)
    w = normal_bf16((G, K, 2 * N), 1.0 / np.sqrt(K), rng)
    h = _guard((M, N), torch.bfloat16)
    parts = [_guard((M, 2 * N), torch.bfloat16)] if keep == "bf16" else [
        _guard((M, 2 * N), torch.uint8), _guard((2 * N // 128, M), torch.float32)]
    kept = parts[0].t if keep == "bf16" else (parts[0].t, parts[1].t)
    work = gmm.Workspace(G, M)
    gmm.swiglu_fwd(to_dev_bf16(x), to_dev_bf16(w), to_dev(np.array(sizes, np.int32)), keep=keep, workspace=work,
                   out=(h.t, kept))
    torch.cuda.synchronize()
    assert work.status() == 0
    for p in [h] + parts:
        p.check("forward output")
    rh, rh_err, gu, err = R.swiglu_fwd(_f64(x), _f64(w), sizes)
    R.check(bf16_to_np64(h.t), rh, rh_err, "h")
    if keep == "bf16":
        R.check(bf16_to_np64(kept), gu, R.BF16 * np.abs(gu) + err + R.TINY, "gate | up")
        assert torch.all(kept[S:] == 0)
    else:
        codes, scales = kept[0].cpu().numpy(), kept[1].cpu().numpy().astype(np.float64)
        amax = np.abs(gu).reshape(M, -1, 128).max(2).T
        amax_err = err.reshape(M, -1, 128).max(2).T
        R.check(scales, amax / 448, amax / 448 * 2.0 ** -22 + amax_err / 448 + R.TINY, "scales")
        step = np.repeat(scales.T, 128, axis=1) * 2.0 ** -10
        R.check(R.dequant_e4m3(codes, scales), gu, 2.0 ** -4 * np.abs(gu) * 1.0001 + step + 2 * err + R.TINY, "codes")
        assert np.all(codes[S:] == 0) and np.all(scales[:, S:] == 0)
    assert torch.all(h.t[S:] == 0)


def _kept(rng, M, N, keep):
    """Device values of gate | up as the forward keeps them, and what they stand for in float64."""
    gu = to_dev_bf16(normal_bf16((M, 2 * N), 2.0, rng, outlier_p=0.01))
    if keep == "bf16":
        return gu, bf16_to_np64(gu)
    q, s = gmm.quantize_lhs(gu)
    return (q, s), R.dequant_e4m3(q.cpu().numpy(), s.cpu().numpy())


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,M,K,N", EDGE)
def test_backward(sizes, M, K, N, keep):
    rng = np.random.default_rng(M + K + 5 * N)
    G, S = len(sizes), sum(sizes)
    dy = normal_bf16((M, K), 1.0, rng)
    w2 = normal_bf16((G, N, K), 1.0 / np.sqrt(N), rng)
    kept, gu = _kept(rng, M, N, keep)
    dgu, h = _guard((M, 2 * N), torch.bfloat16), _guard((M, N), torch.bfloat16)
    work = gmm.Workspace(G, M)
    st = to_dev(np.array(sizes, np.int32))
    gmm.swiglu_bwd(to_dev_bf16(dy), to_dev_bf16(w2), kept, st, workspace=work, out=(dgu.t, h.t))
    torch.cuda.synchronize()
    assert work.status() == 0
    dgu.check("dgu")
    h.check("h")
    rd, rd_err, rh, rh_err = R.swiglu_bwd(_f64(dy), _f64(w2), gu, sizes)
    R.check(bf16_to_np64(dgu.t), rd, rd_err, "dgu")
    R.check(bf16_to_np64(h.t), rh, rh_err, "h")
    assert torch.all(dgu.t[S:] == 0) and torch.all(h.t[S:] == 0)
    only, none = gmm.swiglu_bwd(to_dev_bf16(dy), to_dev_bf16(w2), kept, st, with_h=False)
    assert none is None and torch.equal(only.view(torch.int16), dgu.t.view(torch.int16))


@pytest.mark.parametrize("sizes,M,K,N", EDGE)
def test_wgrad(sizes, M, K, N):
    rng = np.random.default_rng(7 * M + K + N)
    G = len(sizes)
    x = normal_bf16((M, K), 1.0, rng, outlier_p=0.01)
    dy = normal_bf16((M, N), 1.0, rng)
    xq, xs = gmm.quantize_lhs(to_dev_bf16(x))
    dw = _guard((G, K, N), torch.bfloat16)
    work = gmm.Workspace(G, M)
    gmm.tgmm_ckpt(xq, xs, to_dev_bf16(dy), to_dev(np.array(sizes, np.int32)), dw=dw.t, workspace=work)
    torch.cuda.synchronize()
    assert work.status() == 0
    dw.check("dw")
    ref, err = R.wgrad(xq.cpu().numpy(), xs.cpu().numpy(), _f64(dy), sizes)
    R.check(bf16_to_np64(dw.t), ref, err, "dw")


@pytest.mark.parametrize("sizes,M,K,N", [
    ([5000], 5000, 128, 128), ([4097], 4100, 256, 384), ([0, 9000, 70, 1], 9100, 384, 256), ([600, 2500], 3100, 512, 256)])
def test_wgrad_of_few_tiles_splits_the_rows(sizes, M, K, N):
    rng = np.random.default_rng(M + K + N)
    G = len(sizes)
    assert gmm.tgmm_fp8_ckpt_scratch_bytes(G, M, K, N) >= 2 * 4 * G * K * N
    xq, xs = gmm.quantize_lhs(to_dev_bf16(normal_bf16((M, K), 1.0, rng, outlier_p=0.01)))
    dy = normal_bf16((M, N), 1.0, rng)
    args = (xq, xs, to_dev_bf16(dy), to_dev(np.array(sizes, np.int32)))
    dw = _guard((G, K, N), torch.bfloat16)
    work = gmm.Workspace(G, M)
    gmm.tgmm_ckpt(*args, dw=dw.t, workspace=work)
    torch.cuda.synchronize()
    assert work.status() == 0
    dw.check("dw")
    ref, err = R.wgrad(xq.cpu().numpy(), xs.cpu().numpy(), _f64(dy), sizes)
    R.check(bf16_to_np64(dw.t), ref, err, "dw in parts")
    again = gmm.tgmm_ckpt(*args, workspace=work)
    assert torch.equal(again.view(torch.int16), dw.t.view(torch.int16))  # the parts are added in order
    # without scratch, each tile is one pair's work
    whole = torch.empty_like(dw.t)
    assert gmm.tgmm_fp8_ckpt(*args, G, M, K, N, whole, None, 0, work.buf, work.nbytes) == 0
    R.check(bf16_to_np64(whole), ref, err, "dw whole")
    short = torch.empty(64, dtype=torch.uint8, device="cuda")
    assert gmm.tgmm_fp8_ckpt(*args, G, M, K, N, whole, short, 64, work.buf, work.nbytes) == 8
    assert work.status() == 0


def test_gradients_against_differences():
    """The loss sum(dy * y), y = h W2, differentiated by central differences of
    the 64-bit forward in every coordinate of one row's gate | up values and
    in sampled coordinates of w; the bound adds the differences' own error."""
    rng = np.random.default_rng(5)
    sizes, M, K, N = [3, 0, 4], 8, 128, 128
    x = normal_bf16((M, K), 1.0, rng)
    w = normal_bf16((3, K, 2 * N), 1.0 / np.sqrt(K), rng)
    w2 = normal_bf16((3, N, K), 1.0 / np.sqrt(N), rng)
    dy = normal_bf16((M, K), 1.0, rng)
    st = to_dev(np.array(sizes, np.int32))
    _, gu = gmm.swiglu_fwd(to_dev_bf16(x), to_dev_bf16(w), st)
    dgu, _ = gmm.swiglu_bwd(to_dev_bf16(dy), to_dev_bf16(w2), gu, st)
    g64, w264, dy64 = bf16_to_np64(gu), _f64(w2), _f64(dy)
    group = np.repeat([0, 2], [3, 4])

    def loss(row, v):
        return dy64[row] @ ((R.silu(v[..., :N]) * v[..., N:]) @ w264[group[row]]).T

    eps = 1e-4
    got = bf16_to_np64(dgu)
    for row in (0, 2, 5):
        step = eps * np.eye(2 * N)
        diff = (loss(row, g64[row] + step) - loss(row, g64[row] - step)) / (2 * eps)
        _, err, _, _ = R.swiglu_bwd(dy64, w264, g64, sizes)
        R.check(got[row], diff, err[row] + 1e-6, f"dgu row {row}")
    # the weight gradient: d loss / d w[g, k, j] through gate | up
    xq, xs = gmm.quantize_lhs(to_dev_bf16(x))
    dw = bf16_to_np64(gmm.tgmm_ckpt(xq, xs, dgu, st))
    x64 = R.dequant_e4m3(xq.cpu().numpy(), xs.cpu().numpy())
    for g, rows in ((0, range(0, 3)), (2, range(3, 7))):
        for k, j in ((0, 0), (17, 200), (127, 255), (64, 31)):
            e = np.zeros(2 * N)
            e[j] = eps
            diff = sum((loss(r, g64[r] + x64[r, k] * e) - loss(r, g64[r] - x64[r, k] * e)) / (2 * eps) for r in rows)
            # dgu and the expanded x are bf16 (2^-9 each), summed over at most four rows
            mag = sum(abs(x64[r, k]) * abs(got[r, j]) for r in rows)
            assert abs(dw[g, k, j] - diff) <= R.BF16 * abs(diff) + 2 * R.BF16 * mag + 1e-6
    assert np.all(dw[1] == 0)


def test_rows_of_others_do_not_leak():
    """NaN and infinities in the rows of no group and in another group's rows
    reach neither a group's outputs nor its weight gradient."""
    rng = np.random.default_rng(11)
    sizes, M, K, N = [37, 50, 0, 41], 150, 256, 256
    G, S = len(sizes), sum(sizes)
    st = to_dev(np.array(sizes, np.int32))
    x, dy, dn = (to_dev_bf16(normal_bf16(s, 1.0, rng)) for s in ((M, K), (M, K), (M, N)))
    w, w2 = to_dev_bf16(normal_bf16((G, K, 2 * N), 0.05, rng)), to_dev_bf16(normal_bf16((G, N, K), 0.05, rng))
    gu = to_dev_bf16(normal_bf16((M, 2 * N), 1.0, rng))
    xq, xs = gmm.quantize_lhs(x)

    def outputs(x, dy, gu, xq, xs, dn):
        h, (q, s) = gmm.swiglu_fwd(x, w, st, keep="e4m3")
        d, h2 = gmm.swiglu_bwd(dy, w2, gu, st)
        return h, q, s.t().contiguous(), d, h2, gmm.tgmm_ckpt(xq, xs, dn, st)

    clean = outputs(x, dy, gu, xq, xs, dn)
    bad = [slice(37, 87), slice(S, M)]  # the second group, and the rows of none
    dirty = [t.clone() for t in (x, dy, gu, xq, xs, dn)]
    for r in bad:
        for t in (dirty[0], dirty[1], dirty[2], dirty[5]):
            t[r] = float("nan")
            t[r, ::3] = float("inf")
        dirty[3][r] = 0x7f  # NaN codes
        dirty[4][:, r] = float("inf")
    got = outputs(*dirty)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[37:87] = False
    for a, b in zip(clean[:5], got[:5]):
        assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))
        assert torch.all(b[S:].view(torch.uint8) == 0)
    for g in (0, 2, 3):
        assert torch.equal(clean[5][g].view(torch.int16), got[5][g].view(torch.int16))


def test_offsets_past_32_bits():
    """gate | up and dgu of more than 2^31 elements: the last rows, and a row on each side of
    element 2^31, against the 64-bit formulas."""
    K, N = 128, 1024
    M = 2 ** 31 // (2 * N) + 700  # 1,049,276 rows
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((1, K, 2 * N), generator=g, device="cuda", dtype=torch.bfloat16) / 16
    w2 = torch.randn((1, N, K), generator=g, device="cuda", dtype=torch.bfloat16) / 16
    st = torch.tensor([M - 3], dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 2 ** 31 // (2 * N) - 1, 2 ** 31 // (2 * N), M - 4], device="cuda")
    sub = [len(rows)]
    work = gmm.Workspace(1, M)
    h, gu = gmm.swiglu_fwd(x, w, st, workspace=work)
    rh, rh_err, rgu, err = R.swiglu_fwd(bf16_to_np64(x[rows]), bf16_to_np64(w), sub)
    R.check(bf16_to_np64(h[rows]), rh, rh_err, "h")
    R.check(bf16_to_np64(gu[rows]), rgu, R.BF16 * np.abs(rgu) + err + R.TINY, "gate | up")
    assert torch.all(gu[M - 3:] == 0)
    dgu, h2 = gmm.swiglu_bwd(x, w2, gu, st, workspace=work)
    rd, rd_err, rh, rh_err = R.swiglu_bwd(bf16_to_np64(x[rows]), bf16_to_np64(w2), bf16_to_np64(gu[rows]), sub)
    R.check(bf16_to_np64(dgu[rows]), rd, rd_err, "dgu")
    R.check(bf16_to_np64(h2[rows]), rh, rh_err, "h again")
    assert torch.all(dgu[M - 3:] == 0)
    assert work.status() == 0


def test_saturated_activation():
    """Gates far outside exp's range give the limits 0 and a, without NaN."""
    M, N, K = 4, 128, 128
    gu = torch.zeros((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    gu[0, :N], gu[1, :N], gu[2, :N], gu[3, :N] = -1000.0, 1000.0, -88.0, 3.0e38
    gu[:, N:] = 2.0
    gu[3, N:] = 1e-30
    dy = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    w2 = torch.full((1, N, K), 1.0 / K, dtype=torch.bfloat16, device="cuda")  # dh = 1
    dgu, h = gmm.swiglu_bwd(dy, w2, gu, torch.tensor([M], dtype=torch.int32, device="cuda"))
    d, h = bf16_to_np64(dgu), bf16_to_np64(h)
    assert np.all(d[0] == 0) and np.all(h[0] == 0)
    assert np.all(d[1, :N] == 2.0) and np.allclose(d[1, N:], 1000.0, rtol=R.BF16) and np.allclose(h[1], 2000.0, rtol=R.BF16)
    assert np.all(np.abs(d[2]) < 1e-30) and np.all(np.abs(h[2]) < 1e-30)
    assert np.all(np.isfinite(d[3])) and np.all(np.isfinite(h[3]))


def test_other_stream_reused_metadata_and_repeat():
    """On a stream of the caller's, with the metadata of an earlier call: the same bits, twice."""
    rng = np.random.default_rng(3)
    sizes, M, K, N = [300, 1, 211], 600, 256, 256
    st = to_dev(np.array(sizes, np.int32))
    x, w = to_dev_bf16(normal_bf16((M, K), 1.0, rng)), to_dev_bf16(normal_bf16((3, K, 2 * N), 0.06, rng))
    w2, dy = to_dev_bf16(normal_bf16((3, N, K), 0.06, rng)), to_dev_bf16(normal_bf16((M, K), 1.0, rng))
    work = gmm.Workspace(3, M)

    def step(sizes, stream):
        h, kept = gmm.swiglu_fwd(x, w, sizes, keep="e4m3", workspace=work, stream=stream)
        dgu, h2 = gmm.swiglu_bwd(dy, w2, kept, None, workspace=work, stream=stream)
        xq, xs = gmm.quantize_lhs(x, stream=stream)
        return (h, *kept, dgu, h2, gmm.tgmm_ckpt(xq, xs, dgu, None, workspace=work, stream=stream))

    first = step(st, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = step(st, side)
    side.synchronize()
    assert work.status() == 0
    for a, b in zip(first, second):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the counters are back at zero for the next launch
    assert work.buf[16:24].view(torch.int32).tolist() == [0, 0]


@pytest.mark.parametrize("G", [1, 9, 256, 257, 700])
def test_metadata_left_for_later_calls(G):
    """A call with group_sizes leaves the workspace as group_metadata does, whether it read the
    sizes in the kernel (up to 256 groups) or after a metadata pass, and its results agree with a
    later call that reuses the metadata."""
    rng = np.random.default_rng(G)
    K, N = 128, 128
    sizes = np.where(rng.random(G) < 0.3, 0, rng.integers(0, 7, G)).astype(np.int32)
    sizes[rng.integers(G)] = 300
    M = int(sizes.sum()) + 5
    x, w = to_dev_bf16(normal_bf16((M, K), 1.0, rng)), to_dev_bf16(normal_bf16((G, K, 2 * N), 0.08, rng))
    st = to_dev(sizes)
    want, got = gmm.Workspace(G, M), gmm.Workspace(G, M)
    gmm.group_metadata(st, M, workspace=want)
    h, gu = gmm.swiglu_fwd(x, w, st, workspace=got)
    torch.cuda.synchronize()
    assert got.header() == want.header() and got.offsets() == want.offsets() and got.order() == want.order()
    assert torch.equal(got.tiles(), want.tiles()) and torch.equal(got.pair_tiles(), want.pair_tiles())
    h2, gu2 = gmm.swiglu_fwd(x, w, None, workspace=got)
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    assert torch.equal(gu.view(torch.int16), gu2.view(torch.int16))
    ref, err, _, _ = R.swiglu_fwd(_f64(normal_bits(x)), _f64(normal_bits(w)), sizes)
    R.check(bf16_to_np64(h), ref, err, "h")
    mx = gmm.mx4_quantize_lhs(x) + gmm.mx4_quantize_rhs(w)
    a = gmm.mx4_fwd(*mx, st, fuse=True, workspace=want)
    b = gmm.mx4_fwd(*mx, None, fuse=True, workspace=got)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    xq, xs = gmm.quantize_lhs(x)
    fresh = gmm.Workspace(G, M)
    dw = gmm.tgmm_ckpt(xq, xs, gu, st, workspace=fresh)
    assert fresh.header() == want.header() and fresh.order() == want.order()
    dw2 = gmm.tgmm_ckpt(xq, xs, gu, None, workspace=got)
    assert torch.equal(dw.view(torch.int16), dw2.view(torch.int16))
    assert want.status() == got.status() == fresh.status() == 0


def normal_bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def test_invalid_sizes_are_reported():
    work = gmm.Workspace(2, 256)
    x = torch.zeros((256, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 128, 256), dtype=torch.bfloat16, device="cuda")
    gmm.swiglu_fwd(x, w, torch.tensor([200, 100], dtype=torch.int32, device="cuda"), workspace=work)
    assert work.status() == gmm.binding.GMM_ERR_GROUP_SIZES
    gmm.swiglu_bwd(x, w.transpose(1, 2).contiguous(), torch.zeros((256, 512), dtype=torch.bfloat16, device="cuda"),
                   torch.tensor([-5, 100], dtype=torch.int32, device="cuda"), workspace=work)
    assert work.status() == gmm.binding.GMM_ERR_GROUP_SIZES
    mx = gmm.mx4_quantize_lhs(x) + gmm.mx4_quantize_rhs(w)
    gmm.mx4_fwd(*mx, torch.tensor([255, 2], dtype=torch.int32, device="cuda"), workspace=work)
    assert work.status() == gmm.binding.GMM_ERR_GROUP_SIZES
    xq, xs = gmm.quantize_lhs(x)
    gmm.tgmm_ckpt(xq, xs, x, torch.tensor([-1, 100], dtype=torch.int32, device="cuda"), workspace=work)
    assert work.status() == gmm.binding.GMM_ERR_GROUP_SIZES
    assert work.status() == 0


def test_strides_types_and_sizes_are_refused():
    x = torch.zeros((64, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 256, 256), dtype=torch.bfloat16, device="cuda")
    st = torch.tensor([30, 20], dtype=torch.int32, device="cuda")
    bad = [lambda: gmm.swiglu_fwd(x.float(), w, st), lambda: gmm.swiglu_fwd(x.t().contiguous().t(), w, st),
           lambda: gmm.swiglu_fwd(x, w[:, :, ::2], st), lambda: gmm.swiglu_fwd(x, w, st.long()),
           lambda: gmm.swiglu_fwd(x, w, st[:1]), lambda: gmm.swiglu_fwd(x, w, st, out=(x[:32], x)),
           lambda: gmm.swiglu_bwd(x, w.transpose(1, 2), torch.zeros((64, 512), dtype=torch.bfloat16, device="cuda"), st),
           lambda: gmm.swiglu_bwd(x, w, torch.zeros((64, 510), dtype=torch.bfloat16, device="cuda"), st),
           lambda: gmm.tgmm_ckpt(x.view(torch.uint8)[:, ::2], torch.zeros((2, 64), device="cuda"), x, st),
           lambda: gmm.tgmm_ckpt(x.view(torch.uint8)[:, :256].contiguous(), torch.zeros((2, 63), device="cuda"), x, st),
           lambda: gmm.mx4_quantize_lhs(x[:, ::2]),
           lambda: gmm.mx4_fwd(*gmm.mx4_quantize_lhs(x), *[t[:1] for t in gmm.mx4_quantize_rhs(w)], st)]
    for call in bad:
        with pytest.raises(ValueError, match="expected a contiguous CUDA tensor"):
            call()


def test_no_rows():
    work = gmm.Workspace(2, 0)
    sizes = torch.zeros(2, dtype=torch.int32, device="cuda")
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, gu = gmm.swiglu_fwd(empty(0, 128), empty(2, 128, 256), sizes, workspace=work)
    dgu, h2 = gmm.swiglu_bwd(empty(0, 128), empty(2, 128, 128), gu, sizes, workspace=work)
    dw = torch.full((2, 128, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    gmm.tgmm_ckpt(torch.empty((0, 128), dtype=torch.uint8, device="cuda"),
                  torch.empty((1, 0), dtype=torch.float32, device="cuda"), dgu, sizes, dw=dw, workspace=work)
    torch.cuda.synchronize()
    assert work.status() == 0 and h.numel() == h2.numel() == 0 and torch.all(dw == 0)
