"""Host-side checks of the feed-forward block's entry points (no GPU needed):
refusals, all made before any launch, and the plain implementation that the GPU
tests compare with, against values worked out by hand and by differences."""
import numpy as np
import pytest

from tests import ffn_ref as R

FAKE = 1 << 20  # an aligned non-null pointer value; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    from fp8_blockwise_quantized_gb300 import build as b
    b.build()
    import fp8_blockwise_quantized_gb300 as g
    return g.load()


def _call(fn, names, values, kw):
    a = dict(zip(names, values))
    a.update(kw)
    return fn(*[a[n] for n in names])


TAIL = ["work", "wbytes", "stream"]
SIZES = ["gs", "G", "M", "K", "N"]
TAIL_V, SIZES_V = [FAKE, 1 << 20, None], [FAKE, 4, 512, 256, 256]

FWD = (["x", "w"] + SIZES + ["h", "gu", "guq", "gus"] + TAIL, [FAKE, FAKE] + SIZES_V + [FAKE, FAKE, None, None] + TAIL_V)
BWD = (["dy", "w2", "gu", "guq", "gus"] + SIZES + ["dgu", "h"] + TAIL,
       [FAKE, FAKE, None, FAKE, FAKE] + SIZES_V + [FAKE, FAKE] + TAIL_V)
WGRAD = (["xq", "xs", "dy"] + SIZES + ["dw", "scratch", "sbytes"] + TAIL,
         [FAKE] * 3 + SIZES_V + [FAKE, FAKE, 1 << 30] + TAIL_V)
MX4 = (["xq", "xs", "wq", "ws"] + SIZES + ["fuse", "out"] + TAIL, [FAKE] * 4 + SIZES_V + [0, FAKE] + TAIL_V)
MX4Q = (["xq", "xs", "wq", "ws"] + SIZES + ["h", "hq", "hs"] + TAIL, [FAKE] * 4 + SIZES_V + [FAKE] * 3 + TAIL_V)

COMMON = [(dict(K=100), 2), (dict(N=0), 2), (dict(G=0), 2), (dict(G=5000), 2), (dict(M=-1), 2), (dict(M=1 << 31), 2),
          (dict(gs=FAKE + 4), 3), (dict(work=None), 8), (dict(wbytes=16), 8), (dict(work=FAKE + 8), 3)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(x=None), 1), (dict(w=None), 1), (dict(h=None), 1), (dict(gu=None), 1), (dict(x=FAKE + 2), 3),
    (dict(gu=None, guq=FAKE), 1), (dict(gu=None, gus=FAKE), 1), (dict(guq=FAKE, gus=FAKE), 4),
    (dict(gu=FAKE + 8), 3), (dict(gu=None, guq=FAKE + 1, gus=FAKE), 3)])
def test_swiglu_fwd_refusals(lib, kw, code):
    assert _call(lib.gmm_bf16_swiglu_fwd, *FWD, kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), 1), (dict(w2=None), 1), (dict(dgu=None), 1), (dict(guq=None), 1), (dict(gus=None), 1),
    (dict(guq=None, gus=None), 1), (dict(gu=FAKE), 4), (dict(h=FAKE + 2), 3), (dict(dgu=FAKE + 4), 3)])
def test_swiglu_bwd_refusals(lib, kw, code):
    assert _call(lib.gmm_bf16_swiglu_bwd, *BWD, kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(xq=None), 1), (dict(xs=None), 1), (dict(dy=None), 1), (dict(dw=None), 1), (dict(xq=FAKE + 8), 3),
    (dict(dw=FAKE + 2), 3), (dict(scratch=FAKE + 4), 3)])
def test_wgrad_refusals(lib, kw, code):
    assert _call(lib.tgmm_fp8_ckpt, *WGRAD, kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(xq=None), 1), (dict(xs=None), 1), (dict(wq=None), 1), (dict(ws=None), 1), (dict(out=None), 1),
    (dict(ws=FAKE + 8), 3), (dict(out=FAKE + 2), 3)])
def test_mx4_refusals(lib, kw, code):
    assert _call(lib.gmm_mx4_fwd, *MX4, kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(hq=None), 1), (dict(hs=None), 1), (dict(h=FAKE + 8), 3),
                                              (dict(hs=FAKE + 4), 3)])
def test_mx4_swiglu_quant_refusals(lib, kw, code):
    assert _call(lib.gmm_mx4_fwd_swiglu_quant, *MX4Q, kw) == code


def test_mx4_quantize_refusals(lib):
    q, r = lib.gmm_mx4_quantize_lhs, lib.gmm_mx4_quantize_rhs
    assert q(FAKE, 10, 100, FAKE, FAKE, None) == 2
    assert q(FAKE, -1, 128, FAKE, FAKE, None) == 2
    assert q(None, 10, 128, FAKE, FAKE, None) == 1
    assert q(FAKE, 10, 128, FAKE, FAKE + 4, None) == 3
    assert q(None, 0, 128, None, None, None) == 0  # empty: nothing to do
    assert r(FAKE, 0, 128, 128, FAKE, FAKE, None) == 2
    assert r(FAKE, 2, 128, 130, FAKE, FAKE, None) == 2
    assert r(FAKE, 2, 128, 128, None, FAKE, None) == 1
    assert r(FAKE, 2, 128, 128, FAKE + 8, FAKE, None) == 3


def test_unknown_keep_is_refused():
    import torch
    import fp8_blockwise_quantized_gb300 as g
    with pytest.raises(ValueError, match="keep"):
        g.swiglu_fwd(torch.zeros(1, 128), torch.zeros(1, 128, 256), None, keep="fp16")


def test_reference_quantiser_by_hand():
    bits = np.zeros((1, 32), np.uint16)
    vals = np.array([6.0, 5.0, -5.5, 0.25, 0.75, 1.25, -1.75, 3.5, 7.0], np.float32)
    bits[0, :9] = vals.view(np.uint32) >> 16
    codes, byte = R.mx4_quantize(bits)
    # largest value 7: exponent 129, so the scale is 2^(127 - 127) = 1
    assert byte[0, 0] == 127
    want = [7, 6, 15, 0, 2, 2, 12, 6, 7]
    assert list(codes[0, :9]) == want and not codes[0, 9:].any()
    bits[0, 0] = 0x7f80  # infinity
    assert R.mx4_quantize(bits)[1][0, 0] == 255
    assert R.mx4_quantize(np.zeros((1, 32), np.uint16))[1][0, 0] == 0


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(0)
    M, K, N, sizes = 3, 5, 4, [2, 1]
    dy, w2, gu = rng.standard_normal((M, K)), rng.standard_normal((2, N, K)), rng.standard_normal((M, 2 * N))
    dgu, _, h, _ = R.swiglu_bwd(dy, w2, gu, sizes)
    group = [0, 0, 1]

    def loss(v):
        return sum(dy[m] @ ((R.silu(v[m, :N]) * v[m, N:]) @ w2[group[m]]) for m in range(M))

    for m in range(M):
        for j in range(2 * N):
            e = np.zeros_like(gu)
            e[m, j] = 1e-6
            assert abs((loss(gu + e) - loss(gu - e)) / 2e-6 - dgu[m, j]) < 1e-7 * (1 + abs(dgu[m, j]) * 100)
    assert np.allclose(h, R.silu(gu[:, :N]) * gu[:, N:])


def test_python_entry_points_refuse_what_kernels_cannot_take():
    """Tensors on the host, of another type, size or stride are refused before anything reads them."""
    import torch
    import fp8_blockwise_quantized_gb300 as g
    bf, u8 = torch.bfloat16, torch.uint8
    x, w, w2 = torch.zeros(4, 128, dtype=bf), torch.zeros(2, 128, 256, dtype=bf), torch.zeros(2, 128, 128, dtype=bf)
    xq, xs = torch.zeros(4, 128, dtype=u8), torch.zeros(1, 4)
    q4, s4 = torch.zeros(4, 64, dtype=u8), torch.zeros(1, 4, 4, dtype=u8)
    wq, ws = torch.zeros(2, 128, 64, dtype=u8), torch.zeros(2, 1, 1, 512, dtype=u8)
    for call in (lambda: g.swiglu_fwd(x, w, None), lambda: g.swiglu_bwd(x, w2, torch.zeros(4, 256, dtype=bf), None),
                 lambda: g.tgmm_ckpt(xq, xs, x, torch.zeros(2, dtype=torch.int32)), lambda: g.mx4_quantize_lhs(x),
                 lambda: g.mx4_quantize_rhs(w), lambda: g.mx4_fwd(q4, s4, wq, ws, None),
                 lambda: g.mx4_fwd_swiglu_quant(q4, s4, torch.zeros(2, 256, 64, dtype=u8),
                                                torch.zeros(2, 2, 1, 512, dtype=u8), None)):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            call()


def test_kept_values_of_another_form_are_refused():
    import torch
    from fp8_blockwise_quantized_gb300 import binding as b
    with pytest.raises(ValueError, match="kept"):
        b._need_kept(None, 4, 128)
    with pytest.raises(ValueError, match="kept"):
        b._need_kept(torch.zeros(4, 256, dtype=torch.bfloat16), 4, 128, "e4m3")
    with pytest.raises(ValueError, match="kept"):
        b._need_kept((torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)), 4, 128, "bf16")
