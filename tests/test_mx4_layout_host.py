"""MXFP4 scales in another order than the kernels read are refused (no GPU needed).
The bytes of [M, K/32] are as many as those of [K/128, M, 4]: counted alone they
passed, and the product used each row's scales for other rows."""
import pytest

from tests.test_device_host import BF, F32, G, K, M, N, U8, Tensor, Work, binding, sizes  # noqa: F401

CODES, WCODES = (M, K // 2), (G, 2 * N, K // 2)


def _calls(g, xs, ws, out_hs):
    x, w = Tensor(U8, *CODES), Tensor(U8, *WCODES)
    xs, ws, out_hs = Tensor(U8, *xs), Tensor(U8, *ws), Tensor(U8, *out_hs)
    work = Work()
    return {"fwd": lambda: g.mx4_fwd(x, xs, w, ws, sizes(), out=Tensor(BF, M, 2 * N), workspace=work),
            "fused": lambda: g.mx4_fwd(x, xs, w, ws, sizes(), fuse=True, out=Tensor(BF, M, N), workspace=work),
            "quant": lambda: g.mx4_fwd_swiglu_quant(x, xs, w, ws, sizes(), workspace=work,
                                                    out=(None, Tensor(U8, M, N // 2), out_hs)),
            "quantize": lambda: g.mx4_quantize_lhs(Tensor(BF, M, K), out=(x, xs))}


XS, WS, HS = (K // 128, M, 4), (G, 2 * N // 128, K // 128, 512), (N // 128, M, 4)


@pytest.mark.parametrize("name,bad", [
    ("fwd", dict(xs=(M, K // 32))), ("fwd", dict(xs=(M, K // 128, 4))), ("fwd", dict(ws=(G, 2 * N, K // 32))),
    ("fused", dict(xs=(M, K // 32))), ("fused", dict(ws=(G, K // 128, 2 * N // 128, 512))),
    ("quant", dict(xs=(M, K // 32))), ("quant", dict(ws=(G, 2 * N, K // 32))), ("quant", dict(out_hs=(M, N // 32))),
    ("quantize", dict(xs=(M, K // 32)))])
def test_scales_of_another_order_are_refused(binding, name, bad):  # noqa: F811
    g, launched = binding
    kw = dict(xs=XS, ws=WS, out_hs=HS)
    kw.update(bad)
    with pytest.raises(ValueError, match="expected a contiguous CUDA tensor"):
        _calls(g, **kw)[name]()
    assert not launched


@pytest.mark.parametrize("name", ["fwd", "fused", "quant", "quantize"])
@pytest.mark.parametrize("flat", [False, True])
def test_scales_as_written_and_flat_pass(binding, name, flat):  # noqa: F811
    g, launched = binding

    def shape(s):
        n = 1
        for v in s:
            n *= v
        return (n,) if flat else s

    _calls(g, shape(XS), shape(WS), shape(HS))[name]()
    assert launched
