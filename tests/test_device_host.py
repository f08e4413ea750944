"""Operands of another GPU than the call's are refused on the host (no GPU
needed: the tensors are stand-ins).  A kernel launched on one device would read
the other device's addresses."""
import pytest
import torch

G, M, K, N = 2, 4, 128, 128
BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
HERE, OTHER = 0, 1


class Tensor:
    """What the checks look at, of a dense CUDA tensor."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), HERE

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return ()

    def data_ptr(self):
        return 1 << 20


class Work:
    G, M, nbytes = G, M, 1 << 20

    def __init__(self):
        self.buf = Tensor(U8, 1 << 20)

    def fits(self, G, M):
        return True


def sizes():
    return Tensor(I32, G)


# operator -> (positional arguments, out); `kept` pairs and outputs are tuples
CASES = {
    "swiglu_fwd e4m3": lambda: ([Tensor(BF, M, K), Tensor(BF, G, K, 2 * N), sizes()],
                                dict(keep="e4m3", out=(Tensor(BF, M, N), (Tensor(U8, M, 2 * N), Tensor(F32, 2, M))))),
    "swiglu_bwd": lambda: ([Tensor(BF, M, K), Tensor(BF, G, N, K), (Tensor(U8, M, 2 * N), Tensor(F32, 2, M)), sizes()],
                           dict(out=(Tensor(BF, M, 2 * N), Tensor(BF, M, N)))),
    "tgmm_ckpt": lambda: ([Tensor(U8, M, K), Tensor(F32, 1, M), Tensor(BF, M, N), sizes()],
                          dict(dw=Tensor(BF, G, K, N))),
    "mx4_quantize_lhs": lambda: ([Tensor(BF, M, K)], dict(out=(Tensor(U8, M, K // 2), Tensor(U8, 1, M, 4)))),
    "mx4_fwd": lambda: ([Tensor(U8, M, K // 2), Tensor(U8, 1, M, 4), Tensor(U8, G, N, K // 2),
                         Tensor(U8, G, 1, 1, 512), sizes()], dict(out=Tensor(BF, M, N))),
    "mx4_fwd_swiglu_quant": lambda: ([Tensor(U8, M, K // 2), Tensor(U8, 1, M, 4), Tensor(U8, G, 2 * N, K // 2),
                                      Tensor(U8, G, 2, 1, 512), sizes()],
                                     dict(out=(Tensor(BF, M, N), Tensor(U8, M, N // 2), Tensor(U8, 1, M, 4)))),
}


def _tensors(v):
    if isinstance(v, Tensor):
        return [v]
    if isinstance(v, dict):
        v = list(v.values())
    return [t for o in v for t in _tensors(o)] if isinstance(v, (list, tuple)) else []


@pytest.fixture
def binding(monkeypatch):
    from fp8_blockwise_quantized_gb300 import build as b
    b.build()
    from fp8_blockwise_quantized_gb300 import binding as g
    launched = []
    for name in g.EXPORTED:
        if hasattr(g, name) and name.startswith(("gmm_mx4", "gmm_bf16_swiglu", "tgmm_fp8_ckpt")):
            monkeypatch.setattr(g, name, lambda *a, _n=name, **k: launched.append(_n) or 0)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: HERE)
    return g, launched


def _call(g, name, args, kw):
    work = Work()
    if "quantize" not in name.replace("swiglu_quant", ""):
        kw = dict(kw, workspace=work)
    return lambda: getattr(g, name.split()[0])(*args, **kw), work


@pytest.mark.parametrize("name", CASES)
def test_each_operand_of_another_device_is_refused(binding, name):
    g, launched = binding
    args, kw = CASES[name]()
    call, work = _call(g, name, args, kw)
    call()
    assert launched  # as they are, they pass
    for t in _tensors(args) + _tensors(kw):
        launched.clear()
        t.index = OTHER
        with pytest.raises(ValueError, match="cuda:1"):
            call()
        assert not launched
        t.index = HERE


@pytest.mark.parametrize("name", [n for n in CASES if n != "mx4_quantize_lhs"])
def test_a_workspace_of_another_device_is_refused(binding, name):
    g, launched = binding
    call, work = _call(g, name, *CASES[name]())
    work.buf.index = OTHER
    with pytest.raises(ValueError, match="cuda:1"):
        call()
    assert not launched


@pytest.mark.parametrize("name", CASES)
def test_tensors_of_a_device_that_is_not_current_are_refused(binding, name):
    g, launched = binding
    args, kw = CASES[name]()
    call, work = _call(g, name, args, kw)
    for t in _tensors(args) + _tensors(kw) + [work.buf]:
        t.index = OTHER
    with pytest.raises(ValueError, match="cuda:1"):
        call()
    assert not launched


def test_quantised_weights_of_another_device_are_refused(binding):
    g, launched = binding
    w = Tensor(BF, G, K, N)
    w.index = OTHER
    with pytest.raises(ValueError, match="cuda:1"):
        g.mx4_quantize_rhs(w)
    assert not launched
