"""The wrappers around the experts on stand-ins (no GPU needed): operands of another GPU
than the call's are refused, and what a wrapper allocates belongs to the stream that it is
given, as its launch does (test_device_host, test_stream_host: why)."""
import contextlib

import pytest
import torch

T, k, E, K = 4, 2, 8, 128
BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
HERE, OTHER, CURRENT, SIDE = 0, 1, 11, 77


class Tensor:
    """What the wrappers look at, of a dense CUDA tensor."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.index, self.dense = dtype, torch.Size(shape), HERE, True

    device = property(lambda self: torch.device("cuda", self.index) if self.index >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.dense

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return ()

    def data_ptr(self):
        return 1 << 20


def ids():
    return Tensor(I32, T, k)


def w():
    return Tensor(F32, T, k)


def x(dtype=BF):
    return Tensor(dtype, T, K)


def col():
    return Tensor(F32, K)


# operator -> (positional arguments, keywords, outputs given: keyword and tensors)
CASES = {
    "route": lambda: ([Tensor(F32, T, E), k], dict(bias=Tensor(F32, E)), ("out", (ids(), w()))),
    "route_bwd": lambda: ([w(), Tensor(BF, T, E), ids()], {}, ("out", Tensor(BF, T, E))),
    "sort_rows": lambda: ([ids(), E], {}, ("out", (ids(), Tensor(I32, E)))),
    "gather_rows": lambda: ([x(), ids()], {}, ("out", Tensor(BF, T * k, K))),
    "gather_quantize": lambda: ([x(), ids()], {}, ("out", (Tensor(U8, T * k, K), Tensor(F32, K // 128, T * k)))),
    "gather_mx4_quantize": lambda: ([x(), ids()], {},
                                    ("out", (Tensor(U8, T * k, K // 2), Tensor(U8, K // 128, T * k, 4)))),
    "combine_rows": lambda: ([Tensor(BF, T * k, K), ids(), w()], {}, ("out", x())),
    "combine_rows_bwd": lambda: ([x(), Tensor(BF, T * k, K), ids(), w()], {}, ("out", (Tensor(BF, T * k, K), w()))),
    "norm_join": lambda: ([x(F32), x(), col(), col(), col()], {}, ("out", (x(F32), x()))),
    "norm_join full": lambda: ([x(), x(), col(), x(), col()], {}, ("out", (x(), x()))),
    "norm_join_bwd": lambda: ([x(F32), x(), x(F32), x(), col(), col(), col()], {}, ("into", (x(F32), x()))),
    "norm_join_bwd full": lambda: ([x(), x(), x(), x(), col(), x(), col()], {}, ("into", (x(), x()))),
    "clip_grads": lambda: ([[Tensor(BF, 5), Tensor(F32, 2, 3)], 1.0], {}, ("out", [Tensor(BF, 5), Tensor(F32, 6)])),
}


def _tensors(v):
    if isinstance(v, Tensor):
        return [v]
    if isinstance(v, dict):
        v = list(v.values())
    return [t for o in v for t in _tensors(o)] if isinstance(v, (list, tuple)) else []


class Stream:
    def __init__(self, handle=CURRENT, device=None):
        self.cuda_stream, self.device = handle, torch.device("cuda:0")


class Library:
    """Counts launches (with their streams) and says that every call went well."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 64

        def call(*a):
            self.log.append(("launch", a[-1]))
            return 0
        return call


@pytest.fixture
def machine(monkeypatch):
    """The binding over stand-ins; log: ("alloc" | "launch", stream) in order."""
    from fp8_blockwise_quantized_gb300 import build as b
    b.build()
    from fp8_blockwise_quantized_gb300 import binding as g
    log, now = [], [Stream()]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        try:
            yield
        finally:
            now.pop()

    def empty(shape, stride, dtype, device):
        log.append(("alloc", now[-1].cuda_stream))
        return Tensor(dtype, *shape)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(g, "_current_device", lambda: HERE)
    monkeypatch.setattr(g, "_empty", empty)
    monkeypatch.setattr(g, "_like", lambda t: empty(t.shape, None, t.dtype, t.device))
    monkeypatch.setattr(g, "_lib", Library(log))
    for name in ("data_ptr", "is_contiguous", "get_device"):
        monkeypatch.setattr(g, "_" + name, lambda t, _n=name: getattr(t, _n)())
    return g, log, now


def _call(g, name, args, kw, out=None, **more):
    kw = dict(kw, **more)
    if out is not None:
        kw[out[0]] = out[1]
    return getattr(g, name.split()[0])(*args, **kw)


@pytest.mark.parametrize("name", CASES)
def test_each_operand_of_another_device_or_layout_is_refused(machine, name):
    g, log, _ = machine
    args, kw, out = CASES[name]()
    _call(g, name, args, kw, out)
    assert [what for what, _ in log].count("launch") == 1  # as they are, they pass
    for t in _tensors(args) + _tensors(kw) + _tensors(out[1]):
        for change, back in ((dict(index=OTHER), dict(index=HERE)), (dict(dense=False), dict(dense=True)),
                             (dict(dtype=torch.float16), dict(dtype=t.dtype)), (dict(index=-1), dict(index=HERE))):
            log.clear()
            vars(t).update(change)
            with pytest.raises(ValueError):
                _call(g, name, args, kw, out)
            assert ("launch", CURRENT) not in log
            vars(t).update(back)
        if t.dim() == 2 and not (name == "clip_grads" or t in (args[0],)):
            vars(t).update(shape=torch.Size((t.shape[0] + 1, t.shape[1])))
            with pytest.raises(ValueError):
                _call(g, name, args, kw, out)
            vars(t).update(shape=torch.Size((t.shape[0] - 1, t.shape[1])))
    _call(g, name, args, kw, out)


@pytest.mark.parametrize("name", CASES)
def test_tensors_of_a_device_that_is_not_current_are_refused(machine, name):
    g, log, _ = machine
    args, kw, out = CASES[name]()
    for t in _tensors(args) + _tensors(kw) + _tensors(out[1]):
        t.index = OTHER
    with pytest.raises(ValueError, match="cuda:1"):
        _call(g, name, args, kw, out)
    assert not log


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_memory_and_launch_on_the_stream_given(machine, name, as_handle):
    g, log, now = machine
    args, kw, out = CASES[name]()
    _call(g, name, args, kw, out if name == "clip_grads" else None, stream=SIDE if as_handle else Stream(SIDE))
    assert [what for what, _ in log].count("launch") == 1 and [what for what, _ in log].count("alloc") >= 1
    assert {s for _, s in log} == {SIDE}, log
    assert len(now) == 1  # the caller's stream is current again


@pytest.mark.parametrize("name", CASES)
def test_the_current_stream_without_one(machine, name):
    g, log, _ = machine
    args, kw, _ = CASES[name]()
    _call(g, name, args, kw)
    assert {s for _, s in log} == {CURRENT}, log


def test_the_callers_stream_is_current_again_after_a_refusal(machine):
    g, log, now = machine
    with pytest.raises(ValueError):
        g.gather_rows(x(F32), ids(), stream=Stream(SIDE))
    assert len(now) == 1 and not log
