"""The wrappers' own memory belongs to the stream that they are given (no GPU
needed: torch's streams and allocations and the C entry points are stand-ins).

A wrapper that allocates on the current stream while its kernel runs on
another one hands that kernel memory which nothing orders before it: the zero
fill of a temporary workspace may run during or after the kernel, and the
memory may serve another tensor of the current stream while the kernel still
writes to it."""
import contextlib

import pytest
import torch

CURRENT, SIDE = 11, 77  # raw handles
G, M, K, N = 2, 4, 128, 128
BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


_zeros = torch.zeros  # the inputs are not the wrappers' allocations


def z(*shape, dtype=BF):
    return _zeros(shape, dtype=dtype)


SIZES = torch.tensor([3, 1], dtype=torch.int32)
CASES = {
    "quantize_lhs": lambda g, **k: g.quantize_lhs(z(M, K), **k),
    "quantize_rhs": lambda g, **k: g.quantize_rhs(z(G, K, N), **k),
    "quantize_rhs_w4": lambda g, **k: g.quantize_rhs_w4(z(G, K, N), **k),
    "fp8_fwd": lambda g, **k: g.fp8_fwd(z(M, K, dtype=U8), z(1, M, dtype=F32), z(G, N, K, dtype=U8),
                                        z(G, 1, 1, dtype=F32), SIZES, **k),
    "fp8_fwd_swiglu_quant": lambda g, **k: g.fp8_fwd_swiglu_quant(
        z(M, K, dtype=U8), z(1, M, dtype=F32), z(G, 2 * N, K, dtype=U8), z(G, 1, 2, dtype=F32), SIZES, **k),
    "fp8_w4_fwd": lambda g, **k: g.fp8_w4_fwd(z(M, K, dtype=U8), z(1, M, dtype=F32), z(G, N, K // 2, dtype=U8),
                                              z(G, 1, 1, dtype=F32), SIZES, **k),
    "fp8_w4_fwd_swiglu_quant": lambda g, **k: g.fp8_w4_fwd_swiglu_quant(
        z(M, K, dtype=U8), z(1, M, dtype=F32), z(G, 2 * N, K // 2, dtype=U8), z(G, 1, 2, dtype=F32), SIZES, **k),
    "bf16_fwd": lambda g, **k: g.bf16_fwd(z(M, K), z(G, K, N), SIZES, **k),
    "dgrad": lambda g, **k: g.dgrad(z(M, N), z(G, K, N), SIZES, **k),
    "tgmm": lambda g, **k: g.tgmm(z(M, K), z(M, N), SIZES, **k),
    "group_metadata": lambda g, **k: g.group_metadata(SIZES, M, **k),
    "swiglu_fwd": lambda g, **k: g.swiglu_fwd(z(M, K), z(G, K, 2 * N), SIZES, **k),
    "swiglu_fwd e4m3": lambda g, **k: g.swiglu_fwd(z(M, K), z(G, K, 2 * N), SIZES, keep="e4m3", **k),
    "swiglu_bwd": lambda g, **k: g.swiglu_bwd(z(M, K), z(G, N, K), z(M, 2 * N), SIZES, **k),
    "tgmm_ckpt": lambda g, **k: g.tgmm_ckpt(z(M, K, dtype=U8), z(1, M, dtype=F32), z(M, N), SIZES, **k),
    "mx4_quantize_lhs": lambda g, **k: g.mx4_quantize_lhs(z(M, K), **k),
    "mx4_quantize_rhs": lambda g, **k: g.mx4_quantize_rhs(z(G, K, N), **k),
    "mx4_fwd": lambda g, **k: g.mx4_fwd(z(M, K // 2, dtype=U8), z(1, M, 4, dtype=U8), z(G, N, K // 2, dtype=U8),
                                        z(G, 1, 1, 512, dtype=U8), SIZES, **k),
    "mx4_fwd_swiglu_quant": lambda g, **k: g.mx4_fwd_swiglu_quant(
        z(M, K // 2, dtype=U8), z(1, M, 4, dtype=U8), z(G, 2 * N, K // 2, dtype=U8), z(G, 2, 1, 512, dtype=U8), SIZES,
        **k),
}


class Stream:
    def __init__(self, handle=CURRENT, device=None):
        self.cuda_stream, self.device = handle, torch.device("cuda:0")


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

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[-1].cuda_stream, raising=False)

    def spy(real):
        def alloc(*a, **k):
            k.pop("device", None)
            log.append(("alloc", now[-1].cuda_stream))
            return real(*a, **k)
        return alloc

    for name in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, name, spy(getattr(torch, name)))
    monkeypatch.setattr(g, "_need", lambda *a, **k: None)
    monkeypatch.setattr(g, "_need_sizes", lambda *a: None)
    monkeypatch.setattr(g, "_here", lambda on: None)  # the tensors' device
    for name in g.EXPORTED:
        if name.startswith(("gmm_", "tgmm_")) and name not in ("gmm_workspace_bytes", "gmm_tiles_offset") and hasattr(g, name):
            def launch(*a, **k):
                stream = k.get("stream", a[-1])
                log.append(("launch", now[-1].cuda_stream if stream is None else g._s(stream)))
                return 0
            monkeypatch.setattr(g, name, launch)
    monkeypatch.setattr(g, "tgmm_fp8_ckpt_scratch_bytes", lambda *a: 64)
    return g, log, now


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_memory_and_launch_on_the_stream_given(machine, name, as_handle):
    g, log, now = machine
    call = CASES[name]
    call(g, stream=SIDE if as_handle else Stream(SIDE))
    assert [k for k, _ in log].count("launch") >= 1 and [k for k, _ in log].count("alloc") >= 1
    assert {s for _, s in log} == {SIDE}, log
    assert len(now) == 1  # the caller's stream is current again


@pytest.mark.parametrize("name", CASES)
def test_the_current_stream_without_one(machine, name):
    g, log, now = machine
    CASES[name](g)
    assert {s for _, s in log} == {CURRENT}, log


def test_the_callers_stream_is_current_again_after_a_refusal(machine, monkeypatch):
    g, log, now = machine
    monkeypatch.setattr(g, "gmm_bf16_swiglu_fwd", lambda *a: 2)
    with pytest.raises(g.GmmError):
        CASES["swiglu_fwd"](g, stream=Stream(SIDE))
    assert len(now) == 1


@pytest.mark.parametrize("handle", [0, 1])
@pytest.mark.parametrize("name", ["swiglu_fwd", "tgmm_ckpt", "mx4_fwd", "fp8_fwd", "quantize_lhs"])
def test_the_default_streams_handles(machine, monkeypatch, name, handle):
    """cudaStreamLegacy and 0 both name the default stream; torch has no external stream for
    them: it makes a new stream of 0 and refuses 1."""
    g, log, now = machine

    def external(h, device=None):
        assert h > 1, "torch would make a new stream" if h == 0 else "torch refuses this handle"
        return Stream(h)

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    CASES[name](g, stream=handle)
    assert {s for k, s in log if k == "alloc"} == {0} and {s for k, s in log if k == "launch"} <= {0, 1}, log
    assert len(now) == 1
