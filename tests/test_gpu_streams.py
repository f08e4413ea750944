"""Calls with `stream=` that is not the current stream, and without a workspace: the
wrappers' own memory (outputs, scratch, temporary workspace) is that stream's, whatever
the current stream allocates and writes meanwhile."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import normal_bf16
from tests.gpu_util import to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

SIZES, M, K, N = [300, 1, 0, 211], 600, 256, 256
G = len(SIZES)


@pytest.fixture(scope="module")
def data():
    rng = np.random.default_rng(21)
    d = {"st": to_dev(np.array(SIZES, np.int32)),
         "x": to_dev_bf16(normal_bf16((M, K), 1.0, rng)), "dy": to_dev_bf16(normal_bf16((M, N), 1.0, rng)),
         "w": to_dev_bf16(normal_bf16((G, K, N), 0.06, rng)), "wgu": to_dev_bf16(normal_bf16((G, K, 2 * N), 0.06, rng)),
         "w2": to_dev_bf16(normal_bf16((G, N, K), 0.06, rng)), "gu": to_dev_bf16(normal_bf16((M, 2 * N), 1.0, rng)),
         "one": to_dev(np.array([9000], np.int32)), "xl": to_dev_bf16(normal_bf16((9000, K), 1.0, rng)),
         "dl": to_dev_bf16(normal_bf16((9000, N), 1.0, rng))}
    d["q"], d["q4"], d["ql"] = gmm.quantize_lhs(d["x"]), gmm.mx4_quantize_lhs(d["x"]), gmm.quantize_lhs(d["xl"])
    d["wq"], d["wq4"], d["wgu4"] = (gmm.quantize_rhs(d["w"]), gmm.mx4_quantize_rhs(d["w"]),
                                    gmm.mx4_quantize_rhs(d["wgu"]))
    torch.cuda.synchronize()
    return d


CALLS = {
    "swiglu_fwd": lambda d, **k: gmm.swiglu_fwd(d["x"], d["wgu"], d["st"], **k),
    "swiglu_fwd e4m3": lambda d, **k: gmm.swiglu_fwd(d["x"], d["wgu"], d["st"], keep="e4m3", **k),
    "swiglu_bwd": lambda d, **k: gmm.swiglu_bwd(d["x"], d["w2"], d["gu"], d["st"], **k),
    "tgmm_ckpt": lambda d, **k: gmm.tgmm_ckpt(*d["q"], d["dy"], d["st"], **k),
    "tgmm_ckpt in parts": lambda d, **k: gmm.tgmm_ckpt(*d["ql"], d["dl"], d["one"], **k),
    "mx4_quantize_lhs": lambda d, **k: gmm.mx4_quantize_lhs(d["x"], **k),
    "mx4_fwd": lambda d, **k: gmm.mx4_fwd(*d["q4"], *d["wq4"], d["st"], **k),
    "mx4_fwd_swiglu_quant": lambda d, **k: gmm.mx4_fwd_swiglu_quant(*d["q4"], *d["wgu4"], d["st"], **k),
    "bf16_fwd": lambda d, **k: gmm.bf16_fwd(d["x"], d["w"], d["st"], **k),
    "fp8_fwd": lambda d, **k: gmm.fp8_fwd(*d["q"], *d["wq"], d["st"], **k),
    "tgmm": lambda d, **k: gmm.tgmm(d["x"], d["dy"], d["st"], **k),
    "dgrad": lambda d, **k: gmm.dgrad(d["dy"], d["w"], d["st"], **k),
}


def _flat(out):
    return [t for o in out for t in _flat(o)] if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_a_busy_stream_that_is_not_current(data, name, as_handle):
    want = [t.clone() for t in _flat(CALLS[name](data))]
    busy = torch.zeros((2, 8192, 8192), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):  # 6 ms: the call below is queued behind it
            torch.mm(busy[0], busy[0], out=busy[1])
    got = _flat(CALLS[name](data, stream=side.cuda_stream if as_handle else side))
    # what the current stream takes and writes now must not be the call's memory
    junk = [torch.full((1 << i,), 0xFF, dtype=torch.uint8, device="cuda") for i in range(9, 24) for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    for a, b in zip(want, got, strict=True):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(bool((j == 0xFF).all()) for j in junk)


@pytest.mark.parametrize("handle", [0, 1, 2])
@pytest.mark.parametrize("name", ["swiglu_fwd e4m3", "tgmm_ckpt in parts", "mx4_fwd", "fp8_fwd"])
def test_handles_of_the_default_streams(data, name, handle):
    """The legacy default stream (0 and 1) and the calling thread's (2), while another one is current."""
    want = [t.clone() for t in _flat(CALLS[name](data))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _flat(CALLS[name](data, stream=handle))
        junk = [torch.full((1 << i,), 0xFF, dtype=torch.uint8, device="cuda") for i in range(9, 24)]
    torch.cuda.synchronize()
    for a, b in zip(want, got, strict=True):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(bool((j == 0xFF).all()) for j in junk)
