"""The work counters in the workspace: left at zero by every launch of the operators that
claim their units, and put right by group_metadata when something overwrote them."""
import numpy as np
import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from fp8_blockwise_quantized_gb300.workloads import normal_bf16
from tests.gpu_util import to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def test_counters_after_every_operator_and_restored_by_group_metadata():
    rng = np.random.default_rng(2)
    sizes, M, K, N = [700, 0, 33, 5000], 5800, 128, 1024
    G = len(sizes)
    st = to_dev(np.array(sizes, np.int32))
    x, dn = to_dev_bf16(normal_bf16((M, K), 1.0, rng)), to_dev_bf16(normal_bf16((M, N), 1.0, rng))
    w, w2 = to_dev_bf16(normal_bf16((G, K, 2 * N), 0.08, rng)), to_dev_bf16(normal_bf16((G, N, K), 0.04, rng))
    q, q4, w4 = gmm.quantize_lhs(x), gmm.mx4_quantize_lhs(x), gmm.mx4_quantize_rhs(w)
    _, kept = gmm.swiglu_fwd(x, w, st)
    calls = [lambda k: gmm.swiglu_fwd(x, w, st, keep="e4m3", workspace=k)[1][0],
             lambda k: gmm.swiglu_bwd(x, w2, kept, st, workspace=k)[0],
             lambda k: gmm.tgmm_ckpt(*q, dn, st, workspace=k),
             lambda k: gmm.mx4_fwd(*q4, *w4, st, workspace=k),
             lambda k: gmm.mx4_fwd_swiglu_quant(*q4, *w4, st, workspace=k)[1]]
    for call in calls:
        work = gmm.Workspace(G, M)
        want = call(work)
        counters = work.buf[16:24].view(torch.int32)
        assert counters.tolist() == [0, 0]
        counters.copy_(torch.tensor([3, 1], dtype=torch.int32))
        gmm.group_metadata(st, M, workspace=work)
        assert counters.tolist() == [0, 0]
        got = call(work)
        assert torch.equal(want.view(torch.uint8), got.view(torch.uint8)) and work.status() == 0
        assert counters.tolist() == [0, 0]
