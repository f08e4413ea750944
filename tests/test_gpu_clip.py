"""Gradient clipping against 64 bits.  The norm: fp32 sums of a few hundred squares, then
doubles: F32 relative.  A scaled value: the factor's F32 and its type's rounding."""
import math

import pytest
import torch

import fp8_blockwise_quantized_gb300 as gmm
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _grads(counts, dtypes, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(c, generator=gen, device="cuda") * std).to(t) for c, t in zip(counts, dtypes)]


def _norm(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt().item() if grads else 0.0


def _check(grads, max_norm, in_place):
    before, norm = [g.clone() for g in grads], _norm(grads)
    out = None if in_place else [torch.full_like(g, math.nan) for g in grads]
    got = gmm.clip_grads(grads, max_norm, out=out)
    assert got.shape == (1,) and abs(got.item() - norm) <= R.F32 * norm
    by = min(1.0, max_norm / norm) if norm > 0 else 1.0
    for g, o, b in zip(grads, out or grads, before):
        want = b.double() * by
        half = R.U if b.dtype == F32 else R.BF16
        R.assert_within(o, want, (half + R.F32) * want.abs() if by < 1 else 0.0, "scaled")
        if not in_place:
            assert torch.equal(g, b)


LISTS = [[1], [7], [8, 1, 0, 4096, 4097], [0], [3, 100000, 5], [33000] * 70, list(range(1, 200)), [1] * 1500,
         [40000000, 3], [257] * 2003, [262144], [262143, 1], [262144, 1], [8191] * 32]


@pytest.mark.parametrize("counts", LISTS, ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(counts, kind, in_place):
    dtypes = {"bf16": [BF], "fp32": [F32], "mixed": [BF, F32, F32]}[kind]
    grads = _grads(counts, [dtypes[i % len(dtypes)] for i in range(len(counts))], len(counts))
    norm = max(_norm(grads), 1e-3)
    _check(grads, 0.31 * norm, in_place)
    _check(grads, 5.0 * norm, in_place)


def test_shapes_and_views_off_16_bytes():
    """Gradients that are views of one buffer start anywhere."""
    flat, out = _grads([100000], [BF])[0], torch.zeros(100003, dtype=BF, device="cuda")
    flat32 = _grads([50000], [F32])[0]
    grads = [flat[1:1001].view(10, 100), flat[1001:60002], flat[60002:60003], flat32[1:40002], flat32[40002:]]
    want, norm = [g.double() for g in grads], _norm(grads)
    got = gmm.clip_grads(grads[:3], 1.0, out=[out[2:1002].view(10, 100), out[1002:60003], out[60003:60004]])
    n3 = _norm(grads[:3])
    assert abs(got.item() - n3) <= R.F32 * n3
    R.assert_within(out[1002:60003], want[1] / n3, (R.BF16 + R.F32) * want[1].abs() / n3, "out")
    assert not bool(out[:2].any()) and not bool(out[60004:].any())
    edge = (flat[0].item(), flat32[0].item())
    got = gmm.clip_grads(grads, 1.0)
    assert abs(got.item() - norm) <= R.F32 * norm
    assert edge == (flat[0].item(), flat32[0].item())
    for g, w in zip(grads, want):
        half = R.U if g.dtype == F32 else R.BF16
        R.assert_within(g, w / norm, (half + R.F32) * w.abs() / norm, "in place")


@pytest.mark.parametrize("value", [3e38, 1e30, 1e-20, 1e-30, 2e-38])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_squares_beyond_the_range_of_32_bits(value, dtype):
    g = torch.full((9,), value, dtype=dtype, device="cuda")
    g[4:] *= 0.125
    z = torch.zeros(70000, dtype=dtype, device="cuda")  # zeros beside it
    want = _norm([g, z])
    got = gmm.clip_grads([z, g], math.inf).item()
    if want > torch.finfo(F32).max:
        assert got == math.inf
    else:
        assert abs(got - want) <= 2 * R.F32 * want
    assert not bool(z.any())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    grads = _grads([5000, 77], [BF, F32])
    grads[0][4321] = bad
    before = [g.clone() for g in grads]
    norm = gmm.clip_grads(grads, 1.0)
    assert not math.isfinite(norm.item())
    for g, b in zip(grads, before):
        assert torch.equal(g.view(torch.uint8), b.view(torch.uint8))
    out = [torch.zeros_like(g) for g in grads]
    gmm.clip_grads(grads, 1.0, out=out)
    for g, b in zip(out, before):
        assert torch.equal(g.view(torch.uint8), b.view(torch.uint8))


def test_zero_gradients_and_a_largest_norm_of_zero():
    grads = [torch.zeros(1000, device="cuda"), torch.zeros(0, dtype=BF, device="cuda")]
    assert gmm.clip_grads(grads, 0.0).item() == 0.0
    assert gmm.clip_grads([], 1.0).item() == 0.0
    g = torch.ones(100, device="cuda")
    assert gmm.clip_grads([g], 0.0).item() == 10.0
    assert not bool(g.any())


def test_the_norm_alone_leaves_the_gradients():
    grads = _grads([12345, 6], [BF, F32])
    before = [g.clone() for g in grads]
    n = gmm.clip_grads(grads, math.inf).item()
    assert abs(n - _norm(before)) <= R.F32 * n
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


def test_an_infinite_largest_norm_copies():
    grads = _grads([12345, 6], [BF, F32])
    out = [torch.zeros_like(g) for g in grads]
    gmm.clip_grads(grads, math.inf, out=out)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))


def test_runs_repeat_bit_for_bit():
    grads = _grads([3000000, 17, 400001], [BF, F32, F32])
    out = [torch.empty_like(g) for g in grads]
    first = gmm.clip_grads(grads, 0.5, out=out).item()
    kept = [o.clone() for o in out]
    for _ in range(3):
        assert gmm.clip_grads(grads, 0.5, out=out).item() == first
        assert all(torch.equal(a, b) for a, b in zip(out, kept))


def test_outputs_that_share_memory_are_refused_and_gradients_may():
    g = _grads([1000], [F32])[0]
    with pytest.raises(gmm.GmmError):
        gmm.clip_grads([g, g], 1.0)
    with pytest.raises(gmm.GmmError):
        gmm.clip_grads([g[:600], g[400:]], 1.0)
    out = [torch.empty_like(g), torch.empty_like(g)]
    norm = gmm.clip_grads([g, g], 1.0, out=out).item()  # read twice, written apart
    want = math.sqrt(2) * g.double().norm().item()
    assert abs(norm - want) <= R.F32 * want and torch.equal(out[0], out[1])
    mixed = [g.clone(), g.clone()]
    kept = torch.empty_like(g)
    gmm.clip_grads(mixed, 1.0, out=[mixed[0], kept])  # one in place, one not
    assert torch.equal(mixed[0], out[0]) and torch.equal(kept, out[1]) and torch.equal(mixed[1], g)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_negative_zeros_and_tiny_values_beside_others(dtype):
    """-0 is nothing; what vanishes beside the rest may, and what stands alone may not."""
    z = torch.zeros(300000, dtype=dtype, device="cuda").neg()
    tiny = torch.full((300000,), 1e-22, dtype=dtype, device="cuda")
    one = torch.ones(1, dtype=dtype, device="cuda")
    assert gmm.clip_grads([z], math.inf).item() == 0.0
    assert gmm.clip_grads([z, one, tiny], math.inf).item() == 1.0
    want = _norm([tiny])
    assert abs(gmm.clip_grads([z, tiny], math.inf).item() - want) <= R.F32 * want
