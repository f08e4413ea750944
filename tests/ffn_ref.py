"""Plain 64-bit implementations of the feed-forward block's operators for the
tests (numpy), and the bounds their results are compared with.

Bounds (derived here once, used by every test of these operators):
  - a product's fp32 sum is off by at most SUM * sum|terms|: the tensor core
    multiplies the 8- or 4-bit-mantissa inputs exactly and adds at most a few
    thousand of them in fp32 (2^-24 a step, errors of both signs); SUM = 2^-18
    leaves room for truncating adders;
  - one rounding to bf16 is 2^-9 relative; BF16 = 2^-8 covers it together with
    the hardware exponential and divide (a few 2^-22);
  - silu' and its factor lie within [-0.1, 1.1], so an error d of the gate's
    sum reaches h with at most 1.1 d |up|;
  - an e4m3 code is within 2^-4 of its value, or half of the smallest step
    (2^-10 scales) near zero.
"""
import numpy as np

from fp8_blockwise_quantized_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits

SUM = 2.0 ** -18
BF16 = 2.0 ** -8
TINY = 1e-30

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E2M1 = np.concatenate([E2M1, -E2M1])


def bf16_round(a):
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(a, np.float32))).astype(np.float64)


def e4m3_table():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


def dequant_e4m3(codes, scales):
    """codes [M, C] bytes, scales [C/128, M] -> float64 [M, C]."""
    return e4m3_table()[codes] * np.repeat(scales.astype(np.float64).T, 128, axis=1)


def offsets(sizes):
    return np.concatenate([[0], np.cumsum(np.asarray(sizes, np.int64))])


def grouped(x, w, sizes):
    """x [M, K], w [G, K, N] float64 -> (sums [M, N], sums of |terms|); rows of no group are zero."""
    out = np.zeros((x.shape[0], w.shape[2]))
    mag = np.zeros_like(out)
    off = offsets(sizes)
    for g in range(w.shape[0]):
        r = slice(off[g], off[g + 1])
        out[r] = x[r] @ w[g]
        mag[r] = np.abs(x[r]) @ np.abs(w[g])
    return out, mag


def logistic(a):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-a))


def silu(a):
    return a * logistic(a)


def swiglu_fwd(x, w, sizes):
    """-> h, its bound, gate | up sums, their bound."""
    n = w.shape[2] // 2
    gu, mag = grouped(x, w, sizes)
    err = SUM * mag
    a, b = gu[:, :n], gu[:, n:]
    h = silu(a) * b
    h_err = BF16 * np.abs(h) + 1.1 * err[:, :n] * np.abs(b) + (np.abs(silu(a)) + 1.1 * err[:, :n]) * err[:, n:] + TINY
    return h, h_err, gu, err


def swiglu_bwd(dy, w2, gu, sizes):
    """dy [M, K], w2 [G, N, K], gu [M, 2N] -> dgu, its bound, h, its bound."""
    n = w2.shape[1]
    dh, mag = grouped(dy, w2.transpose(0, 2, 1), sizes)
    rows = np.arange(dy.shape[0]) < int(np.sum(sizes))
    gu = np.where(rows[:, None], gu, 0.0)
    a, b = gu[:, :n], gu[:, n:]
    sg = logistic(a)
    fa, fb = b * sg * (1 + a * (1 - sg)), a * sg
    dgu = np.concatenate([dh * fa, dh * fb], 1)
    # 1 + a (1 - sg) and dh may cancel: absolute terms from each factor
    fa_err = 2.0 ** -20 * np.abs(b) * sg * (1 + np.abs(a))
    err = np.concatenate([SUM * mag * np.abs(fa) + np.abs(dh) * fa_err, SUM * mag * np.abs(fb)], 1)
    h = a * sg * b
    return dgu, BF16 * np.abs(dgu) + err + TINY, h, BF16 * np.abs(h) + TINY


def wgrad(xq, xs, dy, sizes):
    """codes, scales and dy -> dw [G, K, N] from the bf16 values that the codes expand to, and its bound."""
    x = bf16_round(e4m3_table()[xq].astype(np.float32) * np.repeat(xs.T, 128, axis=1))
    off = offsets(sizes)
    dw = np.zeros((len(sizes), x.shape[1], dy.shape[1]))
    mag = np.zeros_like(dw)
    for g in range(len(sizes)):
        r = slice(off[g], off[g + 1])
        dw[g] = x[r].T @ dy[r]
        mag[g] = np.abs(x[r]).T @ np.abs(dy[r])
    return dw, BF16 * np.abs(dw) + SUM * mag + TINY


def mx4_quantize(bits):
    """bf16 bits [..., C] -> codes [..., C] (one per element), scale bytes [..., C/32]."""
    u = bits.astype(np.int64).reshape(*bits.shape[:-1], -1, 32)
    e = ((u & 0x7fff) >> 7).max(-1)
    byte = np.where(e == 255, 255, np.maximum(e - 2, 0))
    v = bf16_bits_to_f32(bits).astype(np.float64).reshape(u.shape)
    with np.errstate(invalid="ignore"):
        t = np.abs(v) / 2.0 ** (byte[..., None] - 127.0)
        dist = np.abs(t[..., None] - E2M1[:8])
    # nearest value; of two equally near the one with the even code
    best = np.argmin(dist + np.array([0, 1, 0, 1, 0, 1, 0, 1]) * 1e-12, axis=-1)
    codes = best | np.where(np.signbit(v), 8, 0)
    return codes.reshape(bits.shape).astype(np.uint8), byte.astype(np.uint8)


def mx4_values(codes, byte):
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return E2M1[codes] * np.repeat(s, 32, axis=-1)


def unpack4(packed):
    """[..., C/2] bytes -> [..., C] codes, the low 4 bits first."""
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def mx4_lhs_scales(xs):
    """[K/128, M, 4] -> [M, K/32]."""
    return np.ascontiguousarray(xs.transpose(1, 0, 2)).reshape(xs.shape[1], -1)


def mx4_rhs_scales(ws):
    """[G, N/128, K/128, 512] -> [G, N, K/32]."""
    G, NB, KB, _ = ws.shape
    return ws.reshape(G, NB, KB, 32, 4, 4).transpose(0, 1, 4, 3, 2, 5).reshape(G, NB * 128, KB * 4)


def check(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} beyond the bound; first at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r} +- {bound[i]!r}")
