"""Measured cases of the MoE feed-forward operators: the gated feed-forward
block with its backward pass, the weight gradient from 8-bit activation
checkpoints, and the microscaled 4-bit (MXFP4) product.

With ``own = False`` a case runs in plain form: elementary torch operations in
32 bits, rounded once at the end.  With ``own = True`` it makes the calls a
user of this package makes.  Rows are sorted by expert: group g owns the next
``sizes[g]`` rows, the rows after the last group belong to none, and their
outputs are zero.

Operators (op):
  ffn_fwd   x [M,K], w [G,K,2N] (gate | up): h = silu(gate) * up, and the kept
            gate/up values, in bf16 (keep = "bf16") or as e4m3 codes with one
            scale per row and 128 columns, absmax / 448 (keep = "e4m3")
  ffn_bwd   dy [M,K], w2 [G,N,K], the kept values: the gradient of gate | up
            (dgu [M,2N]) and h, recomputed for the second weight's gradient
  wgrad     8-bit checkpoint of x (codes [M,K], scales [K/128,M]), dy [M,N]:
            dw[g] = x_g^T dy_g
  mx4       x [M,K] bf16 quantised to MXFP4 and multiplied with MXFP4 weights;
            fuse: w holds gate | up and the output is silu(gate) * up
  mx4_mlp   the 4-bit expert block: x -> gate/up -> h in MXFP4 -> y [M,K]
MXFP4: E2M1 codes, blocks of 32 along K with a power-of-two (E8M0) scale,
2^(floor(log2(absmax)) - 2).
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a handful of tokens through a small expert layer while a model is
        # being brought up: launch and latency
        dict(name="ffn_fwd tiny", op="ffn_fwd", keep="e4m3", G=4, M=512, tail=0, K=256, N=256, routing="even"),
        # one expert-parallel shard of a training step, activations kept whole
        dict(name="ffn_fwd dev bf16", op="ffn_fwd", keep="bf16", G=32, M=8192, tail=0, K=2048, N=512, routing="even"),
        # the production layer's training step, activations kept in 8 bits
        dict(name="ffn_fwd prod e4m3", op="ffn_fwd", keep="e4m3", G=256, M=65536, tail=0, K=2048, N=512,
             routing="zipf"),
        # its backward pass on one shard; rows past the last group are padding
        dict(name="ffn_bwd dev e4m3", op="ffn_bwd", keep="e4m3", G=32, M=8192, tail=37, K=2048, N=512,
             routing="zipf"),
        # the production layer's backward pass from whole activations
        dict(name="ffn_bwd prod bf16", op="ffn_bwd", keep="bf16", G=256, M=65536, tail=0, K=2048, N=512,
             routing="zipf"),
        # weight gradient of a narrow layer, ragged groups
        dict(name="wgrad odd", op="wgrad", G=24, M=5000, tail=11, K=1152, N=640, routing="zipf"),
        # weight gradient of the production gate/up layer
        dict(name="wgrad prod", op="wgrad", G=256, M=65536, tail=0, K=2048, N=1024, routing="zipf"),
        # serving, one token to eight experts: latency and weight reads
        dict(name="mx4 one token", op="mx4", fuse=True, G=32, M=8, tail=0, K=2048, N=512, routing="even"),
        # serving a mid-sized batch, second projection
        dict(name="mx4 dev wo", op="mx4", fuse=False, G=32, M=8192, tail=0, K=512, N=2048, routing="even"),
        # the production layer's gate/up projection as a prompt is read
        dict(name="mx4 prod wi", op="mx4", fuse=True, G=256, M=65536, tail=0, K=2048, N=512, routing="zipf"),
        # the whole expert block while 32 sequences are decoded
        dict(name="mx4_mlp decode", op="mx4_mlp", G=32, M=256, tail=0, K=2048, N=512, routing="zipf"),
        # the whole expert block at the production size
        dict(name="mx4_mlp prod", op="mx4_mlp", G=256, M=65536, tail=0, K=2048, N=512, routing="zipf"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("ffn_fwd", "ffn_bwd", "wgrad", "mx4", "mx4_mlp"))
        G, M = spread(1, 256), spread(1, 65536)
        K, N = 128 * spread(1, 32), 128 * spread(1, 16)
        # no more than the production layer: weights, products and row tiles
        if K * N > 2048 * 1024 or G * K * N > 256 * 2048 * 512 or M * K * N > 65536 * 2048 * 512:
            continue
        if M * (K + N) > 65536 * 2560 or 3072 in (M, K, N, 2 * N):
            continue
        case = dict(op=op, G=G, M=M, tail=rng.choice((0, 0, M // 9)), K=K, N=N, routing=rng.choice(("even", "zipf")))
        if op in ("ffn_fwd", "ffn_bwd"):
            case["keep"] = rng.choice(("bf16", "e4m3"))
        if op == "mx4":
            case["fuse"] = rng.choice((False, True))
        return case


# --------------------------------------------------------------------------- inputs

def _odds(case):
    """Odds of the experts: even, or Zipf(1.1) popularity with some experts never chosen."""
    G = case["G"]
    if case["routing"] == "even":
        return np.full(G, 1.0 / G)
    p = np.arange(1.0, G + 1.0) ** -1.1
    p[G - G // 32:] = 0.0
    return p / p.sum()


def _sizes(case, seed):
    """Rows of each expert."""
    rng = np.random.default_rng(seed)
    return rng.multinomial(case["M"] - case["tail"], rng.permutation(_odds(case))).astype(np.int32)


def _normal(gen, shape, std=1.0, outliers=False):
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * std
    if outliers:  # 1% of the activations are fifty times as large
        v = torch.where(torch.rand(shape, generator=gen, device="cuda", dtype=torch.bfloat16) < 0.01, v * 50, v)
    return v


def _e4m3(v):
    """v [M, C] -> e4m3 codes (bytes) [M, C], scales [C/128, M]."""
    b = v.float().view(v.shape[0], -1, 128)
    s = b.abs().amax(2) / 448.0
    inv = torch.where(s == 0, 0.0, 1.0 / s)
    q = (b * inv[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(v.shape).view(torch.uint8), s.t().contiguous()


def _mx4(v):
    """v [R, C] -> packed E2M1 codes [R, C/2] (even column in the low nibble), E8M0 scale bytes [R, C/32]."""
    b = v.float().view(v.shape[0], -1, 32)
    field = b.abs().amax(2).view(torch.int32) >> 23  # biased exponent of the block's largest value
    byte = torch.where(field == 255, 255, (field - 2).clamp(min=0))
    a = b * ((254 - byte.clamp(max=253)) << 23).view(torch.float32)[:, :, None]
    m = a.abs()
    # nearest, ties to the even code; 6 is the largest value
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code | ((a.view(torch.int32) < 0).to(torch.uint8) << 3)
    code = code.view(v.shape[0], -1, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), byte.to(torch.uint8)


def _pow2(byte):
    """E8M0 bytes -> the powers of two they stand for."""
    byte = byte.to(torch.int32)
    return torch.where(byte == 0, 1 << 22, byte << 23).view(torch.float32)


def _mx4_value(packed, scale):
    """codes [..., C/2] and scale bytes [..., C/32] -> fp32 values [..., C]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    v = torch.stack((lut[(packed & 15).int()], lut[(packed >> 4).int()]), -1)
    v = v.view(*packed.shape[:-1], -1, 32) * _pow2(scale)[..., None]
    return v.view(*packed.shape[:-1], -1)


def _mx4_weights(w):
    """w [G, K, N] -> codes [G, N, K/2] and scales [G, N/128, K/128, 512]: the byte of column n, block k/32 lies
    at (n % 32) * 16 + (n % 128 / 32) * 4 + k / 32 % 4 of its 512."""
    G, K, N = w.shape
    codes = torch.empty((G, N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((G, N // 128, K // 128, 32, 4, 4), dtype=torch.uint8, device=w.device)
    for g in range(0, G, 32):
        part = w[g:g + 32].transpose(1, 2).reshape(-1, K)
        q, s = _mx4(part)
        codes[g:g + 32] = q.view(-1, N, K // 2)
        scales[g:g + 32] = s.view(-1, N // 128, 4, 32, K // 128, 4).permute(0, 1, 4, 3, 2, 5)
    return codes, scales.view(G, N // 128, K // 128, 512)


def _mx4_weight_scales(s, K):
    """[G, N/128, K/128, 512] -> [G, N, K/32]."""
    G, NB, KB, _ = s.shape
    return s.view(G, NB, KB, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(G, NB * 128, KB * 4)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, G, M, K, N = (case[k] for k in ("op", "G", "M", "K", "N"))
    sizes = _sizes(case, seed)
    s = dict(case, sizes=torch.from_numpy(sizes).cuda())
    if own:  # the handle that a user keeps beside the layer: room for the groups' offsets and tiles
        import fp8_blockwise_quantized_gb300 as gmm
        s["workspace"] = gmm.Workspace(G, M)
    if op == "ffn_fwd":
        s["x"] = _normal(gen, (M, K), outliers=True)
        s["w"] = _normal(gen, (G, K, 2 * N), K ** -0.5)
    elif op == "ffn_bwd":
        s["dy"] = _normal(gen, (M, K))
        s["w2"] = _normal(gen, (G, N, K), N ** -0.5)
        gu = _normal(gen, (M, 2 * N), 1.5)
        s["kept"] = gu if case["keep"] == "bf16" else _e4m3(gu)
    elif op == "wgrad":
        s["xq"], s["xs"] = _e4m3(_normal(gen, (M, K), outliers=True))
        s["dy"] = _normal(gen, (M, N))
    else:
        s["x"] = _normal(gen, (M, K), outliers=True)
        fuse = op == "mx4_mlp" or case["fuse"]
        s["wq"], s["ws"] = _mx4_weights(_normal(gen, (G, K, 2 * N if fuse else N), K ** -0.5))
        if op == "mx4_mlp":
            s["w2q"], s["w2s"] = _mx4_weights(_normal(gen, (G, N, K), N ** -0.5))
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_blockwise_quantized_gb300 as gmm

    op, sizes, work = s["op"], s["sizes"], s["workspace"]
    if op == "ffn_fwd":
        h, kept = gmm.swiglu_fwd(s["x"], s["w"], sizes, keep=s["keep"], workspace=work)
        return _kept_out(h, kept)
    if op == "ffn_bwd":
        dgu, h = gmm.swiglu_bwd(s["dy"], s["w2"], s["kept"], sizes, workspace=work)
        return {"dgu": dgu, "h": h}
    if op == "wgrad":
        return {"dw": gmm.tgmm_ckpt(s["xq"], s["xs"], s["dy"], sizes, workspace=work)}
    xq, xs = gmm.mx4_quantize_lhs(s["x"])
    if op == "mx4":
        return {"out": gmm.mx4_fwd(xq, xs, s["wq"], s["ws"], sizes, fuse=s["fuse"], workspace=work)}
    _, hq, hs = gmm.mx4_fwd_swiglu_quant(xq, xs, s["wq"], s["ws"], sizes, with_h=False, workspace=work)
    # the same routing: the second projection reads the groups that the first has left in the workspace
    return {"y": gmm.mx4_fwd(hq, hs, s["w2q"], s["w2s"], None, workspace=work)}


def _kept_out(h, kept):
    if isinstance(kept, tuple):
        return {"h": h, "codes": kept[0].view(torch.float8_e4m3fn), "scales": kept[1]}
    return {"h": h, "gu": kept}


def _tiling(s):
    """Row tiles that lie in one group each: group [C], rows [C, T] (M where there is none)."""
    G, M, sizes = s["G"], s["M"], s["sizes"].long()
    T = 128 if M >= 64 * G else 16
    C = -(-M // T) + G
    tiles = (sizes + T - 1) // T
    ends = tiles.cumsum(0)
    t = torch.arange(C, device="cuda")
    g = torch.searchsorted(ends, t, right=True).clamp(max=G - 1)
    first = (sizes.cumsum(0) - sizes)[g] + (t - (ends - tiles)[g]) * T
    rows = first[:, None] + torch.arange(T, device="cuda")
    stop = sizes.cumsum(0)[g]
    live = (rows < stop[:, None]) & (t < ends[-1])[:, None]
    return g, torch.where(live, rows, M)


def _take(v, rows):
    """Rows of v in fp32, zeros where a tile has none."""
    live = (rows < v.shape[0])[..., None]
    return torch.where(live, v[rows.clamp(max=v.shape[0] - 1)].float(), 0.0)


def _put(tiles, rows, M):
    out = torch.zeros((M + 1, tiles.shape[-1]), device=tiles.device)
    out[rows.reshape(-1)] = tiles.reshape(-1, tiles.shape[-1])
    return out[:M]


def _grouped(x, w, s):
    """x [M, K] times w [G, K, N] by groups, in fp32; zeros in the rows of no group."""
    g, rows = _tiling(s)
    return _put(torch.bmm(_take(x, rows), w[g].float()), rows, s["M"])


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _run_plain(s):
    op, M, N, bf16 = s["op"], s["M"], s["N"], torch.bfloat16
    if op == "ffn_fwd":
        gu = _grouped(s["x"], s["w"], s)
        h = (_silu(gu[:, :N]) * gu[:, N:]).to(bf16)
        return _kept_out(h, gu.to(bf16) if s["keep"] == "bf16" else _e4m3(gu))
    if op == "ffn_bwd":
        dh = _grouped(s["dy"], s["w2"].transpose(1, 2), s)
        if s["keep"] == "bf16":
            gu = s["kept"].float()
        else:
            q, sc = s["kept"]
            gu = (q.view(torch.float8_e4m3fn).float().view(M, -1, 128) * sc.t()[:, :, None]).view(M, -1)
        gu = torch.where((torch.arange(M, device="cuda") < s["sizes"].sum())[:, None], gu, 0.0)
        gate, up = gu[:, :N], gu[:, N:]
        sig = 1.0 / (1.0 + torch.exp(-gate))
        dgate = dh * up * sig * (1.0 + gate * (1.0 - sig))
        return {"dgu": torch.cat((dgate, dh * gate * sig), 1).to(bf16), "h": (gate * sig * up).to(bf16)}
    if op == "wgrad":
        g, rows = _tiling(s)
        x = s["xq"].view(torch.float8_e4m3fn).float().view(M, -1, 128) * s["xs"].t()[:, :, None]
        part = torch.bmm(_take(x.view(M, -1), rows).transpose(1, 2), _take(s["dy"], rows))
        dw = torch.zeros((s["G"], s["K"], N), device="cuda")
        return {"dw": dw.index_add_(0, g, part).to(bf16)}
    x = _mx4_value(*_mx4(s["x"]))
    w = _mx4_value(s["wq"], _mx4_weight_scales(s["ws"], s["K"]))
    out = _grouped(x, w.transpose(1, 2), s)
    if op == "mx4_mlp" or s["fuse"]:
        out = _silu(out[:, :N]) * out[:, N:]
    if op == "mx4":
        return {"out": out.to(bf16)}
    h = _mx4_value(*_mx4(out.to(bf16)))
    w2 = _mx4_value(s["w2q"], _mx4_weight_scales(s["w2s"], N))
    return {"y": _grouped(h, w2.transpose(1, 2), s).to(bf16)}


# --------------------------------------------------------------------------- in 64 bits

def _by_group(case, seed, a, weight, cols):
    """a [M, *] times weight(g), one group after the other, in float64."""
    out = torch.zeros((a.shape[0], cols), dtype=torch.float64, device="cuda")
    at = 0
    for g, n in enumerate(_sizes(case, seed).tolist()):
        if n:
            out[at:at + n] = a[at:at + n].double() @ weight(g)
        at += n
    return out


def _four_bits(t):
    """Rows of t [M, C] as MXFP4 rounds them, in float64: each value to the nearest of the type's, ties to even."""
    t = t.double().reshape(t.shape[0], -1, 32)
    top = t.abs().amax(2, keepdim=True)
    e = (torch.frexp(torch.where(top > 0, top, 1.0))[1].long() - 3).clamp(min=-127)
    scale = ((e + 1023) << 52).view(torch.float64)  # 2^e
    u = t / scale
    step = torch.where(u.abs() < 2.0, 0.5, torch.where(u.abs() < 4.0, 1.0, 2.0))
    u = (torch.round(u / step) * step).clamp(-6.0, 6.0)
    return (u * scale).reshape(t.shape[0], -1)


def _weight64(codes, scales, g):
    """MXFP4 weight g [K, N] in float64."""
    c = codes[g].long()
    c = torch.stack((c % 16, c // 16), 2).reshape(c.shape[0], -1)
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[c % 8]
    N, K = c.shape
    n, b = torch.arange(N, device="cuda")[:, None], torch.arange(K // 32, device="cuda")[None, :]
    e = scales[g][n // 128, b // 4, (n % 32) * 16 + (n % 128 // 32) * 4 + b % 4].long()
    scale = ((e - 127 + 1023) << 52).view(torch.float64)
    return (torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(32, 1)).t()


def exact(case, seed):
    s = prepare(case, seed)
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    if op == "ffn_fwd":
        gu = _by_group(case, seed, s["x"], lambda g: s["w"][g].double(), 2 * N)
        h = gu[:, :N] * torch.sigmoid(gu[:, :N]) * gu[:, N:]
        if case["keep"] == "bf16":
            return {"h": h, "gu": gu}
        return {"h": h, "codes": None, "scales": gu.reshape(M, -1, 128).abs().amax(2).t().contiguous() / 448}
    if op == "ffn_bwd":
        dh = _by_group(case, seed, s["dy"], lambda g: s["w2"][g].double().t(), N)
        kept = s["kept"]
        if case["keep"] == "e4m3":
            kept = kept[0].view(torch.float8_e4m3fn).double() * kept[1].double().t().repeat_interleave(128, 1)
        kept = kept.double()
        kept[M - case["tail"]:] = 0
        gate, up, sig = kept[:, :N], kept[:, N:], torch.sigmoid(kept[:, :N])
        return {"dgu": torch.cat((dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig), 1), "h": gate * sig * up}
    if op == "wgrad":
        x = s["xq"].view(torch.float8_e4m3fn).double() * s["xs"].double().t().repeat_interleave(128, 1)
        dw = torch.zeros((case["G"], K, N), dtype=torch.float64, device="cuda")
        at = 0
        for g, n in enumerate(_sizes(case, seed).tolist()):
            dw[g] = x[at:at + n].t() @ s["dy"][at:at + n].double()
            at += n
        return {"dw": dw}
    fuse = op == "mx4_mlp" or case["fuse"]
    out = _by_group(case, seed, _four_bits(s["x"]), lambda g: _weight64(s["wq"], s["ws"], g), 2 * N if fuse else N)
    if fuse:
        out = out[:, :N] * torch.sigmoid(out[:, :N]) * out[:, N:]
    if op == "mx4":
        return {"out": out}
    h = _four_bits(out.bfloat16())
    return {"y": _by_group(case, seed, h, lambda g: _weight64(s["w2q"], s["w2s"], g), K)}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Inputs read once (the weights of the experts that are expected to have rows), outputs written once; two
    operations a product."""
    op, G, M, K, N = (case[k] for k in ("op", "G", "M", "K", "N"))
    S = M - case["tail"]
    live = float(np.sum(1.0 - (1.0 - _odds(case)) ** S))
    if op == "ffn_fwd":
        kept = 4 * N if case["keep"] == "bf16" else 2 * N + 8 * N / 128
        return {"bytes": 2 * S * K + 4 * live * K * N + M * (2 * N + kept), "flops": 4 * S * K * N}
    if op == "ffn_bwd":
        kept = 4 * N if case["keep"] == "bf16" else 2 * N + 8 * N / 128
        return {"bytes": S * (2 * K + kept) + 2 * live * K * N + 6 * M * N, "flops": 2 * S * K * N}
    if op == "wgrad":
        return {"bytes": S * (K + 4 * K / 128 + 2 * N) + 2 * G * K * N, "flops": 2 * S * K * N}
    cols = 2 * N if op == "mx4_mlp" or case["fuse"] else N
    bits4 = 0.5 + 1 / 32  # bytes a value in MXFP4
    total = {"bytes": 2 * S * K + live * K * cols * bits4 + 2 * M * N, "flops": 2 * S * K * cols}
    if op == "mx4_mlp":
        total["bytes"] += live * N * K * bits4 + 2 * M * K - 2 * M * N
        total["flops"] += 2 * S * K * N
    return total
