"""Plain 64-bit implementations (torch, any device) of what surrounds the experts:
router, sorted rows, norms with their residual stream, clipping; and the bounds the
tests compare with.

Bounds (relative to the sum of the magnitudes that a value is made of, unless said):
  - U = 2^-24, half a step of fp32; a chain of n fp32 additions is off by n U of the
    sum of its terms' magnitudes; exp, log1p, sqrt, divisions: a few U each, F32 =
    2^-20 covers sixteen of them;
  - one rounding to bf16 is half a step, 2^-8 of the value (BF16);
  - exp(l - m) is off by |l - m| U through the rounding of l - m, besides.
"""
import numpy as np
import torch

U = 2.0 ** -24
F32 = 2.0 ** -20
BF16 = 2.0 ** -8
INF = float("inf")


def places(ids, G):
    """rows (of ids' shape) and group sizes of a stable sort by expert (numpy)."""
    flat = np.asarray(ids).ravel().astype(np.int64)
    group = np.where((flat >= 0) & (flat < G), flat, G)
    order = np.argsort(group, kind="stable")
    rows = np.empty(flat.size, np.int64)
    rows[order] = np.arange(flat.size)
    rows = np.where(group < G, rows, -1 - rows)
    return rows.reshape(np.shape(ids)).astype(np.int32), np.bincount(group, minlength=G + 1)[:G].astype(np.int32)


def chosen(logits, bias, k):
    """ids of the k largest fp32 keys above -inf, ties to the lower id, else -1 (numpy)."""
    l = logits.float().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l).astype(np.float32)
    with np.errstate(invalid="ignore"):
        key = l if bias is None else l + bias.cpu().numpy()[None]
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(key, ids, 1) > -np.inf, ids, -1).astype(np.int32)


def route_weights(l, ids, score, renorm, scale):
    """Weights [T, k] in 64 bits of logits l (float64, may require grad) at ids."""
    l = torch.where(torch.isnan(l), -INF, l)
    at, live = ids.long().clamp(min=0), (ids >= 0) & (ids < l.shape[1])
    at = at.clamp(max=l.shape[1] - 1)
    lc = torch.where(live, l.gather(1, at), -INF)
    if score == "softmax":
        over = lc if renorm else l
        top = over.detach().amax(1, keepdim=True)
        top = torch.where(top > -INF, top, 0.0)
        w = torch.exp(lc - top) / torch.exp(over - top).sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.sigmoid(lc)
        if renorm:
            log_w = torch.where(live, torch.nn.functional.logsigmoid(torch.where(live, lc, 0.0)), -INF)
            top = log_w.detach().amax(1, keepdim=True)
            top = torch.where(top > -INF, top, 0.0)
            w = torch.exp(log_w - top)
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return scale * torch.where(live, w, 0.0)


def route_bwd(dw, l, ids, score, renorm, scale):
    """dlogits, and the sum of the magnitudes it is made of."""
    l = torch.where(torch.isnan(l), -INF, l).double()
    E = l.shape[1]
    live = (ids >= 0) & (ids < E)
    at = ids.long().clamp(0, E - 1)
    g = torch.where(live, scale * dw.double(), 0.0)
    lc = torch.where(live, l.gather(1, at), -INF)
    w = route_weights(l, ids, score, renorm, 1.0)
    if renorm:
        mean, mag = (g * w).sum(1, keepdim=True), (g * w).abs().sum(1, keepdim=True)
        slope = torch.sigmoid(-lc) if score == "sigmoid" else torch.ones_like(lc)
        d, m = w * (g - mean) * slope, w * (g.abs() + mag) * slope
    elif score == "sigmoid":
        d = g * torch.sigmoid(lc) * torch.sigmoid(-lc)
        m = d.abs()
    else:
        top = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(top > -INF, top, 0.0))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        mean, mag = (g * w).sum(1, keepdim=True), (g * w).abs().sum(1, keepdim=True)
        return (torch.zeros_like(l).scatter_add_(1, at, g * w) - p * mean,
                torch.zeros_like(l).scatter_add_(1, at, (g * w).abs()) + p * mag)
    d, m = torch.where(live, d, 0.0), torch.where(live, m, 0.0)
    return torch.zeros_like(l).scatter_add_(1, at, d), torch.zeros_like(l).scatter_add_(1, at, m)


def tokens_of(rows):
    """For each sorted row: its token and choice, and whether it belongs to a group (numpy)."""
    flat = np.asarray(rows).ravel().astype(np.int64)
    place = np.where(flat >= 0, flat, -1 - flat)
    entry = np.empty(flat.size, np.int64)
    entry[place] = np.arange(flat.size)
    live = np.zeros(flat.size, bool)
    live[place] = flat >= 0
    return entry // np.shape(rows)[1], entry % np.shape(rows)[1], live


def combine(y, rows, w):
    """out [T, K] in 64 bits and the sum of its terms' magnitudes."""
    rows = rows.long()
    live = rows >= 0
    w = torch.where(live, w.double(), 0.0) if w is not None else live.double()
    v = torch.where(live[:, :, None], y[rows.clamp(min=0)].double(), 0.0) * w[:, :, None]
    return v.sum(1), v.abs().sum(1)


def unit(v, eps):
    """v over the root of its mean square, and that root's reciprocal."""
    r = (v.square().mean(1, keepdim=True) + eps).rsqrt()
    return v * r, r


def norm_join(x, b, w_post, gate, w_next, alpha, beta, eps):
    """(out, n, |alpha x| + |beta gate z|) in the type of the arguments (64 bits)."""
    if b is None:
        out, mag = x, x.abs()
    else:
        z = b if w_post is None else unit(b, eps)[0] * w_post
        z = z if gate is None else z * gate
        out, mag = alpha * x + beta * z, (alpha * x).abs() + (beta * z).abs()
    n = None if w_next is None else unit(out, eps)[0] * w_next
    return out, n, mag


def norm_join_bwd(dout, dn, out, b, w_post, gate, w_next, alpha, beta, eps):
    """Gradients (dx, db, dw_post, dgate, dw_next) in 64 bits and a like tuple of magnitudes."""
    zero = torch.zeros_like(out)
    d = zero if dout is None else dout
    mag = d.abs()
    dw_next = m_next = None
    if w_next is not None:
        dw_next = m_next = zero.sum(0)
    if dn is not None:
        o, r = unit(out, eps)
        c = dn * w_next
        d = d + r * (c - o * (o * c).mean(1, keepdim=True))
        mag = mag + r * (c.abs() + o.abs() * (o * c).abs().mean(1, keepdim=True))
        dw_next, m_next = (dn * o).sum(0), (dn * o).abs().sum(0)
    if b is None:
        return (d, None, None, None, dw_next), (mag, None, None, None, m_next)
    u, um = beta * d, abs(beta) * mag
    bn, rb = unit(b, eps) if w_post is not None else (b, None)
    z = bn if w_post is None else bn * w_post
    g = torch.ones_like(out[:1]) if gate is None else gate
    dgate = mgate = None
    if gate is not None:
        dgate, mgate = u * z, um * z.abs()
        if gate.dim() == 1:
            dgate, mgate = dgate.sum(0), mgate.sum(0)
    dz, dzm = u * g, um * g.abs()
    if w_post is None:
        return (alpha * d, dz, None, dgate, dw_next), (abs(alpha) * mag, dzm, None, mgate, m_next)
    c, cm = dz * w_post, dzm * w_post.abs()
    db = rb * (c - bn * (bn * c).mean(1, keepdim=True))
    dbm = rb * (cm + bn.abs() * (bn.abs() * cm).mean(1, keepdim=True))
    return ((alpha * d, db, (dz * bn).sum(0), dgate, dw_next),
            (abs(alpha) * mag, dbm, (dzm * bn.abs()).sum(0), mgate, m_next))


def assert_within(got, want, allowed, what=""):
    """|got - want| <= allowed everywhere, and both finite; in 64 bits."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    bad = ~((got - want).abs() <= allowed + 1e-37)  # the smallest normal number of bf16 and fp32
    if bool(bad.any()):
        i = tuple(int(j) for j in bad.nonzero()[0])
        a = allowed if not isinstance(allowed, torch.Tensor) else allowed.expand_as(got)[i].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} out of tolerance; first at {i}: got "
                             f"{got[i].item()!r}, want {want[i].item()!r}, allowed {a!r}")
