"""Measured cases of what surrounds the grouped products in an MoE layer: the
router, rows sorted by expert and joined again, the norms around the block, and
the clipping of the gradients by their global norm.

With ``own = False`` a case runs in plain form: elementary torch operations in
32 bits, rounded once at the end.  With ``own = True`` it makes the calls a
user of this package makes.

Operators (op; dir "fwd" or "bwd" where there is a gradient):
  route     logits [T,E] -> the k experts with the largest logit + bias (ties to
            the lower id) and their weights: softmax or sigmoid of the logit
            alone, over the chosen ones when renorm.  An expert at -inf is never
            chosen; where fewer than k are left, the id is -1 and the weight 0.
            bwd: gradient of the logits
  dispatch  ids [T,k] -> rows [T,k], the place of each choice among the rows
            sorted by expert (by token within one), group_sizes [E], and x's
            rows at their places, as bf16 or as e4m3 codes with a scale per 128
            columns, absmax / 448.  A choice outside 0..E-1 belongs to no group:
            its place r is behind them, rows holds -1 - r, and its row is zero
  combine   y [T k,K], rows, weights -> out[t] = sum over j of weights[t,j] *
            y[rows[t,j]], choices without a group left out.
            bwd: gradients of y and of the weights
  join      z = norm(b) * w_post; out = a x + c gate z; n = norm(out) * w_next,
            norm dividing by the root of the mean square.  gate: none, one value
            per column, or one per element.  bwd: gradients of all of them
  clip      gradients of many tensors scaled by min(1, max_norm / norm), norm
            the root of the sum of all squares
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


def listed():
    return [
        # 16 sequences decoded: the router of every layer at its smallest
        dict(name="route decode", op="route", dir="fwd", T=16, E=256, k=8, dtype="bf16", score="sigmoid", renorm=True,
             bias=True, pad=0),
        # a training step of the production layer (8192 tokens), the batch padded at its end
        dict(name="route prod", op="route", dir="fwd", T=8192, E=256, k=8, dtype="fp32", score="softmax", renorm=True,
             bias=True, pad=100),
        # its gradient, from the softmax over all experts
        dict(name="route bwd prod", op="route", dir="bwd", T=8192, E=256, k=8, dtype="fp32", score="softmax",
             renorm=False, bias=False, pad=0),
        # 32 sequences decoded in 8 bits: latency
        dict(name="dispatch decode e4m3", op="dispatch", T=32, E=32, k=8, K=2048, form="e4m3", routing="even", pad=0),
        # one expert-parallel shard, ragged: most choices fall on experts of other shards
        dict(name="dispatch shard e4m3", op="dispatch", T=4999, E=32, k=8, K=2048, form="e4m3", routing="even",
             pad=4321),
        # the production layer's training step
        dict(name="dispatch prod bf16", op="dispatch", T=8192, E=256, k=8, K=2048, form="bf16", routing="zipf", pad=0),
        # the way back after a prompt at the production size
        dict(name="combine prod", op="combine", dir="fwd", T=8192, E=256, k=8, K=2048, routing="zipf", pad=0),
        # its gradient on the development shape, padded
        dict(name="combine bwd dev", op="combine", dir="bwd", T=1024, E=32, k=8, K=2048, routing="even", pad=37),
        # between two blocks while 16 sequences are decoded
        dict(name="join decode", op="join", dir="fwd", T=16, K=2048, stream="bf16", gate="none", post=True),
        # and its gradient over a training step's tokens, with a learned gate per column and a 32-bit residual stream
        dict(name="join bwd prod", op="join", dir="bwd", T=8192, K=2048, stream="fp32", gate="column", post=True),
        # a small model's parameters, odd sizes and both types
        dict(name="clip small", op="clip", n=60, total=3000000, dtype="mixed", clipped=True),
        # the production layer's: gate | up and down weights of 256 experts, and a handful of vectors
        dict(name="clip prod", op="clip", n=9, total=805306368, dtype="bf16", clipped=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("route", "dispatch", "combine", "join", "clip"))
    if op == "clip":
        n = spread(1, 60)
        return dict(op=op, n=n, total=max(n, spread(1000, 300000000)), dtype=rng.choice(("bf16", "fp32", "mixed")),
                    clipped=rng.choice((True, True, False)))
    while True:
        T = spread(1, 16384)
        pad = rng.choice((0, 0, T // 7))
        if op == "join":
            K = 8 * spread(4, 1024)
            if T * K > 8192 * 2048:
                continue
            return dict(op=op, dir=rng.choice(("fwd", "bwd")), T=T, K=K, stream=rng.choice(("bf16", "fp32")),
                        gate=rng.choice(("none", "column", "full")), post=rng.choice((True, True, False)))
        E = spread(1, 512)
        k = min(E, rng.choice((1, 2, 4, 6, 8)))
        if op == "route":
            if T * E > 8192 * 256:
                continue
            return dict(op=op, dir=rng.choice(("fwd", "bwd")), T=T, E=E, k=k, dtype=rng.choice(("bf16", "fp32")),
                        score=rng.choice(("softmax", "sigmoid")), renorm=rng.choice((True, False)),
                        bias=rng.choice((True, False)), pad=pad)
        K = 128 * spread(1, 64)
        if T * k * K > 65536 * 2048:
            continue
        case = dict(op=op, T=T, E=E, k=k, K=K, routing=rng.choice(("even", "zipf")), pad=pad)
        if op == "dispatch":
            case["form"] = rng.choice(("bf16", "e4m3"))
        else:
            case["dir"] = rng.choice(("fwd", "bwd"))
        return case


# --------------------------------------------------------------------------- inputs

def _normal(gen, shape, std=1.0, dtype=torch.bfloat16, outliers=False):
    v = torch.randn(shape, generator=gen, device="cuda", dtype=dtype) * std
    if outliers:  # 1% of the activations are fifty times as large
        v = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, v * 50, v)
    return v


def _routing(case, gen):
    """ids [T, k]: k distinct experts a token, in proportion to an even or a Zipf(1.1) popularity; the last `pad` tokens
    have none."""
    T, E, k = case["T"], case["E"], case["k"]
    logp = torch.zeros(E, device="cuda")
    if case["routing"] == "zipf":
        logp = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        logp = logp[torch.randperm(E, generator=gen, device="cuda")]
    gumbel = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-9, 1 - 1e-6)))
    ids = torch.topk(logp + gumbel, k, dim=1).indices.int()
    ids[T - case["pad"]:] = -1
    return ids


def _places(ids, E):
    """rows [T, k] and group_sizes [E] of the choices."""
    flat = ids.reshape(-1).long()
    group = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(group, stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(group < E, rows, -1 - rows)
    sizes = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    sizes.index_add_(0, group, torch.ones_like(group, dtype=torch.int32))
    return rows.int().view(ids.shape), sizes[:E]


def _clip_counts(case):
    """Elements of each tensor: for a handful the production layer's two weights and vectors, else spread over a
    factor of a thousand."""
    n, total = case["n"], case["total"]
    if n == 9 and total == 805306368:
        return [256 * 2048 * 1024, 256 * 512 * 2048] + [2048] * 6 + [256 * 2048]
    share = np.exp(np.random.default_rng(n * 7919 + total).uniform(0, math.log(1000.0), n))
    return np.maximum(1, total * share / share.sum()).astype(np.int64).tolist()


def _clip_types(case):
    types = {"bf16": (torch.bfloat16,), "fp32": (torch.float32,), "mixed": (torch.bfloat16, torch.float32)}
    types = types[case["dtype"]]
    return [types[i % len(types)] for i in range(len(_clip_counts(case)))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], dict(case)
    bf16, f32 = torch.bfloat16, torch.float32
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal(gen, (T, E), 1.5, f32).to(bf16 if case["dtype"] == "bf16" else f32)
        s["logits"][T - case["pad"]:] = -math.inf  # padded tokens take no expert
        s["bias"] = _normal(gen, (E,), 0.1, f32) if case["bias"] else None
        if case["dir"] == "bwd":
            s["ids"] = _chosen(s)
            s["dweights"] = _normal(gen, (T, k), 1.0, f32)
    elif op == "dispatch":
        s["x"] = _normal(gen, (case["T"], case["K"]), outliers=True)
        s["ids"] = _routing(case, gen)
    elif op == "combine":
        T, k, K = case["T"], case["k"], case["K"]
        s["rows"], _ = _places(_routing(case, gen), case["E"])
        w = torch.rand((T, k), generator=gen, device="cuda") + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["y"] = _normal(gen, (T * k, K))
        if case["dir"] == "bwd":
            s["dout"] = _normal(gen, (T, K), 0.01)
    elif op == "join":
        T, K = case["T"], case["K"]
        stream = f32 if case["stream"] == "fp32" else bf16
        # a residual stream a few times larger than what a block adds
        s["x"] = _normal(gen, (T, K), 4.0, stream)
        s["b"] = _normal(gen, (T, K), 0.5, outliers=True)
        s["w_post"] = 1.0 + _normal(gen, (K,), 0.1, f32) if case["post"] else None
        s["w_next"] = 1.0 + _normal(gen, (K,), 0.1, f32)
        s["gate"] = {"none": None, "column": 0.5 + _normal(gen, (K,), 0.1, f32),
                     "full": torch.sigmoid(_normal(gen, (T, K), dtype=bf16))}[case["gate"]]
        s["scales"] = (0.9, 0.7)
        if case["dir"] == "bwd":
            s["dout"], s["dn"] = _normal(gen, (T, K), 0.01, stream), _normal(gen, (T, K), 0.01)
    else:
        s["grads"] = [_normal(gen, (c,), 0.02, t) for c, t in zip(_clip_counts(case), _clip_types(case))]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        # a norm near 0.02 * sqrt(elements); a good third of it allowed, or twice as much
        s["max_norm"] = 0.02 * math.sqrt(sum(_clip_counts(case))) * (0.37 if case["clipped"] else 2.0)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_blockwise_quantized_gb300 as gmm

    op = s["op"]
    if op == "route":
        how = dict(score=s["score"], renorm=s["renorm"])
        if s["dir"] == "bwd":
            return {"dlogits": gmm.route_bwd(s["dweights"], s["logits"], s["ids"], **how)}
        ids, weights = gmm.route(s["logits"], s["k"], bias=s["bias"], **how)
        return {"ids": ids, "weights": weights}
    if op == "dispatch":
        rows, sizes = gmm.sort_rows(s["ids"], s["E"])
        out = {"rows": rows, "sizes": sizes}
        if s["form"] == "bf16":
            out["x"] = gmm.gather_rows(s["x"], rows)
        else:
            q, out["scales"] = gmm.gather_quantize(s["x"], rows)
            out["codes"] = q.view(torch.float8_e4m3fn)
        return out
    if op == "combine":
        if s["dir"] == "bwd":
            dy, dweights = gmm.combine_rows_bwd(s["dout"], s["y"], s["rows"], s["weights"])
            return {"dy": dy, "dweights": dweights}
        return {"out": gmm.combine_rows(s["y"], s["rows"], s["weights"])}
    if op == "join":
        how = dict(w_post=s["w_post"], gate=s["gate"], w_next=s["w_next"], residual_scale=s["scales"][0],
                   block_scale=s["scales"][1], eps=EPS)
        if s["dir"] == "bwd":
            # x stands in for the forward's out: values of the same kind
            got = gmm.norm_join_bwd(s["dout"], s["dn"], s["x"], s["b"], **how)
            return dict(zip(("dx", "db", "dw_post", "dgate", "dw_next"), got))
        out, n = gmm.norm_join(s["x"], s["b"], **how)
        return {"out": out, "n": n}
    return {"norm": gmm.clip_grads(s["grads"], s["max_norm"], out=s["out"]), "grads": s["out"]}


def _rank_key(s):
    key = s["logits"].float()
    return key if s["bias"] is None else key + s["bias"]


def _chosen(s):
    """ids [T, k] of the largest keys, ties to the lower id; -1 where none is above -inf."""
    top, ids = torch.sort(_rank_key(s), dim=1, descending=True, stable=True)
    ids = torch.where(top > -math.inf, ids, -1)[:, :s["k"]]
    return ids.int().contiguous()


def _scores(l, s):
    """The experts' scores [T, E] in 32 bits; 0 at -inf."""
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.where(l > -math.inf, torch.exp(l - top), 0.0)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def _e4m3(v):
    """v [M, C] -> e4m3 codes [M, C], scales [M, C/128]."""
    b = v.float().view(v.shape[0], -1, 128)
    sc = b.abs().amax(2) / 448.0
    inv = torch.where(sc == 0, 0.0, 1.0 / sc)
    return (b * inv[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(v.shape), sc


def _places_of(rows):
    """The place of every choice, those without a group included."""
    rows = rows.reshape(-1).long()
    return torch.where(rows >= 0, rows, -1 - rows)


def _sent(v, rows):
    """Rows of v [T, C] at their places; zeros at the places of no group."""
    T, k = rows.shape
    out = torch.empty((T * k, v.shape[1]), dtype=v.dtype, device=v.device)
    out[_places_of(rows)] = torch.where((rows >= 0)[:, :, None], v[:, None, :], 0).view(T * k, -1)
    return out


def _norm_back(d, v, w, K):
    """Gradient of v * r * w, r = 1 / sqrt(mean(v^2) + EPS), with respect to v, and of w before its sum."""
    r = 1.0 / torch.sqrt((v * v).sum(1, keepdim=True) / K + EPS)
    c = d * w
    return r * c - v * (r * r * r / K) * (c * v).sum(1, keepdim=True), d * v * r


def _run_plain(s):
    op, bf16 = s["op"], torch.bfloat16
    if op == "route":
        l = s["logits"].float()
        if s["dir"] == "fwd":
            ids = _chosen(s)
            p = _scores(l, s).gather(1, ids.long().clamp(min=0))
            p = torch.where(ids >= 0, p, 0.0)
            if s["renorm"]:
                total = p.sum(1, keepdim=True)
                p = torch.where(total > 0, p / total, 0.0)
            return {"ids": ids, "weights": p}
        p, ids = _scores(l, s), s["ids"].long()
        live = ids >= 0
        at = ids.clamp(min=0)
        g = torch.where(live, s["dweights"], 0.0)
        if s["renorm"]:
            q = torch.where(live, p.gather(1, at), 0.0)
            total = q.sum(1, keepdim=True)
            q = torch.where(total > 0, q / total, 0.0)
            d = q * (g - (g * q).sum(1, keepdim=True))
            if s["score"] == "sigmoid":
                d = d * (1.0 - p.gather(1, at))
            dl = torch.zeros_like(l).scatter_add_(1, at, d)
        else:
            dense = torch.zeros_like(l).scatter_add_(1, at, g)
            dl = p * (1.0 - p) * dense if s["score"] == "sigmoid" else p * (dense - (dense * p).sum(1, keepdim=True))
        return {"dlogits": dl.to(s["logits"].dtype)}
    if op == "dispatch":
        rows, sizes = _places(s["ids"], s["E"])
        out = {"rows": rows, "sizes": sizes}
        if s["form"] == "bf16":
            out["x"] = _sent(s["x"], rows)
        else:
            q, sc = _e4m3(s["x"])
            out["codes"] = _sent(q.view(torch.uint8), rows).view(torch.float8_e4m3fn)
            out["scales"] = _sent(sc, rows).t().contiguous()
        return out
    if op == "combine":
        rows = s["rows"].long()
        live = rows >= 0
        w = torch.where(live, s["weights"], 0.0)
        y = torch.where(live[:, :, None], s["y"][rows.clamp(min=0)].float(), 0.0)
        if s["dir"] == "fwd":
            return {"out": (w[:, :, None] * y).sum(1).to(bf16)}
        d = s["dout"].float()[:, None, :]
        dy = torch.empty(s["y"].shape, dtype=bf16, device="cuda")
        dy[_places_of(rows)] = (w[:, :, None] * d).to(bf16).view(dy.shape)
        return {"dy": dy, "dweights": torch.where(live, (y * d).sum(2), 0.0)}
    if op == "join":
        a, c = s["scales"]
        x, b, K = s["x"].float(), s["b"].float(), s["K"]
        g = 1.0 if s["gate"] is None else s["gate"].float()
        if s["dir"] == "fwd":
            z = b
            if s["post"]:
                z = b * (1.0 / torch.sqrt((b * b).sum(1, keepdim=True) / K + EPS)) * s["w_post"]
            out = a * x + c * g * z
            n = out * (1.0 / torch.sqrt((out * out).sum(1, keepdim=True) / K + EPS)) * s["w_next"]
            return {"out": out.to(s["x"].dtype), "n": n.to(bf16)}
        d, dw_next = _norm_back(s["dn"].float(), x, s["w_next"], K)
        d = d + s["dout"].float()
        u = c * d
        z = b
        if s["post"]:
            z = b * (1.0 / torch.sqrt((b * b).sum(1, keepdim=True) / K + EPS)) * s["w_post"]
        got = {"dx": (a * d).to(s["x"].dtype), "db": u * g, "dw_post": None, "dgate": None, "dw_next": dw_next.sum(0)}
        if s["gate"] is not None:
            got["dgate"] = (u * z).sum(0) if s["gate"].dim() == 1 else (u * z).to(bf16)
        if s["post"]:
            got["db"], dw = _norm_back(u * g, b, s["w_post"], K)
            got["dw_post"] = dw.sum(0)
        got["db"] = got["db"].to(bf16)
        return got
    flat = torch.cat(s["grads"]).float()
    norm = (flat * flat).sum(dtype=torch.float64).sqrt()
    flat *= torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    if s["dtype"] == "bf16":
        flat = flat.to(bf16)
    parts = flat.split([g.numel() for g in s["grads"]])
    return {"norm": norm.float().view(1), "grads": [p.to(g.dtype) for p, g in zip(parts, s["grads"])]}


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = s["logits"].double()
        if case["dir"] == "fwd":
            ids = _chosen(s)
        else:
            ids = s["ids"]
        live = ids >= 0
        lc = torch.where(live, l.gather(1, ids.long().clamp(min=0)), -math.inf)
        if case["score"] == "softmax":
            over = lc if case["renorm"] else l
            log_p = lc - torch.logsumexp(over, 1, keepdim=True)
        else:
            log_p = torch.nn.functional.logsigmoid(lc)
            if case["renorm"]:
                log_p = log_p - torch.logsumexp(log_p, 1, keepdim=True)
        w = torch.nan_to_num(torch.exp(log_p), nan=0.0)
        if case["dir"] == "fwd":
            return {"ids": None, "weights": w}
        # by the Jacobian of log w, one row at a time: dL/dl = sum_j dw_j w_j dlog w_j/dl
        gw = torch.where(live, s["dweights"].double() * w, 0.0)
        total = gw.sum(1, keepdim=True)
        slope = torch.sigmoid(-lc) if case["score"] == "sigmoid" else torch.ones_like(lc)
        if case["score"] == "softmax" and not case["renorm"]:
            dl = -total * torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
            part = gw
        else:
            dl = torch.zeros_like(l)
            part = (gw - w * total if case["renorm"] else gw) * slope
        part = torch.where(live, part, 0.0)
        for j in range(case["k"]):
            at = ids[:, j:j + 1].long().clamp(min=0)
            dl.scatter_add_(1, at, part[:, j:j + 1])
        return {"dlogits": dl}
    if op == "dispatch":
        rows, _ = _places(s["ids"], case["E"])
        out = {"rows": None, "sizes": None}
        token = torch.zeros(rows.numel(), dtype=torch.long, device="cuda")
        flat = rows.reshape(-1).long()
        n = int((flat >= 0).sum())
        token[torch.where(flat >= 0, flat, -1 - flat)] = torch.arange(rows.numel(), device="cuda") // case["k"]
        x = s["x"].double()[token]
        x[n:] = 0
        if case["form"] == "bf16":
            return {**out, "x": x}
        return {**out, "codes": None, "scales": x.reshape(x.shape[0], -1, 128).abs().amax(2).t().contiguous() / 448}
    if op == "combine":
        rows, w = s["rows"].long(), s["weights"].double()
        out = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda") if case["dir"] == "bwd" else None
        for j in range(case["k"]):
            t = torch.nonzero(rows[:, j] >= 0)[:, 0]
            r = rows[t, j]
            y = s["y"][r].double()
            if dy is None:
                out[t] += w[t, j, None] * y
            else:
                d = s["dout"][t].double()
                dy[r] = w[t, j, None] * d
                dw[t, j] = torch.linalg.vecdot(y, d)
        return {"out": out} if dy is None else {"dy": dy, "dweights": dw}
    if op == "join":
        a, c = s["scales"]
        t64 = {k: None if s[k] is None else s[k].double() for k in ("x", "b", "w_post", "gate", "w_next")}
        one = torch.ones((), dtype=torch.float64, device="cuda")
        g = one if t64["gate"] is None else t64["gate"]

        def unit(v):  # v over the root of its mean square, and that root's reciprocal
            r = (v.square().mean(1, keepdim=True) + EPS).rsqrt()
            return v * r, r

        bn, rb = unit(t64["b"])
        z = bn * t64["w_post"] if case["post"] else t64["b"]
        if case["dir"] == "fwd":
            out = a * t64["x"] + c * (g * z)
            return {"out": out, "n": unit(out)[0] * t64["w_next"]}
        xn, rx = unit(t64["x"])
        dn = s["dn"].double()
        dxn = dn * t64["w_next"]
        d = s["dout"].double() + rx * (dxn - xn * (xn * dxn).mean(1, keepdim=True))
        dz = c * d * g
        got = {"dx": a * d, "db": dz, "dw_post": None, "dgate": None, "dw_next": (dn * xn).sum(0)}
        if case["gate"] != "none":
            got["dgate"] = c * d * z if case["gate"] == "full" else (c * d * z).sum(0)
        if case["post"]:
            dbn = dz * t64["w_post"]
            got["db"] = rb * (dbn - bn * (bn * dbn).mean(1, keepdim=True))
            got["dw_post"] = (dz * bn).sum(0)
        return got
    norm = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        norm += torch.linalg.vector_norm(g.double()) ** 2
    norm = norm.sqrt()
    factor = torch.clamp(s["max_norm"] / norm, max=1.0)
    return {"norm": norm.view(1), "grads": [g.double() * factor for g in s["grads"]]}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Inputs read once, outputs written once; a few operations for each value."""
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        elem = 2 if case["dtype"] == "bf16" else 4
        if case["dir"] == "fwd":
            return {"bytes": T * E * elem + 8 * T * k + 4 * E * case["bias"], "flops": 4 * T * E}
        return {"bytes": (2 if case["score"] == "softmax" and not case["renorm"] else 1) * T * E * elem + 8 * T * k,
                "flops": 4 * T * E}
    if op in ("dispatch", "combine"):
        T, k, K = case["T"], case["k"], case["K"]
        live = T - case["pad"]
        if op == "dispatch":
            held = 2.0 if case["form"] == "bf16" else 1 + 4 / 128
            return {"bytes": live * K * 2 + T * k * K * held + 8 * T * k + 4 * case["E"], "flops": 2 * T * K}
        if case["dir"] == "fwd":
            return {"bytes": live * k * K * 2 + T * K * 2 + 8 * T * k, "flops": 2 * live * k * K}
        return {"bytes": live * K * 2 + live * k * K * 2 + T * k * K * 2 + 12 * T * k, "flops": 3 * live * k * K}
    if op == "join":
        T, K = case["T"], case["K"]
        stream = 4 if case["stream"] == "fp32" else 2
        gate = T * K * 2 * (case["gate"] == "full")
        if case["dir"] == "fwd":
            return {"bytes": T * K * (2 * stream + 4) + gate, "flops": 10 * T * K}
        return {"bytes": T * K * (3 * stream + 6) + 2 * gate, "flops": 20 * T * K}
    held = sum(c * t.itemsize for c, t in zip(_clip_counts(case), _clip_types(case)))
    return {"bytes": 2 * held, "flops": 3 * sum(_clip_counts(case))}
