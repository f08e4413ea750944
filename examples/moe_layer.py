"""One whole MoE layer, trained and then served in 4 bits: norm, router, sorted rows, gated experts, joined rows,
and the norm, gate and residual stream around them, forward and backward, with the
gradients clipped by their global norm.

    n = norm(x) w_pre;  logits = n w_router^T;  b[t] = sum over the chosen experts of
    weight * expert(n[t]);  out = x + gate * norm(b) w_post;  the next block takes
    norm(out) w_next

    python examples/moe_layer.py            # needs a GB300 and the built library
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_blockwise_quantized_gb300 as gmm  # noqa: E402

EPS = 1e-6


class MoELayer:
    """E experts of width N on K columns, k of them a token.  Parameters are fp32; the
    grouped products take bf16 copies."""

    def __init__(self, E, K, N, k, tokens, device="cuda", seed=0, score="softmax"):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        one = lambda: 1.0 + 0.1 * normal(K)  # noqa: E731
        self.k, self.E, self.score = k, E, score
        self.params = {"w_pre": one(), "w_router": normal(E, K) / K ** 0.5, "w": normal(E, K, 2 * N) / K ** 0.5,
                       "w2": normal(E, N, K) / N ** 0.5, "w_post": one(), "gate": 0.3 * one(), "w_next": one()}
        self.bias = torch.zeros(E, device=device)  # moves the choice, not the weights
        self.workspace = gmm.Workspace(E, tokens * k, device)

    def forward(self, x, absent=None):
        """x bf16 [T, K]; absent: tokens (bool [T]) that take no expert, as padding.  Returns (out, n) and keeps
        what backward needs."""
        p, ws = self.params, self.workspace
        w, w2 = p["w"].bfloat16(), p["w2"].bfloat16()
        _, n = gmm.norm_join(x, w_next=p["w_pre"], eps=EPS)
        logits = n.float() @ p["w_router"].t()
        if absent is not None:
            logits.masked_fill_(absent[:, None], float("-inf"))
        ids, weights = gmm.route(logits, self.k, bias=self.bias, score=self.score, renorm=True)
        rows, sizes = gmm.sort_rows(ids, self.E)
        xs = gmm.gather_rows(n, rows)
        h, kept = gmm.swiglu_fwd(xs, w, sizes, workspace=ws)
        y = gmm.bf16_fwd(h, w2, None, workspace=ws)  # None: the same rows
        b = gmm.combine_rows(y, rows, weights)
        out, n_next = gmm.norm_join(x, b, p["w_post"], p["gate"], p["w_next"], eps=EPS)
        self.kept = x, n, logits, ids, weights, rows, xs, kept, y, b, out, w, w2
        return out, n_next

    def backward(self, dout, dn):
        """Gradients of out (bf16, or None) and of n -> (dx, {parameter: gradient})."""
        p, ws = self.params, self.workspace
        x, n, logits, ids, weights, rows, xs, kept, y, b, out, w, w2 = self.kept
        grads = {}
        dx, db, grads["w_post"], grads["gate"], grads["w_next"] = gmm.norm_join_bwd(
            dout, dn, out, b, p["w_post"], p["gate"], p["w_next"], eps=EPS)
        dy, dweights = gmm.combine_rows_bwd(db, y, rows, weights)
        dgu, h = gmm.swiglu_bwd(dy, w2, kept, None, workspace=ws)
        grads["w2"] = gmm.tgmm(h, dy, None, dw=torch.empty_like(w2), workspace=ws)
        grads["w"] = gmm.tgmm(xs, dgu, None, dw=torch.empty_like(w), workspace=ws)
        dlogits = gmm.route_bwd(dweights, logits, ids, score=self.score, renorm=True)
        grads["w_router"] = dlogits.t() @ n.float()
        dn_in = gmm.combine_rows(gmm.dgrad(dgu, w, None, workspace=ws), rows).float() + dlogits @ p["w_router"]
        dx, _, _, _, grads["w_pre"] = gmm.norm_join_bwd(dx, dn_in.bfloat16(), x, w_next=p["w_pre"], eps=EPS)
        return dx, grads

    def serve(self):
        """The layer with MXFP4 experts, as a function of x bf16 [T, K] that returns (out, n)."""
        p, ws = self.params, self.workspace
        wq, wqs = gmm.mx4_quantize_rhs(p["w"].bfloat16())
        w2q, w2qs = gmm.mx4_quantize_rhs(p["w2"].bfloat16())

        def forward(x):
            _, n = gmm.norm_join(x, w_next=p["w_pre"], eps=EPS)
            logits = n.float() @ p["w_router"].t()
            ids, weights = gmm.route(logits, self.k, bias=self.bias, score=self.score, renorm=True)
            rows, sizes = gmm.sort_rows(ids, self.E)
            xq, xs = gmm.gather_mx4_quantize(n, rows)
            _, hq, hs = gmm.mx4_fwd_swiglu_quant(xq, xs, wq, wqs, sizes, with_h=False, workspace=ws)
            y = gmm.mx4_fwd(hq, hs, w2q, w2qs, None, workspace=ws)
            return gmm.norm_join(x, gmm.combine_rows(y, rows, weights), p["w_post"], p["gate"], p["w_next"], eps=EPS)

        return forward

    def step(self, x, target, lr, max_norm=1.0):
        """One step on mean((n - target)^2) / 2; returns the loss and the gradients' norm before clipping."""
        _, n = self.forward(x)
        diff = n.float() - target.float()
        _, grads = self.backward(None, (diff / diff.numel()).bfloat16())
        norm = gmm.clip_grads(list(grads.values()), max_norm)
        for name, g in grads.items():
            self.params[name] -= lr * g.float()
        return 0.5 * diff.square().mean().item(), norm.item()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--choices", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=1.0)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.dim), generator=g, device="cuda").bfloat16()
    size = (a.experts, a.dim, a.hidden, a.choices, a.tokens)
    _, target = MoELayer(*size, seed=2).forward(x)
    layer = MoELayer(*size, seed=3)
    losses = []
    for i in range(a.steps):
        loss, norm = layer.step(x, target, a.lr)
        losses.append(loss)
        print(f"step {i:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")
    exact, (served, _) = layer.forward(x)[0].float(), layer.serve()(x)
    print(f"served in MXFP4: {((served.float() - exact).norm() / exact.norm()).item():.3f} off the bf16 layer")
    if layer.workspace.status() != 0:
        raise SystemExit("a kernel reported an error")
    return losses


if __name__ == "__main__":
    main()
