"""One MoE expert block, trained a few steps and then served in 4 bits.

Training keeps 8-bit checkpoints between the passes: the e4m3 codes of x and of
the gate | up values, half of what bf16 takes, and no h at all.
Serving quantises the trained weights to MXFP4 once and runs

    x -> MXFP4 -> gate/up -> silu(gate) * up in MXFP4 -> y

so no activation between the two projections leaves the 4-bit format.

    python examples/moe_block.py            # needs a GB300 and the built library
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_blockwise_quantized_gb300 as gmm  # noqa: E402


class ExpertBlock:
    """Weights of G experts: w [G, K, 2N] (gate | up) and w2 [G, N, K]; rows come sorted by expert."""

    def __init__(self, G, K, N, max_rows, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        # fp32 master weights; the kernels take bf16
        self.w = normal(G, K, 2 * N) / K ** 0.5
        self.w2 = normal(G, N, K) / N ** 0.5
        self.workspace = gmm.Workspace(G, max_rows, device)

    def step(self, x, sizes, target, lr):
        """One gradient step on mean((y - target)^2) / 2 over the rows; returns the loss."""
        ws, rows = self.workspace, x.shape[0]
        w, w2 = self.w.bfloat16(), self.w2.bfloat16()
        # forward: h, and gate | up in 8 bits; x's codes are the FP8 forward's operands
        xq, xs = gmm.quantize_lhs(x)
        h, kept = gmm.swiglu_fwd(x, w, sizes, keep="e4m3", workspace=ws)
        y = gmm.bf16_fwd(h, w2, None, workspace=ws)  # None: the same rows, the same metadata
        del h
        diff = y.float() - target.float()
        dy = (diff / rows).bfloat16()
        # backward: h again and the gradient of gate | up in one pass over dy
        dgu, h = gmm.swiglu_bwd(dy, w2, kept, None, workspace=ws)
        dw2 = gmm.tgmm(h, dy, None, dw=torch.empty_like(w2), workspace=ws)
        dw = gmm.tgmm_ckpt(xq, xs, dgu, None, dw=torch.empty_like(w), workspace=ws)
        dx = gmm.dgrad(dgu, w, None, workspace=ws)  # to the layers before
        self.w -= lr * dw.float()
        self.w2 -= lr * dw2.float()
        return 0.5 * diff.square().sum().item() / rows, dx

    def serve(self):
        """The block with MXFP4 weights, as a function of (x, sizes)."""
        wq, ws = gmm.mx4_quantize_rhs(self.w.bfloat16())
        w2q, w2s = gmm.mx4_quantize_rhs(self.w2.bfloat16())

        def forward(x, sizes):
            xq, xs = gmm.mx4_quantize_lhs(x)
            _, hq, hs = gmm.mx4_fwd_swiglu_quant(xq, xs, wq, ws, sizes, with_h=False, workspace=self.workspace)
            return gmm.mx4_fwd(hq, hs, w2q, w2s, None, workspace=self.workspace)

        return forward

    def reference(self, x, sizes):
        ws = self.workspace
        h, _ = gmm.swiglu_fwd(x, self.w.bfloat16(), sizes, workspace=ws)
        return gmm.bf16_fwd(h, self.w2.bfloat16(), None, workspace=ws)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.3)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.rows, a.dim), generator=g, device="cuda").bfloat16()
    # a routing with an expert that gets no rows
    odds = torch.arange(1, a.experts + 1, dtype=torch.float32, device="cuda")
    odds[a.experts // 2] = 0
    sizes = torch.bincount(torch.multinomial(odds, a.rows, replacement=True, generator=g), minlength=a.experts).int()
    teacher = ExpertBlock(a.experts, a.dim, a.hidden, a.rows, seed=2)
    target = teacher.reference(x, sizes)
    block = ExpertBlock(a.experts, a.dim, a.hidden, a.rows, seed=3)
    losses = []
    for i in range(a.steps):
        loss, _ = block.step(x, sizes, target, a.lr)
        losses.append(loss)
        print(f"step {i:3d}  loss {loss:.4f}")
    exact = block.reference(x, sizes).float()
    served = block.serve()(x, sizes)
    rel = ((served.float() - exact).norm() / exact.norm()).item()
    print(f"served in MXFP4: {rel:.3f} off the bf16 block")
    if block.workspace.status() != 0:
        raise SystemExit("a kernel reported an error")
    return losses, block, x, sizes, served


if __name__ == "__main__":
    main()
