"""A residual gated feed-forward block on the library's kernels: training steps, then the
same weights answering token by token.

    python examples/feed_forward.py [--tokens 2048] [--width 1024] [--hidden 4096] [--steps 20]

    y = x + (silu(x Wg^T) * (x Wu^T)) Wd^T

A step is gated_ffn (both projections, activation and product in one kernel), linear_act with
the residual in its epilogue, the backward passes of both, grad_norm_clip over the three weight
gradients, and a gradient step.  The block learns to imitate another block with random weights.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_conv_tcgen05_gb300 as igc  # noqa: E402


class FeedForward:
    """The block's weights (bf16) with fp32 master copies, and the buffers of a step."""

    def __init__(self, width, hidden, gen, device="cuda"):
        shapes = {"Wg": (hidden, width), "Wu": (hidden, width), "Wd": (width, hidden)}
        self.master = {n: torch.randn(s, generator=gen, device=device) * s[1] ** -0.5
                       for n, s in shapes.items()}
        self.w = {n: t.bfloat16() for n, t in self.master.items()}
        self.grad = {n: torch.empty_like(t) for n, t in self.master.items()}   # fp32

    def forward(self, x, keep=False):
        """y, and what the backward pass needs: (H, G, U)."""
        hidden = self.w["Wg"].shape[0]
        G, U = ((torch.empty((x.shape[0], hidden), dtype=x.dtype, device=x.device)
                 for _ in range(2)) if keep else (None, None))
        H = igc.gated_ffn(x, self.w["Wg"], self.w["Wu"], act="silu", G=G, U=U)
        y = igc.linear_act(H, self.w["Wd"], residual=x)
        return y, (H, G, U)

    def backward(self, x, kept, dy):
        """The weights' gradients (into self.grad); returns that of x."""
        H, G, U = kept
        dH = torch.empty_like(H)
        igc.linear_act_backward(dy, H, self.w["Wd"], dX=dH, dW=self.grad["Wd"])
        dx = torch.empty_like(x)
        igc.gated_ffn_backward(dH, G, U, x, self.w["Wg"], self.w["Wu"], act="silu", dX=dx,
                               dWg=self.grad["Wg"], dWu=self.grad["Wu"])
        return dx.add_(dy)   # the residual path

    def update(self, lr, max_norm):
        """Clips the global gradient norm and takes a step; returns the norm (on the device)."""
        norm = igc.grad_norm_clip(list(self.grad.values()), max_norm)
        for n, t in self.master.items():
            t.add_(self.grad[n], alpha=-lr)
            self.w[n].copy_(t)
        return norm


def train(tokens, width, hidden, steps, lr=0.3, max_norm=1.0, seed=1):
    """The losses of the steps, and the trained block."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, block = (FeedForward(width, hidden, gen) for _ in range(2))
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
        target, _ = teacher.forward(x)
        y, kept = block.forward(x, keep=True)
        diff = y.float() - target.float()
        losses.append(diff.square().mean())
        block.backward(x, kept, (diff * (2.0 / width)).bfloat16())
        for g in block.grad.values():
            g.div_(tokens)
        block.update(lr * width, max_norm)
    return [float(v) for v in losses], block


def serve(block, prompt):
    """The block's answers for a prompt at once and token by token."""
    whole, _ = block.forward(prompt)
    steps = torch.cat([block.forward(prompt[i:i + 1])[0] for i in range(prompt.shape[0])])
    return whole, steps


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    losses, block = train(a.tokens, a.width, a.hidden, a.steps)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    prompt = torch.randn((8, a.width), device="cuda").bfloat16()
    whole, steps = serve(block, prompt)
    print("prompt and token-by-token answers differ by at most",
          float((whole.float() - steps.float()).abs().max()))
    rc = igc.igc_check_device_status()
    if rc != igc.IGC_OK:
        raise igc.IGCError(rc, "feed_forward")


if __name__ == "__main__":
    main()
