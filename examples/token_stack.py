"""A stack of residual feed-forward blocks over token embeddings, trained on the library's kernels.

    python examples/token_stack.py [--tokens 4096] [--vocabulary 8192] [--width 512]
                                   [--hidden 2048] [--blocks 2] [--steps 20]

    s = scale E[token]
    for each block:  h = norm(s);  s = s + drop((silu(h Wg^T) * (h Wu^T)) Wd^T)
    logits = norm(s) E^T

The branch of a block joins the residual stream inside the next block's layer_norm, which drops,
adds and normalises in one pass; its backward pass sends the gradient on along the stream and,
through the same dropout, into the branch.  No mask is stored: a step has an offset, each block a
seed.  The stream is fp32, everything that feeds a product bf16.  The table's gradient is the sum
of the output product's and the lookup's (embedding_backward with accumulate).  The stack learns to
name the token that a fixed permutation sends each token to.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_conv_tcgen05_gb300 as igc  # noqa: E402

BF16 = torch.bfloat16


class Stack:
    """The weights (bf16 copies of fp32 masters; the norms' fp32), and their fp32 gradients."""

    def __init__(self, vocabulary, width, hidden, blocks, gen, p=0.1, device="cuda"):
        shapes = {"E": (vocabulary, width)}
        for i in range(blocks):
            shapes.update({f"Wg{i}": (hidden, width), f"Wu{i}": (hidden, width),
                           f"Wd{i}": (width, hidden)})
        self.master = {n: torch.randn(s, generator=gen, device=device) * s[1] ** -0.5
                       for n, s in shapes.items()}
        for i in range(blocks + 1):
            self.master[f"w{i}"] = torch.ones(width, device=device)
            self.master[f"b{i}"] = torch.zeros(width, device=device)
        self.w = {n: t.to(BF16) if t.dim() == 2 else t for n, t in self.master.items()}
        self.grad = {n: torch.empty_like(t) for n, t in self.master.items()}
        self.blocks, self.p, self.scale = blocks, p, width ** 0.5

    def drop(self, i, offset, p):
        return dict(p=p, seed=1000 + i, offset=offset)

    def forward(self, tokens, offset=0, train=True):
        """The logits, and what the backward pass needs."""
        w, M, width = self.w, tokens.shape[0], self.w["E"].shape[1]
        p = self.p if train else 0.0

        def rows(dtype, n=width):
            return torch.empty((M, n), device=tokens.device, dtype=dtype)

        stream = igc.embedding_lookup(tokens, w["E"], scale=self.scale, Y=rows(torch.float32))
        branch, kept = None, []
        for i in range(self.blocks + 1):
            mean, rstd = (torch.empty(M, device=tokens.device) for _ in range(2))
            h = rows(BF16)
            if branch is None:
                igc.layer_norm(stream, w["w0"], w["b0"], Y=h, mean=mean, rstd=rstd)
            else:
                joined = rows(torch.float32)
                igc.layer_norm(branch, w[f"w{i}"], w[f"b{i}"], residual=stream, S=joined, Y=h,
                               mean=mean, rstd=rstd, **self.drop(i, offset, p))
                stream = joined
            kept.append((stream, mean, rstd, h))
            if i == self.blocks:
                break
            G, U = (rows(BF16, w[f"Wg{i}"].shape[0]) for _ in range(2))
            H = igc.gated_ffn(h, w[f"Wg{i}"], w[f"Wu{i}"], G=G, U=U)
            kept[-1] += (G, U, H)
            branch = igc.linear_act(H, w[f"Wd{i}"])
        logits = igc.linear_act(h, w["E"], Y=rows(torch.float32, w["E"].shape[0]))
        return logits, kept

    def backward(self, tokens, kept, dlogits, offset=0, train=True):
        """All gradients (into self.grad) from that of the logits (bf16)."""
        w, g = self.w, self.grad
        p = self.p if train else 0.0
        dh = torch.empty_like(kept[-1][3])
        igc.linear_act_backward(dlogits, kept[-1][3], w["E"], dX=dh, dW=g["E"])
        dstream = None
        for i in range(self.blocks, -1, -1):
            stream, mean, rstd = kept[i][:3]
            ds = torch.empty_like(stream) if dstream is None else dstream   # (in place)
            dbranch = torch.empty_like(dh) if i > 0 else None
            drop = self.drop(i, offset, p) if i > 0 else {}
            igc.layer_norm_backward(dh, stream, mean, rstd, w[f"w{i}"], dS_add=dstream, dS=ds,
                                    dX=dbranch, dw=g[f"w{i}"], db=g[f"b{i}"], **drop)
            dstream = ds
            if i == 0:
                break
            h, G, U, H = kept[i - 1][3:]
            dH, dh = torch.empty_like(H), torch.empty_like(h)
            igc.linear_act_backward(dbranch, H, w[f"Wd{i - 1}"], dX=dH, dW=g[f"Wd{i - 1}"])
            igc.gated_ffn_backward(dH, G, U, h, w[f"Wg{i - 1}"], w[f"Wu{i - 1}"], dX=dh,
                                   dWg=g[f"Wg{i - 1}"], dWu=g[f"Wu{i - 1}"])
        igc.embedding_backward(tokens, dstream, scale=self.scale, dW=g["E"], accumulate=True)

    def update(self, lr, max_norm):
        """Clips the global gradient norm and takes a step; returns the norm (on the device)."""
        norm = igc.grad_norm_clip(list(self.grad.values()), max_norm)
        for n, t in self.master.items():
            t.add_(self.grad[n], alpha=-lr)
            if t.dim() == 2:
                self.w[n].copy_(t)
        return norm


def train(tokens, vocabulary, width, hidden, blocks, steps, lr=0.5, max_norm=1.0, seed=1):
    """The losses of the steps, and the trained stack."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    stack = Stack(vocabulary, width, hidden, blocks, gen)
    target_of = torch.randperm(vocabulary, generator=gen, device="cuda")
    losses = []
    for step in range(steps):
        batch = torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda")
        logits, kept = stack.forward(batch, offset=step)
        target = target_of[batch][:, None]
        logp = torch.log_softmax(logits, 1)
        losses.append(-logp.gather(1, target).mean())
        dlogits = logp.exp_().scatter_add_(1, target, torch.full_like(target, -1, dtype=logp.dtype))
        stack.backward(batch, kept, dlogits.div_(tokens).to(BF16), offset=step)
        stack.update(lr, max_norm)
    return [float(v) for v in losses], stack


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("vocabulary", 8192), ("width", 512), ("hidden", 2048),
                        ("blocks", 2), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    losses, _ = train(a.tokens, a.vocabulary, a.width, a.hidden, a.blocks, a.steps)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    rc = igc.igc_check_device_status()
    if rc != igc.IGC_OK:
        raise igc.IGCError(rc, "token_stack")


if __name__ == "__main__":
    main()
