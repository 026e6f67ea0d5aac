"""The feed-forward block of examples/feed_forward.py: its gradients against a 64-bit autograd of
the same block, training that learns, and serving that agrees with the prompt pass."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from gpu_helpers import check_device_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "feed_forward_example", os.path.join(ROOT, "examples", "feed_forward.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,width,hidden", [(37, 200, 328), (400, 256, 640)])
def test_block_gradients(example, tokens, width, hidden):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    block = example.FeedForward(width, hidden, gen)
    x = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
    y, kept = block.forward(x, keep=True)
    dx = block.backward(x, kept, dy)
    check_device_ok()
    leaves = {n: w.double().requires_grad_() for n, w in block.w.items()}
    xd = x.double().requires_grad_()
    h = torch.nn.functional.silu(xd @ leaves["Wg"].t()) * (xd @ leaves["Wu"].t())
    want = xd + h @ leaves["Wd"].t()
    want.backward(dy.double())
    # every chained tensor (H, G, U, dH, dG, dU and the results) is rounded to bf16 once: at
    # most six independent relative errors of 2^-9 (rms of a rounding to 8 bits is smaller)
    # against each result's 2-norm
    tol = 6 * 2.0 ** -9
    for got, ref in [(y, want), (dx, xd.grad)] + [(block.grad[n], leaves[n].grad) for n in leaves]:
        off = (got.double() - ref.detach()).norm() / ref.detach().norm()
        assert float(off) <= tol


def test_block_learns_and_serves(example):
    losses, block = example.train(512, 256, 512, 12)
    assert losses[-1] < 0.8 * losses[0]
    prompt = torch.randn((5, 256), device="cuda").bfloat16()
    whole, steps = example.serve(block, prompt)
    check_device_ok()
    # H is the same in both up to a flip of its rounding; y is rounded to 8 bits
    assert float((whole.float() - steps.float()).abs().max()) <= 2.0 ** -5 * \
        float(whole.float().abs().max())


@pytest.mark.parametrize("tokens", [1, 24, 300])
def test_chained_calls_equal_the_same_calls_with_waits_between(example, tokens):
    """Kernels of calls that follow one another overlap (set-up, prefetches, the products of
    a backward pass): a chain in which every call reads what the one before it wrote gives
    the same bits as one with a wait after every call."""
    import implicit_gemm_conv_tcgen05_gb300 as igc
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    width, hidden = 264, 520
    block = example.FeedForward(width, hidden, gen)
    bias = torch.randn(hidden, generator=gen, device="cuda")
    x0 = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()

    def chain(wait):
        x, kept = x0, []
        for _ in range(12):
            G, U = (torch.empty((tokens, hidden), device="cuda", dtype=x.dtype) for _ in range(2))
            H = igc.gated_ffn(x, block.w["Wg"], block.w["Wu"], bg=bias, G=G, U=U)
            wait()
            y = igc.linear_act(H, block.w["Wd"], residual=x, act="gelu")
            wait()
            dH, dWd, _ = igc.linear_act_backward(y, H, block.w["Wd"])
            wait()
            db = [torch.empty(hidden, device="cuda") for _ in range(2)]
            dX, dWg, dWu = torch.empty_like(x), torch.empty_like(block.w["Wg"]), \
                torch.empty_like(block.w["Wu"])
            igc.gated_ffn_backward(dH, G, U, x, block.w["Wg"], block.w["Wu"], dX=dX, dWg=dWg,
                                   dWu=dWu, dbg=db[0], dbu=db[1])
            wait()
            norm = igc.grad_norm_clip([dX, dWg, dWu, dWd, *db], 1.0)
            wait()
            kept += [y, norm, dX, dWg, dWu, dWd, *db]
            x = (y.float() * 0.5 + dX.float()).bfloat16()
        torch.cuda.synchronize()
        return kept

    waited = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), waited))
    check_device_ok()
