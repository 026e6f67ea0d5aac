"""The layer operators together with the feed-forward ones, as examples/token_stack.py uses them:
gradients of the whole stack against a 64-bit autograd with the same dropout, overlapping kernels,
threads and streams, captured steps."""

import importlib.util
import os
import threading

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref
from conftest import ROOT
from gpu_helpers import check_device_ok
from layers_reference import BF16, generator, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "token_stack_example", os.path.join(ROOT, "examples", "token_stack.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def stack64(stack, leaves, tokens, offset):
    """The logits in 64 bits, with autograd."""
    f = torch.nn.functional
    s = leaves["E"][tokens] * stack.scale
    branch = None
    for i in range(stack.blocks + 1):
        if branch is not None:
            mask = ref.keep(s.shape[0], s.shape[1], stack.p, 1000 + i, offset).to(s.device)
            s = s + branch * (mask * (65536 / ref.threshold(stack.p)))
        h = f.layer_norm(s, (s.shape[1],), leaves[f"w{i}"], leaves[f"b{i}"], 1e-5)
        if i < stack.blocks:
            branch = (f.silu(h @ leaves[f"Wg{i}"].t()) * (h @ leaves[f"Wu{i}"].t())) @ \
                leaves[f"Wd{i}"].t()
    return h @ leaves["E"].t()


@pytest.mark.parametrize("M,V,width,hidden,blocks", [(300, 200, 136, 264, 2),
                                                     (1500, 1000, 256, 512, 1)])
def test_gradients_of_the_stack(example, M, V, width, hidden, blocks):
    gen = generator(M, V)
    stack = example.Stack(V, width, hidden, blocks, gen)
    for i in range(blocks + 1):
        stack.w[f"w{i}"].add_(torch.randn(width, generator=gen, device="cuda") * 0.2)
        stack.w[f"b{i}"].add_(torch.randn(width, generator=gen, device="cuda") * 0.2)
    tokens = torch.randint(0, V, (M,), generator=gen, device="cuda")
    dlogits = (torch.randn((M, V), generator=gen, device="cuda") / M).to(BF16)
    logits, kept = stack.forward(tokens, offset=7)
    stack.backward(tokens, kept, dlogits, offset=7)
    check_device_ok()
    leaves = {n: t.double().requires_grad_() for n, t in stack.w.items()}
    want = stack64(stack, leaves, tokens, 7)
    want.backward(dlogits.double())
    # bf16 values on the longest way: h, G, U, H and the branch forwards, the gradients of the
    # branch, H, G, U and h backwards in each block, and h, dh around them: relative errors of at
    # most 2^-9 rms each against a result's 2-norm
    tol = (10 * blocks + 4) * 2.0 ** -9
    for name, got, ref64 in [("logits", logits, want)] + \
            [(n, stack.grad[n], leaves[n].grad) for n in leaves]:
        off = float((got.double() - ref64.detach()).norm() / ref64.detach().norm())
        assert off <= tol, (name, off, tol)


def test_example_runs_and_repeats(example):
    a, first = example.train(256, 500, 128, 256, 2, 4)
    b, second = example.train(256, 500, 128, 256, 2, 4)
    check_device_ok()
    assert a == b and all(v == v for v in a)
    assert all(torch.equal(first.master[n], second.master[n]) for n in first.master)


def chain(stack, tokens, dlogits, steps, wait):
    out = []
    for step in range(steps):
        logits, kept = stack.forward(tokens, offset=step)
        wait()
        stack.backward(tokens, kept, dlogits, offset=step)
        wait()
        norm = igc.grad_norm_clip(list(stack.grad.values()), 1.0)
        wait()
        out += [logits, norm, *(t.clone() for t in stack.grad.values())]
        stack.w["E"].add_(stack.grad["E"].to(BF16), alpha=-1.0)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("M", [1, 40, 1300])
def test_chained_calls_equal_the_same_calls_with_waits_between(example, M):
    """Kernels that follow one another overlap at their ends: the bits are those of calls apart."""
    def run(wait):
        gen = generator(M, 5)
        stack = example.Stack(3000, 264, 520, 2, gen)
        tokens = torch.randint(0, 3000, (M,), generator=gen, device="cuda")
        dlogits = (torch.randn((M, 3000), generator=gen, device="cuda") / M).to(BF16)
        return chain(stack, tokens, dlogits, 4, wait)

    waited = run(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), waited))
    check_device_ok()


def calls_of(kind, gen):
    """A closure of one operator's calls; its outputs."""
    if kind == "norm":
        X, R, dY = (matrix(gen, 3000, 1000, BF16) for _ in range(3))
        m, r = torch.empty(3000, device="cuda"), torch.empty(3000, device="cuda")
        w = torch.randn(1000, generator=gen, device="cuda")

        def call():
            S, dX = torch.empty_like(R), torch.empty_like(X)
            mean, rstd = torch.empty_like(m), torch.empty_like(r)
            y = igc.layer_norm(X, w, residual=R, p=0.1, seed=4, S=S, mean=mean, rstd=rstd)
            dw, db = torch.empty_like(w), torch.empty_like(w)
            igc.layer_norm_backward(dY, S, mean, rstd, w, p=0.1, seed=4, dX=dX, dw=dw, db=db)
            return [y, S, dX, dw, db]
        return call
    if kind == "wide":
        S, dY = (matrix(gen, 200, 12000, BF16) for _ in range(2))
        m, r = torch.zeros(200, device="cuda"), torch.ones(200, device="cuda")
        return lambda: [t for t in igc.layer_norm_backward(dY, S, m, r) if t is not None]
    if kind == "embedding":
        tok = torch.randint(0, 900, (5000,), generator=gen, device="cuda")
        dY = matrix(gen, 5000, 256, BF16)
        return lambda: [igc.embedding_backward(tok, dY, V=900),
                        igc.embedding_lookup(tok, dY[:900])]
    X = matrix(gen, 700, 900, BF16)
    return lambda: [igc.dropout_add(X, 0.3, seed=9, residual=X)]


KINDS = ["norm", "wide", "embedding", "dropout"]


def test_operators_on_streams_of_their_own():
    calls = [calls_of(k, generator(k)) for k in KINDS * 2]
    alone = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    results = [[] for _ in calls]
    for _ in range(20):
        for call, stream, kept in zip(calls, streams, results):
            with torch.cuda.stream(stream):
                kept.append(call())
    torch.cuda.synchronize()
    check_device_ok()
    for kept, want in zip(results, alone):
        for got in kept:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_threads_on_the_default_stream_and_on_their_own():
    calls = [calls_of(k, generator(k, 1)) for k in KINDS]
    alone = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    failures = []

    def work(call, want, own):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own else torch.cuda.default_stream()):
                for _ in range(15):
                    got = call()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        failures.append("bits differ")
        except Exception as e:   # (a thread's exception is the test's)
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(c, a, own))
               for own in (False, True) for c, a in zip(calls, alone)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    check_device_ok()
    assert not failures, failures


def test_captured_step_draws_anew_at_each_replay():
    """A whole training step in a graph, its dropout moved on by a counter in it; two graphs with
    workspaces of their own replayed in turn."""
    gen = generator(8)
    M, V, D = 1200, 400, 128
    E = matrix(gen, V, D, BF16)
    tok = torch.randint(0, V, (M,), generator=gen, device="cuda")
    w = torch.randn(D, generator=gen, device="cuda")
    counter = torch.zeros((), device="cuda", dtype=torch.int64)

    def step(out, counter, offset=0):
        x = igc.embedding_lookup(tok, E)
        drop = dict(p=0.25, seed=3, offset=offset, step=counter)
        igc.layer_norm(x, w, residual=x, S=out["S"], Y=out["Y"], mean=out["mean"],
                       rstd=out["rstd"], **drop)
        igc.layer_norm_backward(out["Y"], out["S"], out["mean"], out["rstd"], w, dX=out["dX"],
                                dw=out["dw"], db=out["db"], **drop)
        igc.embedding_backward(tok, out["dX"], dW=out["dE"])

    def buffers():
        rows = {n: torch.empty((M, D), device="cuda", dtype=BF16) for n in ("S", "Y", "dX")}
        vecs = {n: torch.empty(k, device="cuda")
                for n, k in (("mean", M), ("rstd", M), ("dw", D), ("db", D))}
        return {**rows, **vecs, "dE": torch.empty((V, D), device="cuda")}

    outs, graphs = [buffers() for _ in range(2)], []
    for out in outs:
        out["dE"] = torch.empty((V, D), device="cuda", dtype=BF16)
        step(out, counter)
    torch.cuda.synchronize()
    for k, out in enumerate(outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(out, counter, offset=100 * k)
            counter.add_(1)
        graphs.append(graph)
    counter.zero_()
    want = buffers()
    want["dE"] = torch.empty((V, D), device="cuda", dtype=BF16)
    for n in range(6):
        graphs[n % 2].replay()
        step(want, None, offset=100 * (n % 2) + n)
        torch.cuda.synchronize()
        assert all(torch.equal(outs[n % 2][k], want[k]) for k in want), n
    check_device_ok()
