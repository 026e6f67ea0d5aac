"""Backward passes in which four kernels overlap (the activation's pass, dX, dW and, from 513
rows on, the sums of the bias gradients' chunks), one call after another on one workspace:
chains, threads and graphs give the same bits as the same calls with waits between them."""

import threading

import pytest
import torch

import ffn_reference as ref
import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from test_linear_act_gpu import BF16, F16, F32, d, generator, matrix, width  # noqa: F401

pytestmark = pytest.mark.gpu


def outputs(*shapes):
    return [torch.empty(s, device="cuda", dtype=t) for s, t in shapes]


@pytest.mark.parametrize("tokens", [512, 513, 700, 1300])
def test_chain_of_a_block(tokens, width):
    gen = generator(tokens, 80)
    K, F = 264, 520
    wg, wu = (matrix(gen, F, K, BF16, K ** -0.5) for _ in range(2))
    wd = matrix(gen, K, F, BF16, F ** -0.5)
    bg = torch.randn(F, generator=gen, device="cuda")
    bd = torch.randn(K, generator=gen, device="cuda").to(BF16)
    x0 = matrix(gen, tokens, K, BF16).clone()

    def chain(wait):
        x, kept = x0, []
        for _ in range(8):
            G, U, Z = outputs(((tokens, F), BF16), ((tokens, F), BF16), ((tokens, K), BF16))
            H = igc.gated_ffn(x, wg, wu, bg=bg, G=G, U=U)
            wait()
            y = igc.linear_act(H, wd, bias=bd, residual=x, act="gelu", Z=Z)
            wait()
            dH, dWd, dbd = outputs(((tokens, F), BF16), ((K, F), F32), ((K,), F32))
            igc.linear_act_backward(y, H, wd, act="gelu", Z=Z, dX=dH, dW=dWd, dbias=dbd)
            wait()
            dX, dWg, dWu, dbg, dbu = outputs(((tokens, K), BF16), ((F, K), F32), ((F, K), F32),
                                             ((F,), F32), ((F,), F32))
            igc.gated_ffn_backward(dH, G, U, x, wg, wu, dX=dX, dWg=dWg, dWu=dWu, dbg=dbg, dbu=dbu)
            wait()
            norm = igc.grad_norm_clip([dX, dWg, dWu, dWd, dbd, dbg, dbu], 1.0)
            wait()
            kept += [y, norm, dX, dWg, dWu, dWd, dbd, dbg, dbu]
            x = (y.float() * 0.5 + dX.float()).to(BF16)
        torch.cuda.synchronize()
        assert all(bool(t.isfinite().all()) for t in kept)
        return kept

    waited = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), waited))
    check_device_ok()


@pytest.mark.parametrize("M", [513, 1100])
def test_backward_passes_back_to_back(M, width):
    """Nothing but backward passes: the next call's first kernel overwrites dZ and the partial
    sums in the workspace as soon as the stream lets it."""
    gen = generator(M, 81)
    N, K = 392, 264
    x, w, wu = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16), matrix(gen, N, K, BF16)
    u = matrix(gen, M, N, BF16)
    ins = [(matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)) for _ in range(5)]

    def chain(wait):
        kept = []
        for i in range(20):
            dy, z = ins[i % 5]
            dX, dW, dWu, db, dbu = outputs(((M, K), BF16), ((N, K), BF16), ((N, K), BF16),
                                           ((N,), F32), ((N,), F32))
            if i % 2:
                igc.linear_act_backward(dy, x, w, act="silu", Z=z, dX=dX, dW=dW, dbias=db)
                kept += [dX, dW, db]
            else:
                igc.gated_ffn_backward(dy, z, u, x, w, wu, dX=dX, dWg=dW, dWu=dWu, dbg=db,
                                       dbu=dbu)
                kept += [dX, dW, dWu, db, dbu]
            wait()
        torch.cuda.synchronize()
        return kept

    waited = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), waited))
    check_device_ok()


@pytest.mark.parametrize("own_streams", [False, True])
def test_threads_with_bias_gradients(own_streams):
    gen = generator(82)
    cases, results = [], {}
    for M, N, K in ((600, 200, 136), (513, 520, 264), (900, 72, 328), (128, 300, 200)):
        x, w = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, K ** -0.5)
        dy, z = matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)

        def call(x=x, w=w, dy=dy, z=z, M=M, N=N, K=K):
            dX, dW, db = outputs(((M, K), BF16), ((N, K), F32), ((N,), F32))
            igc.linear_act_backward(dy, x, w, act="silu", Z=z, dX=dX, dW=dW, dbias=db)
            return dX, dW, db

        cases.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream() if own_streams else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            results[i] = [cases[i][0]() for _ in range(30)]
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    check_device_ok()
    for i, (_, want) in enumerate(cases):
        for got in results[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_of_chunked_sums_beside_eager_calls():
    gen = generator(83)
    M, N, K = 700, 136, 264
    x, w = matrix(gen, M, K, F16), matrix(gen, N, K, F16, K ** -0.5)
    dy, g, u = (matrix(gen, M, N, F16) for _ in range(3))
    wu = matrix(gen, N, K, F16, K ** -0.5)
    out = outputs(((M, K), F16), ((N, K), F32), ((N, K), F32), ((N,), F32), ((N,), F32))

    def call(stream_out):
        dX, dWg, dWu, dbg, dbu = stream_out
        igc.gated_ffn_backward(dy, g, u, x, w, wu, act="gelu", dX=dX, dWg=dWg, dWu=dWu, dbg=dbg,
                               dbu=dbu)

    call(out)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
        call(out)
    other = [torch.empty_like(t) for t in out]
    for _ in range(3):
        for t in out:
            t.zero_()
        call(other)
        graph.replay()
        call(other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(other, want))
    check_device_ok()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [511, 512, 513, 544, 545])
def test_row_counts_around_the_change_of_sums(M, dtype, width):
    """Bias gradients are joined in a cluster up to 512 rows, by a second kernel above."""
    N, K = 131, 72
    gen = generator(M, 84)
    x, w, wu = matrix(gen, M, K, dtype), matrix(gen, N, K, dtype), matrix(gen, N, K, dtype)
    dy, z, u = (matrix(gen, M, N, dtype, pad=i) for i in (2, 1, 1))
    dX, dW, dWu, db, dbu = outputs(((M, K), dtype), ((N, K), F32), ((N, K), F32), ((N,), dtype),
                                   ((N,), dtype))
    igc.linear_act_backward(dy, x, w, act="gelu_tanh", Z=z, dX=dX, dW=dW, dbias=db)
    check_device_ok()
    dz, ez = ref.linear_dz(d(dy), d(z), "gelu_tanh")
    wx, ww, wb = ref.grads([dz], [ez], d(x), [d(w)], dtype, F32, dtype)
    for got, want, what in ((dX, wx[0], "dX"), (dW, ww[0], "dW"), (db, wb[0], "db")):
        ref.check(got, want, what)
    igc.gated_ffn_backward(dy, z, u, x, w, wu, dX=dX, dWg=dW, dWu=dWu, dbg=db, dbu=dbu)
    check_device_ok()
    ds, es = ref.gated_dgu(d(dy), d(z), d(u), "silu")
    wx, ww, wb = ref.grads(ds, es, d(x), [d(w), d(wu)], dtype, F32, dtype)
    for got, want, what in ((dX, wx[0], "dX"), (dW, ww[0], "dWg"), (dWu, ww[1], "dWu"),
                            (db, wb[0], "dbg"), (dbu, wb[1], "dbu")):
        ref.check(got, want, what)
