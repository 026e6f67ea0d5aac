"""gated_ffn and gated_ffn_backward against their 64-bit forms."""

import pytest
import torch

import ffn_reference as ref
import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from test_linear_act_gpu import (BF16, F16, F32, d, generator, matrix,  # noqa: F401
                                 padded_out, width)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 777), (2, 5, 8), (16, 130, 1024), (31, 64, 4096),
          (64, 300, 200), (128, 129, 136), (129, 128, 72), (255, 200, 300), (256, 128, 256),
          (300, 1111, 650), (640, 1200, 128), (3, 11000, 64)]


def make(M, F, K, dtype, bias, seed, pad=0):
    gen = generator(M, F, K, seed)
    x = matrix(gen, M, K, dtype, pad=pad)
    wg, wu = (matrix(gen, F, K, dtype, K ** -0.5, pad=pad) for _ in range(2))
    bg, bu = ((matrix(gen, 1, F, dtype)[0].clone() for _ in range(2)) if bias else (None, None))
    return x, wg, wu, bg, bu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,F,K", SHAPES)
def test_forward_shapes(M, F, K, dtype, width):
    i = SHAPES.index((M, F, K))
    name = ref.ACTS[i % 5]
    x, wg, wu, bg, bu = make(M, F, K, dtype, i % 2 == 0, i, pad=8 * (i % 2))
    H, G, U = (torch.full((M, F), 7.0, device="cuda", dtype=dtype) for _ in range(3))
    assert igc.gated_ffn(x, wg, wu, bg=bg, bu=bu, act=name, H=H, G=G, U=U) is H
    bare = igc.gated_ffn(x, wg, wu, bg=bg, bu=bu, act=name)
    check_device_ok()
    wh, wgv, wuv = ref.gated(d(x), d(wg), d(wu), d(bg), d(bu), name, dtype)
    ref.check(G, wgv, "G")
    ref.check(U, wuv, "U")
    ref.check(H, wh, "H")
    assert torch.equal(H, bare)


@pytest.mark.parametrize("M", [5, 200])
def test_forward_one_bias_joined_weights_and_unaligned_outputs(M, width):
    F, K = 203, 264
    gen = generator(M, 31)
    x = matrix(gen, M, K, BF16)
    w = matrix(gen, 2 * F, K, BF16, K ** -0.5)
    bu = torch.randn(F, generator=gen, device="cuda")
    buf = torch.full((3, M + 1, F + 9), 9.0, device="cuda", dtype=BF16)
    H, G, U = (buf[i, :M, 1:F + 1] for i in range(3))
    igc.gated_ffn(x, w[:F], w[F:], bu=bu, act="gelu_tanh", H=H, G=G, U=U)
    check_device_ok()
    wh, wg, wu = ref.gated(d(x), d(w[:F]), d(w[F:]), None, d(bu), "gelu_tanh", BF16)
    ref.check(H, wh, "H")
    ref.check(G, wg, "G")
    ref.check(U, wu, "U")
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, :M, 1:F + 1] = False
    assert bool((buf[keep] == 9.0).all())


@pytest.mark.parametrize("M", [2, 300])
def test_forward_empty_contraction(M):
    F = 41
    bg, bu = torch.randn((2, F), device="cuda").to(F16)
    e = torch.empty((M, 0), device="cuda", dtype=F16)
    we = torch.empty((F, 0), device="cuda", dtype=F16)
    G, U = (torch.empty((M, F), device="cuda", dtype=F16) for _ in range(2))
    H = igc.gated_ffn(e, we, we, bg=bg, bu=bu, act="silu", G=G, U=U)
    check_device_ok()
    h = (ref.act("silu", d(bg)) * d(bu)).expand(M, F)
    ref.check(H, (h, ref.rounded(h, 2e-5 * h.abs(), F16)), "H")
    assert torch.equal(G, bg.expand(M, F)) and torch.equal(U, bu.expand(M, F))
    assert not bool(igc.gated_ffn(e, we, we).any())
    assert igc.gated_ffn(e[:0], we, we).shape == (0, F)


@pytest.mark.parametrize("M", [4, 260])
def test_forward_small_integers_bit_exact(M):
    """Which weight row meets which output column: sums of small integers."""
    F, K = 500, 160
    gen = generator(M, 32)
    x, wg, wu = (torch.randint(-2, 3, (n, K), generator=gen, device="cuda").to(BF16)
                 for n in (M, F, F))
    for width in (0, 128, 256):
        G, U = (torch.empty((M, F), device="cuda", dtype=BF16) for _ in range(2))
        igc.igc_set_tile_width(width)
        try:
            H = igc.gated_ffn(x, wg, wu, act="none", G=G, U=U)
        finally:
            igc.igc_set_tile_width(0)
        check_device_ok()
        g, u = d(x) @ d(wg).t(), d(x) @ d(wu).t()
        assert torch.equal(G, g.to(BF16)) and torch.equal(U, u.to(BF16))
        assert torch.equal(H, (g * u).to(BF16))


BWD_SHAPES = [(1, 1, 1), (1, 64, 64), (3, 5, 8), (50, 129, 200), (129, 130, 72), (301, 1111, 650),
              (256, 256, 256), (1500, 40, 600)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,F,K", BWD_SHAPES)
def test_backward_shapes(M, F, K, dtype, width):
    i = BWD_SHAPES.index((M, F, K))
    name = ref.ACTS[(i + 1) % 5]
    x, wg, wu, _, _ = make(M, F, K, dtype, False, 40 + i, pad=8 * (i % 2))
    gen = generator(M, F, 41)
    dh = matrix(gen, M, F, dtype, 0.5, pad=i % 3)
    g, u = (matrix(gen, M, F, dtype, 2.0, pad=i % 2) for _ in range(2))
    dX = torch.full((M, K), 7.0, device="cuda", dtype=dtype)
    dWg, dWu = (torch.full((F, K), 7.0, device="cuda", dtype=F32 if i % 2 else dtype)
                for _ in range(2))
    dbg, dbu = (torch.full((F,), 7.0, device="cuda", dtype=dtype if i % 2 else F32)
                for _ in range(2))
    igc.gated_ffn_backward(dh, g, u, x, wg, wu, act=name, dX=dX, dWg=dWg, dWu=dWu, dbg=dbg,
                           dbu=dbu)
    check_device_ok()
    ds, es = ref.gated_dgu(d(dh), d(g), d(u), name)
    wx, ww, wb = ref.grads(ds, es, d(x), [d(wg), d(wu)], dtype, dWg.dtype, dbg.dtype)
    ref.check(dX, wx[0], "dX")
    ref.check(dWg, ww[0], "dWg")
    ref.check(dWu, ww[1], "dWu")
    ref.check(dbg, wb[0], "dbg")
    ref.check(dbu, wb[1], "dbu")


def test_backward_each_gradient_alone():
    M, F, K = 150, 131, 200
    x, wg, wu, _, _ = make(M, F, K, F16, False, 50)
    gen = generator(51)
    dh, g, u = (torch.randn((M, F), generator=gen, device="cuda").to(F16) for _ in range(3))
    ds, es = ref.gated_dgu(d(dh), d(g), d(u), "silu")
    wx, ww, wb = ref.grads(ds, es, d(x), [d(wg), d(wu)], F16, F16, F32)
    dX = torch.empty((M, K), device="cuda", dtype=F16)
    igc.gated_ffn_backward(dh, g, u, None, wg, wu, dX=dX)
    dWg, dWu = (torch.empty((F, K), device="cuda", dtype=F16) for _ in range(2))
    igc.gated_ffn_backward(dh, g, u, x, None, None, dWg=dWg, dWu=dWu)
    dbg, dbu = (torch.empty(F, device="cuda") for _ in range(2))
    igc.gated_ffn_backward(dh, g, u, None, None, None, dbg=dbg, dbu=dbu)
    a = igc.gated_ffn_backward(dh, g, u, x, wg, wu)
    check_device_ok()
    for got, want, what in ((dX, wx[0], "dX"), (dWg, ww[0], "dWg"), (dWu, ww[1], "dWu"),
                            (dbg, wb[0], "dbg"), (dbu, wb[1], "dbu")):
        ref.check(got, want, what)
    assert torch.equal(a[0], dX) and torch.equal(a[1], dWg) and torch.equal(a[2], dWu)
    assert a[3] is None and a[4] is None


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_backward_against_differences(name):
    M, F, K = 40, 72, 96
    x, wg, wu, bg, bu = make(M, F, K, F16, True, 60)
    gen = generator(61)
    c = matrix(gen, M, F, F16)
    G, U = (torch.empty((M, F), device="cuda", dtype=F16) for _ in range(2))
    igc.gated_ffn(x, wg, wu, bg=bg, bu=bu, act=name, G=G, U=U)
    dX = torch.empty((M, K), device="cuda", dtype=F16)
    dWg, dWu = (torch.empty((F, K), device="cuda") for _ in range(2))
    dbg, dbu = (torch.empty(F, device="cuda") for _ in range(2))
    igc.gated_ffn_backward(c, G, U, x, wg, wu, act=name, dX=dX, dWg=dWg, dWu=dWu, dbg=dbg,
                           dbu=dbu)
    check_device_ok()

    def loss(px, pg, pu, pbg, pbu):
        return float((d(c) * ref.act(name, px @ pg.t() + pbg) * (px @ pu.t() + pbu)).sum())

    base = [d(x), d(wg), d(wu), d(bg), d(bu)]
    for at, grad in enumerate((dX, dWg, dWu, dbg, dbu)):
        step = torch.randn(base[at].shape, generator=gen, device="cuda").double()
        h = 1e-6
        hi, lo = list(base), list(base)
        hi[at] = base[at] + h * step
        lo[at] = base[at] - h * step
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        got = float((grad.double() * step).sum())
        # as for linear_act: rounding to fp16 of G, U, dG, dU and the result
        terms = float((grad.double() * step).square().sum().sqrt())
        ds, _ = ref.gated_dgu(d(c), d(G), d(U), name)
        spread = float(max(t.abs().max() for t in ds)) * base[at].numel() ** 0.5
        assert abs(got - want) <= 40 * 2.0 ** -11 * (terms + spread), (at, got, want)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("F", [1, 67, 130, 133])
def test_padding_of_outputs_is_kept(M, F, width):
    """As for linear_act: nothing past the last column is written."""
    x, wg, wu, bg, bu = make(M, F, 96, BF16, True, 70)
    (H, hb), (G, gb), (U, ub) = (padded_out(M, F, BF16) for _ in range(3))
    igc.gated_ffn(x, wg, wu, bg=bg, bu=bu, H=H, G=G, U=U)
    gen = generator(M, F, 71)
    x2 = matrix(gen, M, F, BF16)
    wg2, wu2 = (matrix(gen, 72, F, BF16) for _ in range(2))
    dh, g, u = (matrix(gen, M, 72, BF16) for _ in range(3))
    (dX, xb), (dWg, wgb), (dWu, wub) = (padded_out(r, F, BF16) for r in (M, 72, 72))
    igc.gated_ffn_backward(dh, g, u, x2, wg2, wu2, dX=dX, dWg=dWg, dWu=dWu)
    check_device_ok()
    wh, wG, wU = ref.gated(d(x), d(wg), d(wu), d(bg), d(bu), "silu", BF16)
    ds, es = ref.gated_dgu(d(dh), d(g), d(u), "silu")
    wx, ww, _ = ref.grads(ds, es, d(x2), [d(wg2), d(wu2)], BF16, BF16, F32)
    for got, want, buf, what in ((H, wh, hb, "H"), (G, wG, gb, "G"), (U, wU, ub, "U"),
                                 (dX, wx[0], xb, "dX"), (dWg, ww[0], wgb, "dWg"),
                                 (dWu, ww[1], wub, "dWu")):
        ref.check(got, want, what)
        assert bool((buf[:, F:] == 9.0).all()), what
