"""Weights past half of the L2 that few rows of X use once are loaded with an eviction hint
(from 64e6 bytes on, where one block covers the rows): forward products on either side of
that size, with sizes that fill no block and NaN in the rows' padding."""

import pytest
import torch

import ffn_reference as ref
import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from test_linear_act_gpu import BF16, F16, F32, d, generator, matrix

pytestmark = pytest.mark.gpu

THRESHOLD = 64e6   # bytes of weights

# rows of W and K: just below and just above, neither a multiple of a block's 128 or 64
LINEAR = [(7001, 4567), (7009, 4569)]
GATED = [(3499, 4571), (3503, 4571)]


def test_the_sizes_lie_on_either_side():
    for (n, k), scale in [(s, 2) for s in LINEAR] + [(s, 4) for s in GATED]:
        assert n % 64 and k % 64 and abs(scale * n * k - THRESHOLD) < 2e5
    assert [2 * n * k >= THRESHOLD for n, k in LINEAR] == [False, True]
    assert [4 * f * k >= THRESHOLD for f, k in GATED] == [False, True]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [1, 3, 48, 130])
@pytest.mark.parametrize("N,K", LINEAR)
def test_linear(N, K, M, dtype):
    plan = igc.igc_plan_ffn(igc.PLAN_FFN_LINEAR, M, N, K)
    assert plan["small"] and plan["row_blocks"] == 1
    gen = generator(M, N, K, 90)
    x, w = matrix(gen, M, K, dtype, pad=8), matrix(gen, N, K, dtype, K ** -0.5, pad=16)
    b, r = matrix(gen, 1, N, dtype)[0].clone(), matrix(gen, M, N, dtype)
    Y = torch.full((M, N), 7.0, device="cuda", dtype=F32)
    Z = torch.full((M, N), 7.0, device="cuda", dtype=dtype)
    igc.linear_act(x, w, bias=b, act="silu", residual=r, Y=Y, Z=Z)
    check_device_ok()
    want_y, want_z = ref.linear(d(x), d(w), d(b), "silu", d(r), F32, dtype)
    ref.check(Z, want_z, "Z")
    ref.check(Y, want_y, "Y")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [1, 3, 48, 130])
@pytest.mark.parametrize("F,K", GATED)
def test_gated(F, K, M, dtype):
    plan = igc.igc_plan_ffn(igc.PLAN_FFN_GATED, M, F, K)
    assert plan["small"] and plan["row_blocks"] == 1
    gen = generator(M, F, K, 91)
    x = matrix(gen, M, K, dtype, pad=8)
    wg, wu = (matrix(gen, F, K, dtype, K ** -0.5, pad=16) for _ in range(2))
    bg, bu = (matrix(gen, 1, F, dtype)[0].clone() for _ in range(2))
    H, G, U = (torch.full((M, F), 7.0, device="cuda", dtype=dtype) for _ in range(3))
    igc.gated_ffn(x, wg, wu, bg=bg, bu=bu, act="gelu", H=H, G=G, U=U)
    check_device_ok()
    wh, wG, wU = ref.gated(d(x), d(wg), d(wu), d(bg), d(bu), "gelu", dtype)
    for got, want, what in ((G, wG, "G"), (U, wU, "U"), (H, wh, "H")):
        ref.check(got, want, what)


@pytest.mark.parametrize("M", [1, 48])
@pytest.mark.parametrize("gated", [False, True])
def test_small_integers_bit_exact(M, gated):
    """Which row of which weight meets which output column, with the hint."""
    gen = generator(M, 92)
    N, K = GATED[1] if gated else LINEAR[1]
    pad = -(-K // 8) * 8

    def ints(rows):
        t = torch.full((rows, pad), float("nan"), device="cuda", dtype=BF16)
        t[:, :K] = torch.randint(-2, 3, (rows, K), generator=gen, device="cuda")
        return t[:, :K]

    x = ints(M)
    if gated:
        wg, wu = ints(N), ints(N)
        G, U = (torch.empty((M, N), device="cuda", dtype=BF16) for _ in range(2))
        H = igc.gated_ffn(x, wg, wu, act="none", G=G, U=U)
        g, u = d(x) @ d(wg).t(), d(x) @ d(wu).t()
        check_device_ok()
        assert torch.equal(G, g.to(BF16)) and torch.equal(U, u.to(BF16))
        assert torch.equal(H, (g * u).to(BF16))
    else:
        w = ints(N)
        Y = torch.empty((M, N), device="cuda", dtype=F32)
        igc.linear_act(x, w, Y=Y)
        check_device_ok()
        assert torch.equal(Y.double(), d(x) @ d(w).t())
