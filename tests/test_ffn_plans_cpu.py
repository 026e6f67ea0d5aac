"""igc_plan_ffn for the products of backward passes: they are planned by the sizes alone, as of
closely packed rows (padded to 8 elements), which start on 128-byte lines only where a row is a
whole number of them; and dX goes to the tiles where its own then run beside dW's."""

import pytest

import implicit_gemm_conv_tcgen05_gb300 as igc

X, W = igc.PLAN_FFN_GRAD_X, igc.PLAN_FFN_GRAD_W


@pytest.mark.parametrize("op", [X, W])
@pytest.mark.parametrize("n,k", [(1024, 1024), (1001, 1024), (1024, 777), (1001, 777)])
def test_tile_estimate_knows_rows_off_the_lines(op, n, k):
    """3000 rows: dX 12 x 4 tiles over n, dW 4 x 4 over 3000; one round on 76 pairs of CTAs, each
    a column half when at most half of the pairs are busy."""
    for count in (1, 2):
        p = igc.igc_plan_ffn(op, 3000, n, k, count)
        lines = n % 64 == 0 and k % 64 == 0
        stages = -(-n // 128) * count if op == X else -(-3000 // 128)
        tiles = 12 * -(-k // 256) if op == X else -(-n // 256) * -(-k // 256) * count
        whole = max(0.6, 65.536 / (165 if lines else 82))
        half = max(0.32, 49.152 / (165 if lines else 82))
        busy256 = stages * (half if 2 * tiles <= 76 else whole)
        # the plan may take 128-wide tiles where these are done sooner, never a longer schedule
        assert p["tiles_ns"] <= 1000 * (4.5 + busy256) * 1.001 + 1
        if not lines:
            on = igc.igc_plan_ffn(op, 3000, -(-n // 64) * 64, -(-k // 64) * 64, count)
            assert p["tiles_ns"] > 1.15 * on["tiles_ns"]


def test_rows_off_the_lines_near_the_crossover():
    """With whole lines the tiles would be done sooner; as the calls plan them they are not."""
    for op, odd, whole, count in ((X, (900, 1000, 1000), (900, 1024, 1024), 2),
                                  (W, (1500, 1001, 777), (1500, 1024, 832), 1)):
        p = igc.igc_plan_ffn(op, *odd, count)
        assert p["small"] and p["small_ns"] < p["tiles_ns"]
        assert not igc.igc_plan_ffn(op, *whole, count)["small"]


def test_dx_beside_dw():
    """dX and dW of 509 x 1001 x 777: 8 and 16 tiles as column halves run side by side on 152 SMs;
    alone the other kernel would be done sooner."""
    x, w = igc.igc_plan_ffn(X, 509, 1001, 777), igc.igc_plan_ffn(W, 509, 1001, 777)
    assert not w["small"]
    assert not x["small"] and x["small_ns"] < x["tiles_ns"]
    # on a GPU too small for both at once, dX keeps the kernel that is faster alone
    tiny = igc.igc_plan_ffn(X, 509, 1001, 777, sms=24)
    assert tiny["small"] == (tiny["small_ns"] < tiny["tiles_ns"])


def test_estimates_decide_otherwise():
    for op in (X, W):
        for m, n, k in [(1, 64, 64), (64, 4096, 4096), (8192, 8192, 8192), (50, 129, 200)]:
            p = igc.igc_plan_ffn(op, m, n, k)
            assert p["small"] == (p["small_ns"] < p["tiles_ns"]) or op == X
