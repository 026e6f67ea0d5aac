"""The long sums of the layer operators (a table's gradient over all positions of a token, dw and db
over all rows) on small whole numbers: fp32 holds every partial sum, so the results are the
definition's whatever the order, and one row lost, doubled or sent elsewhere shows."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from layers_reference import BF16, F16, F32, generator, matrix

pytestmark = pytest.mark.gpu


def whole(gen, rows, cols, dtype, most=4):
    t = matrix(gen, rows, cols, dtype)
    return t.copy_(torch.randint(-most, most + 1, (rows, cols), generator=gen, device="cuda"))


def tokens_of(gen, M, V, kind):
    if kind == "one":
        return torch.full((M,), V // 2, device="cuda")
    if kind == "few":                       # three tokens, and positions of none
        return torch.randint(-1, 3, (M,), generator=gen, device="cuda") * ((V - 1) // 2)
    if kind == "runs":                      # tokens of 1 to 200 positions: most cross a chunk
        t = torch.arange(M, device="cuda") // 97 % V
        return torch.where(torch.rand(M, generator=gen, device="cuda") < 0.3, V // 3, t)
    t = torch.randint(-1, V + 1, (M,), generator=gen, device="cuda")
    return torch.where(torch.rand(M, generator=gen, device="cuda") < 0.5, V - 1, t)   # frequent


def table(M, V, D, kind, yt=BF16, wt=F32, accumulate=False, scale=0.5):
    gen = generator(M, V, D, kind)
    dY, dW = whole(gen, M, D, yt), whole(gen, V, D, wt)
    tok = tokens_of(gen, M, V, kind)
    inside = (tok >= 0) & (tok < V)
    sums = torch.zeros((V, D), device="cuda", dtype=torch.float64)
    step = max(1, (1 << 26) // D)
    for i in range(0, M, step):
        at = inside[i:i + step]
        sums.index_add_(0, tok[i:i + step][at], dY[i:i + step][at].double())
    assert float(sums.abs().max()) < 2 ** 24 and 4 * M < 2 ** 24
    want = sums * scale + (dW.double() if accumulate else 0)
    igc.embedding_backward(tok, dY, scale=scale, dW=dW, accumulate=accumulate)
    check_device_ok()
    assert torch.equal(dW, want.to(wt)), (dW.double() - want.to(wt).double()).abs().max()


# positions on either side of the lengths of a chunk (32, 64 and 128), for widths of every number
# of chunks to a block: one of 1024 columns and more, up to sixteen of 64
@pytest.mark.parametrize("D,M", [(4096, 8192), (4096, 8193), (4096, 16384), (4096, 16385),
                                 (4096, 16500), (40001, 1664), (40001, 1665), (1024, 65536),
                                 (1024, 65537), (520, 64513), (520, 129025), (256, 262144),
                                 (256, 262145), (128, 524288), (128, 524289), (72, 932100)])
@pytest.mark.parametrize("kind", ["one", "few", "runs", "frequent"])
def test_chunks_of_positions(D, M, kind):
    table(M, 700, D, kind)
    table(M, 700, D, kind, accumulate=True)


@pytest.mark.parametrize("D", [64, 40, 8])
@pytest.mark.parametrize("M", [524289, 1048576, 1048577, 1300003])
def test_blocks_of_sixteen_chunks(D, M):
    """Up to 2048 positions to a block, each chunk of 64 and of 128."""
    for kind in ("one", "runs", "frequent"):
        table(M, 90000, D, kind, yt=F16)
        table(M, 900, D, kind, yt=F32, accumulate=True)


@pytest.mark.parametrize("M", [1, 2, 37, 1023, 1024, 1025, 5000, 33000])
@pytest.mark.parametrize("kind", ["one", "few", "runs", "frequent"])
def test_few_positions_and_their_neighbours(M, kind):
    table(M, 331, 200, kind)
    table(M, 331, 777, kind, yt=F16, accumulate=True)


# rows on either side of the joins in one cluster, and many; widths of every kernel
@pytest.mark.parametrize("N", [61, 64, 122, 250, 256, 504, 777, 1024, 1498, 2048, 2500, 4000, 5992,
                               8192, 12001, 16384, 20400, 32768, 40001])
@pytest.mark.parametrize("M", [1, 7, 9, 600, 3000, 20000])
def test_sums_over_rows(M, N):
    if M * N > 1 << 26:
        M = (1 << 26) // N
    gen = generator(M, N)
    dtype, stream = ((BF16, BF16), (BF16, F32), (F32, F32), (F16, F32))[(M + N) % 4]
    dY, S = whole(gen, M, N, dtype), whole(gen, M, N, stream)
    mean = torch.randint(-2, 3, (M,), generator=gen, device="cuda").float()
    rstd = 2.0 ** torch.randint(-1, 2, (M,), generator=gen, device="cuda").float()
    # (h in steps of 1/2 up to 12, dY h up to 48: sums under 2^24 steps)
    assert M * 96 < 2 ** 24
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dS = torch.empty_like(S)
    igc.layer_norm_backward(dY, S, mean, rstd, dS=dS, dw=dw, db=db)
    check_device_ok()
    y = dY.double()
    h = (S.double() - mean.double()[:, None]) * rstd.double()[:, None]
    assert torch.equal(db.double(), y.sum(0)) and torch.equal(dw.double(), (y * h).sum(0))
    igc.layer_norm_backward(dY, S, mean, rstd, dw=dw)      # without dS, alone
    check_device_ok()
    assert torch.equal(dw.double(), (y * h).sum(0))
