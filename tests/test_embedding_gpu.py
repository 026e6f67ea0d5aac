"""embedding_lookup and embedding_backward against their 64-bit forms."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref
from gpu_helpers import check_device_ok
from layers_reference import BF16, F16, F32, around, check, generator, matrix, rounded

pytestmark = pytest.mark.gpu

TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]


def draw_tokens(gen, M, V, kind, dtype=torch.int64):
    if kind == "one":
        t = torch.full((M,), V // 2, device="cuda")
    elif kind == "few":
        t = torch.randint(0, min(V, 3), (M,), generator=gen, device="cuda") * ((V - 1) // 2)
    elif kind == "frequent":                # half of them one token, the rest anywhere
        t = torch.randint(0, V, (M,), generator=gen, device="cuda")
        t[torch.rand(M, generator=gen, device="cuda") < 0.5] = V - 1
    elif kind == "none":
        t = torch.randint(0, 2, (M,), generator=gen, device="cuda") * (V + 1) - 1   # -1 and V
    else:                                   # anywhere, and outside
        t = torch.randint(-V // 8 - 1, V + V // 8 + 1, (M,), generator=gen, device="cuda")
        t[::7] = -1
        if dtype == torch.int64:
            t[::11] = 2 ** 40 + V // 2      # (its lower half is a token)
            t[5::13] = -2 ** 40
    return t.to(dtype)


def lookup(M, V, D, wt, yt, kind="any", itype=torch.int64, pad=None, shift=0, scale=2.5):
    gen = generator(M, V, D, str(wt), kind)
    W = matrix(gen, V, D, wt, pad=pad, shift=shift)
    tokens = draw_tokens(gen, M, V, kind, itype)
    Y = matrix(gen, M, D, yt, pad=pad, shift=shift)
    assert igc.embedding_lookup(tokens, W, scale=scale, Y=Y) is Y
    check_device_ok()
    y = ref.lookup64(tokens, W, scale)
    check(Y, y, rounded(y, yt, ref.E32 * y.abs()) * (y != 0))
    assert bool((around(Y) == 77.0).all())


def backward(M, V, D, yt, wt, kind="any", itype=torch.int64, pad=None, shift=0, scale=2.5,
             accumulate=False):
    gen = generator(M, V, D, str(yt), kind, 1)
    dY = matrix(gen, M, D, yt, pad=pad, shift=shift)
    tokens = draw_tokens(gen, M, V, kind, itype)
    dW = matrix(gen, V, D, wt, pad=pad, shift=shift)
    old = dW.clone()
    assert igc.embedding_backward(tokens, dY, scale=scale, dW=dW, accumulate=accumulate) is dW
    check_device_ok()
    dw, err = ref.lookup_backward64(tokens, dY, V, scale)
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[tokens[(tokens >= 0) & (tokens < V)].long()] = True
    if accumulate:
        assert torch.equal(dW[~touched], old[~touched])
        dw = dw + old.double()
        err = err + 2 * ref.E32 * dw.abs()
    else:
        assert not bool(dW[~touched].any())
    check(dW[touched], dw[touched], rounded(dw, wt, err)[touched])
    assert bool((around(dW) == 77.0).all())
    return dW


@pytest.mark.parametrize("wt,yt", TYPES)
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_lookup_types(wt, yt, itype):
    for M, D in ((1, 8), (70, 200), (4000, 1000)):
        lookup(M, 331, D, wt, yt, itype=itype)


@pytest.mark.parametrize("M,V,D", [(1, 1, 1), (3, 2, 7), (64, 1000, 4096), (5, 50, 40001),
                                   (20000, 7, 3), (3001, 999, 2056)])
def test_lookup_sizes(M, V, D):
    lookup(M, V, D, BF16, BF16)
    lookup(M, V, D, F32, F32, kind="none")


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (8, 1), (0, 5)])
def test_any_stride_and_alignment(pad, shift):
    for a, b in TYPES:
        lookup(50, 40, 203, a, b, pad=pad, shift=shift)
        for M in (50, 1500):
            backward(M, 40, 203, a, b, pad=pad, shift=shift)
            backward(M, 40, 203, a, b, pad=pad, shift=shift, accumulate=True)


@pytest.mark.parametrize("yt,wt", TYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_backward_types(yt, wt, accumulate, itype):
    for M, V, D in ((1, 5, 8), (70, 331, 200), (3000, 331, 1032), (5000, 20000, 72)):
        backward(M, V, D, yt, wt, accumulate=accumulate, itype=itype)


# the numbers of positions on either side of the change of kernels and of the sort's shares
@pytest.mark.parametrize("M", [1, 2, 31, 32, 33, 127, 129, 1023, 1024, 1025, 1056, 1057, 8191,
                               8193, 16385, 40000])
@pytest.mark.parametrize("kind", ["any", "one", "few", "frequent", "none"])
def test_backward_positions(M, kind):
    backward(M, 700, 24, F32, F32, kind)
    backward(M, 700, 24, BF16, F32, kind, accumulate=True)


# tables on either side of the digits of the sort
@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 33, 63, 64, 511, 512, 513, 131071, 131072, 262143,
                               262144, 300000])
def test_backward_tables(V):
    for M in (100, 4000):
        backward(M, V, 16, BF16, BF16)
        backward(M, V, 16, BF16, F32, "frequent", itype=torch.int32)


@pytest.mark.parametrize("D", [1, 7, 8, 9, 255, 257, 1024, 1025, 3001, 8193, 40001])
def test_backward_widths(D):
    for M in (40, 1100):
        backward(M, 50, D, F16, F32)
        backward(M, 50, D, F32, F32, "one")


@pytest.mark.parametrize("M", [65536, 65537, 131073, 262144, 262145, 1200000])
def test_many_positions(M):
    """The sort's blocks hold one, several and many runs of positions."""
    backward(M, 90000, 9, F32, F32, "frequent")
    backward(M, 1000, 4, BF16, F32, "any", itype=torch.int32)
    backward(M, 300, 8, F32, F32, "any")        # (one pass of the sort)


@pytest.mark.parametrize("D", [8, 16, 40, 64, 100, 128, 500, 520])
def test_narrow_rows_share_blocks(D):
    for M in (1100, 5000, 70000):
        backward(M, 900, D, BF16, F32)
        backward(M, 17, D, F16, F16, "few")


def test_a_token_at_every_position():
    """One token's 70000 rows: sums of sums over all chunks."""
    backward(70000, 3, 512, BF16, F32, "one")
    backward(33000, 3, 64, F32, F32, "few", accumulate=True)


def test_defaults_and_empty():
    W = torch.randn(9, 16, device="cuda").half()
    tok = torch.tensor([3, 3, 8], device="cuda")
    y = igc.embedding_lookup(tok, W)
    assert torch.equal(y, W[tok])
    dW = igc.embedding_backward(tok, y, V=9)
    check_device_ok()
    assert dW.dtype == F16 and dW.shape == (9, 16)
    assert torch.equal(dW[8], y[2]) and not bool(dW[:3].any())
    none = torch.empty(0, device="cuda", dtype=torch.int64)
    assert igc.embedding_lookup(none, W).shape == (0, 16)
    assert igc.embedding_lookup(tok, W[:0]).abs().sum() == 0
    dW = torch.full((9, 16), 3.0, device="cuda")
    empty = torch.empty((0, 16), device="cuda")
    igc.embedding_backward(none, empty, dW=dW, accumulate=True)
    assert bool((dW == 3).all())
    igc.embedding_backward(none, empty, dW=dW)
    check_device_ok()
    assert not bool(dW.any())


def test_infinities_reach_their_rows_alone():
    for M in (60, 2000):
        dY = torch.ones(M, 32, device="cuda")
        tok = torch.arange(M, device="cuda") % 50
        dY[7] = float("inf")
        dY[11, 3] = float("nan")
        tok[20] = -1
        dY[20] = float("nan")
        dW = igc.embedding_backward(tok, dY, V=50)
        check_device_ok()
        assert bool(dW[7].isinf().all()) and int(dW.isnan().sum()) == 1 and bool(dW[11, 3].isnan())
    W = torch.full((3, 8), float("inf"), device="cuda")
    assert not bool(igc.embedding_lookup(torch.tensor([-1, 3], device="cuda"), W, scale=0.0).any())


def test_repeatable_streams_and_graphs():
    gen = generator(5)
    for M in (500, 9000):
        tok = draw_tokens(gen, M, 300, "frequent")
        dY = torch.randn(M, 520, generator=gen, device="cuda")
        first = igc.embedding_backward(tok, dY, V=300)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        second = igc.embedding_backward(tok, dY, V=300, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(first, second)
        dW, y = torch.empty_like(first), torch.empty_like(dY)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            igc.embedding_backward(tok, dY, dW=dW)
            igc.embedding_lookup(tok, dW, Y=y)
        dW.zero_()
        graph.replay()
        check_device_ok()
        assert torch.equal(dW, first) and torch.equal(y, first[tok])


def test_offsets_past_32_bits():
    V, D = 9, 64
    ld = (1 << 28) + 64
    buf = torch.zeros(V * ld, device="cuda", dtype=BF16).view(V, ld)
    W, dW = buf[:, :D], buf[:, D:2 * D]
    w = torch.randn(V, D, device="cuda").bfloat16()
    W.copy_(w)
    for M in (200, 2000):
        tok = torch.arange(M, device="cuda") * 5 % V
        y = igc.embedding_lookup(tok, W, scale=0.5)
        assert torch.equal(y, igc.embedding_lookup(tok, w, scale=0.5))
        igc.embedding_backward(tok, y, dW=dW)
        assert torch.equal(dW, igc.embedding_backward(tok, y, V=V))
    check_device_ok()
