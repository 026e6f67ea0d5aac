"""dropout_add against its 64-bit form and its generator's definition."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref
from gpu_helpers import check_device_ok
from layers_reference import BF16, F16, F32, around, check, generator, matrix, rounded

pytestmark = pytest.mark.gpu

TYPES = [(BF16, BF16), (F16, F16), (F32, F32), (BF16, F32), (F32, BF16), (F16, F32), (F32, F16)]


def one(M, N, xt, yt, residual, p, seed=7, offset=0, pad=None, shift=0):
    gen = generator(M, N, str(xt), str(yt), residual)
    X = matrix(gen, M, N, xt, pad=pad, shift=shift)
    R = matrix(gen, M, N, yt, 2.0, pad=pad, shift=shift) if residual else None
    Y = matrix(gen, M, N, yt, pad=pad, shift=shift)
    assert igc.dropout_add(X, p, seed=seed, offset=offset, residual=R, Y=Y) is Y
    check_device_ok()
    y, err = ref.dropout64(X, p, seed, offset, R)
    check(Y, y, rounded(y, yt, err))
    assert bool((around(Y) == 77.0).all())


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("residual", [True, False])
def test_types(xt, yt, residual):
    for p in (0.0, 0.1, 0.5, 0.999, 1.0):
        one(37, 520, xt, yt, residual, p)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 7), (3, 8), (2, 9), (1, 4096), (129, 31), (1000, 64),
                                 (5, 8191), (33, 8200), (2, 100001), (70000, 3)])
def test_sizes(M, N):
    one(M, N, BF16, BF16, True, 0.3)
    one(M, N, F32, F32, False, 0.3)


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (8, 1), (0, 5)])
def test_any_stride_and_alignment(pad, shift):
    for xt, yt in TYPES:
        one(21, 203, xt, yt, True, 0.2, pad=pad, shift=shift)


@pytest.mark.parametrize("seed,offset", [(0, 0), (2 ** 64 - 1, 2 ** 64 - 1), (2 ** 32, 1),
                                         (5, 2 ** 32), (5, 2 ** 32 - 1)])
def test_seeds_and_offsets(seed, offset):
    one(50, 200, F32, F32, False, 0.4, seed, offset)


def test_share_of_kept_elements():
    """The mask keeps T / 65536 of many elements, within five standard deviations, and masks of
    neighbouring offsets, rows and columns agree as independent ones do."""
    M, N = 2048, 4096
    X = torch.ones(M, N, device="cuda")
    for p in (0.1, 0.5):
        T = ref.threshold(p) / 65536
        a, b = (igc.dropout_add(X, p, seed=3, offset=k) != 0 for k in (0, 1))
        check_device_ok()
        n = M * N
        assert abs(float(a.float().mean(dtype=torch.float64)) - T) <= 5 * (T * (1 - T) / n) ** 0.5
        same = T * T + (1 - T) ** 2
        for u, v in ((a, b), (a[1:], a[:-1]), (a[:, 1:], a[:, :-1]), (a[:, 8:], a[:, :-8])):
            share = float((u == v).float().mean(dtype=torch.float64))
            assert abs(share - same) <= 5 * (same * (1 - same) / u.numel()) ** 0.5


def test_mask_is_the_same_in_every_type_stride_and_operator():
    M, N, drop = 40, 300, dict(p=0.3, seed=21, offset=4)
    mask = ref.keep(M, N, 0.3, 21, 4).cuda()
    for dt in (BF16, F16, F32):
        for cols in (300, 304, 301):
            x = torch.ones(M, cols, device="cuda", dtype=dt)[:, :N]
            assert torch.equal(igc.dropout_add(x, **drop) != 0, mask)
    S = torch.empty(M, N, device="cuda")
    igc.layer_norm(torch.ones(M, N, device="cuda"), S=S, **drop)
    check_device_ok()
    assert torch.equal(S != 0, mask)


def test_in_place_and_the_gradient():
    X, R = (torch.randn(33, 400, device="cuda").bfloat16() for _ in range(2))
    want = igc.dropout_add(X, 0.1, seed=2, residual=R)
    over = R.clone()
    assert igc.dropout_add(X, 0.1, seed=2, residual=over, Y=over) is over
    x = X.clone()
    igc.dropout_add(x, 0.1, seed=2, residual=R, Y=x)
    assert torch.equal(over, want) and torch.equal(x, want)
    # the gradient of sum(dY * Y) is dY where X was kept, scaled
    dY = torch.randn(33, 400, device="cuda")
    dX = igc.dropout_add(dY, 0.1, seed=2, Y=torch.empty_like(X))
    check_device_ok()
    dx = ref.drop64(dY, 0.1, 2, 0)
    check(dX, dx, rounded(dx, BF16, 2.1 * ref.E32 * dx.abs()))


def test_dropped_infinities_and_nan_are_zeros():
    mask = ref.keep(8, 64, 0.5, 1, 0).cuda()
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = igc.dropout_add(torch.full((8, 64), bad, device="cuda"), 0.5, seed=1)
        assert bool((y[~mask] == 0).all())
        assert bool((y[mask].isnan() if bad != bad else y[mask] == bad).all())
        y = igc.dropout_add(torch.full((8, 64), bad, device="cuda", dtype=F16), 1.0, seed=1)
        assert bool((y == 0).all())
    check_device_ok()


def test_empty_and_step_and_streams():
    assert igc.dropout_add(torch.empty(0, 8, device="cuda"), 0.1, seed=1).shape == (0, 8)
    assert igc.dropout_add(torch.empty(8, 0, device="cuda"), 0.1, seed=1).shape == (8, 0)
    X = torch.randn(64, 256, device="cuda")
    step = torch.tensor([2 ** 40 + 1], device="cuda")
    a = igc.dropout_add(X, 0.3, seed=1, offset=5, step=step)
    b = igc.dropout_add(X, 0.3, seed=1, offset=2 ** 40 + 6)
    minus = igc.dropout_add(X, 0.3, seed=1, offset=2 ** 64 - 1, step=step)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = igc.dropout_add(X, 0.3, seed=1, offset=5, step=step, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(minus, igc.dropout_add(X, 0.3, seed=1, offset=2 ** 40))
    check_device_ok()


def test_offsets_past_32_bits():
    M, N, ld = 9, 64, (1 << 28) + 64
    buf = torch.empty(M * ld, device="cuda", dtype=BF16).view(M, ld)
    X, R, Y = (buf[:, k * N:(k + 1) * N] for k in range(3))
    x, r = (torch.randn(M, N, device="cuda").bfloat16() for _ in range(2))
    X.copy_(x)
    R.copy_(r)
    igc.dropout_add(X, 0.2, seed=1, residual=R, Y=Y)
    assert torch.equal(Y, igc.dropout_add(x, 0.2, seed=1, residual=r))
    # and more than 2^31 elements in one call
    M, N = 1 << 15, (1 << 16) + 8
    X = torch.ones(M, N, device="cuda", dtype=F16)
    igc.dropout_add(X, 0.2, seed=1, Y=X)
    check_device_ok()
    last = ref.philox((N // 8 - 1, M - 1, 0, 0), (1, 0))
    bits = [int(v) >> s & 0xFFFF for v in last for s in (0, 16)]
    assert [bool(v) for v in X[-1, -8:]] == [b < ref.threshold(0.2) for b in bits]
