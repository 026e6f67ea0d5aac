"""Layer operators on values whose fp32 sums are exact in any order, so that the results are those
of the definition to the last bit."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from layers_reference import check, generator, matrix, norm_backward64, rounded

pytestmark = pytest.mark.gpu


def constant_rows(M, N, pad):
    """Row i holds i + 1 throughout: every sum over it is a whole number under 2^24."""
    assert M * N < 2 ** 24
    X = matrix(generator(M, N), M, N, torch.float32, pad=pad)
    X.copy_(torch.arange(1, M + 1, device="cuda", dtype=torch.float32)[:, None].expand(M, N))
    return X


# widths of every kernel, for which a rounded 1/N times N i is often not i; pad None: rows on 16-byte boundaries
@pytest.mark.parametrize("N", [61, 122, 241, 488, 749, 1000, 1498, 2021, 2996, 4067, 5992, 8163,
                               12037, 16268, 20002])
@pytest.mark.parametrize("pad", [None, 1])
def test_rows_of_one_value_have_their_mean(N, pad):
    """The mean is the sum divided by N, not multiplied by a rounded 1/N (which puts it one step of
    fp32 off at 1000 columns of 1000.0, and Y there 0.02 off): a row of one value gives b."""
    for M in (5, 800):
        X = constant_rows(M, N, pad)
        gen = generator(N)
        w, b = (torch.randn(N, generator=gen, device="cuda") for _ in range(2))
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        y = igc.layer_norm(X, w, b, eps=2.0 ** -20, mean=mean, rstd=rstd)
        check_device_ok()
        assert torch.equal(mean, X[:, 0]) and bool((rstd == 1024.0).all())
        assert torch.equal(y, b.expand(M, N))


# widths of every kernel of the backward pass
@pytest.mark.parametrize("N", [61, 122, 241, 488, 1000, 1498, 2021, 2500, 4067, 5992, 8163, 12037,
                               16268, 20400, 32001, 40001])
@pytest.mark.parametrize("pad", [None, 1])
def test_gradients_of_one_value_to_a_row_cancel(N, pad):
    """A norm does not change with a shift of its row: where h is 0 the gradient of the row's sum
    is 0, which asks for the mean of g as exactly as the forward pass does for that of S."""
    for M in (5, 400):
        dY = constant_rows(M, N, pad)
        S, dS = (matrix(generator(N), M, N, torch.float32, pad=pad) for _ in range(2))
        S.zero_()
        dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        igc.layer_norm_backward(dY, S, torch.zeros(M, device="cuda"),
                                torch.full((M,), 2.0, device="cuda"), dS=dS, dw=dw, db=db)
        check_device_ok()
        assert not bool(dS.any()) and not bool(dw.any())
        assert bool((db == M * (M + 1) // 2).all())


@pytest.mark.parametrize("N,pad", [(9, 7), (100, 4), (249, 7), (9, 0), (100, 1), (513, 0), (1001, 0),
                                   (7001, 2), (9001, 0)])
@pytest.mark.parametrize("add", [False, True])
def test_rows_far_from_zero_with_a_part_of_a_unit(N, pad, add):
    """Rows of 2^110 whose last unit of eight columns is not whole: what lies past a row's end has
    no part in its sums, also where 2^110 rstd is past fp32's range."""
    M = 70
    X = matrix(generator(N), M, N, torch.float32, pad=pad)
    X.fill_(2.0 ** 110)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    igc.layer_norm(X, eps=2.0 ** -60, mean=mean, rstd=rstd)
    check_device_ok()
    assert bool((mean == 2.0 ** 110).all()) and bool((rstd == 2.0 ** 30).all())
    dY, A, dS = (matrix(generator(N, k), M, N, torch.float32, pad=pad) for k in range(3))
    dY.copy_(torch.randint(-8, 9, (M, N), device="cuda"))
    A = A if add else None
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    igc.layer_norm_backward(dY, X, mean, rstd, dS_add=A, dS=dS, dw=dw, db=db)
    check_device_ok()
    assert not bool(dw.any()) and torch.equal(db, dY.sum(0))
    want, err = norm_backward64(dY, X, mean, rstd, None, A)[:2]
    check(dS, want, rounded(want, torch.float32, err))


def test_offset_and_step_add_up():
    """Calls differ where offset + step does: a neighbour's offset is the next step's."""
    X = torch.ones(64, 512, device="cuda")
    step = torch.tensor(6, device="cuda")
    a = igc.dropout_add(X, 0.5, seed=3, offset=1, step=step)
    step.add_(1)
    b = igc.dropout_add(X, 0.5, seed=3, offset=0, step=step)
    c = igc.dropout_add(X, 0.5, seed=4, offset=0, step=step)
    check_device_ok()
    assert torch.equal(a, b) and not torch.equal(b, c)
