"""layer_norm and layer_norm_backward against their 64-bit forms."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref
from gpu_helpers import check_device_ok
from layers_reference import BF16, F16, F32, around, check, generator, matrix, rounded

pytestmark = pytest.mark.gpu

TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]
SEED, OFFSET = 0x123456789ABCDEF0, 0x100000003


def forward(M, N, dtype, stream, residual, p, pad=None, shift=0, wtype=None, affine=True,
            mean=0.3, store=True, eps=1e-5):
    """One call against the 64-bit form; returns what the backward pass needs."""
    gen = generator(M, N, str(dtype), str(stream), residual, p)
    X = matrix(gen, M, N, dtype if residual or p else stream, 1.5, mean, pad, shift)
    R = matrix(gen, M, N, stream, 2.0, mean, pad, shift) if residual else None
    w = torch.randn(N, generator=gen, device="cuda").to(wtype or F32) if affine else None
    b = torch.randn(N, generator=gen, device="cuda").to(wtype or F32) if affine else None
    Y = matrix(gen, M, N, dtype, pad=pad, shift=shift)
    stype = stream if residual or not p else X.dtype
    S = matrix(gen, M, N, stype, pad=pad, shift=shift) if store else None
    m, r = (torch.empty(M, device="cuda") if store else None for _ in range(2))
    out = igc.layer_norm(X, w, b, eps=eps, residual=R, p=p, seed=SEED, offset=OFFSET, Y=Y, S=S,
                         mean=m, rstd=r)
    check_device_ok()
    assert out is Y
    s, err = ref.dropout64(X, p, SEED, OFFSET, R)
    if residual is False and p == 0.0:
        err = err * 0
    y, dy, mean64, dm, rstd64, dr = ref.norm64(s, err, w, b, eps)
    check(Y, y, rounded(y, dtype, dy), "Y")
    assert bool((around(Y) == 77.0).all())
    if store:
        check(S, s, rounded(s, stype, err), "S")
        check(m, mean64, dm + ref.E32 * mean64.abs(), "mean")
        check(r, rstd64, dr + ref.E32 * rstd64, "rstd")
        assert bool((around(S) == 77.0).all())
    return X, R, w, S, m, r, gen


def backward(M, N, dtype, stream, add, p, pad=None, shift=0, wtype=None, affine=True, dwtype=F32,
             outputs=("dS", "dX", "dw", "db")):
    gen = generator(M, N, str(dtype), str(stream), add, p, 1)
    dY = matrix(gen, M, N, dtype, 0.5, 0.05, pad, shift)
    S = matrix(gen, M, N, stream, 2.0, 0.4, pad, shift)
    A = matrix(gen, M, N, stream, 0.5, 0.0, pad, shift) if add else None
    w = torch.randn(N, generator=gen, device="cuda").to(wtype or F32) if affine else None
    s = S.double()
    mean = s.mean(1).float()
    rstd = torch.rsqrt(s.var(1, correction=0) + 1e-5).float()
    dS = matrix(gen, M, N, stream, pad=pad, shift=shift) if "dS" in outputs else None
    dX = matrix(gen, M, N, dtype, pad=pad, shift=shift) if "dX" in outputs else None
    dw = torch.empty(N, device="cuda", dtype=dwtype) if "dw" in outputs else None
    db = torch.empty(N, device="cuda", dtype=dwtype) if "db" in outputs else None
    got = igc.layer_norm_backward(dY, S, mean, rstd, w, dS_add=A, p=p, seed=SEED, offset=OFFSET,
                                  dS=dS, dX=dX, dw=dw, db=db)
    check_device_ok()
    assert all(a is b for a, b in zip(got, (dS, dX, dw, db)))
    ds, err, dw64, ew, db64, eb = ref.norm_backward64(dY, S, mean, rstd, w, A)
    if dS is not None:
        check(dS, ds, rounded(ds, stream, err), "dS")
        assert bool((around(dS) == 77.0).all())
    if dX is not None:
        dx = ref.drop64(ds, p, SEED, OFFSET)
        scale = 65536 / max(ref.threshold(p), 1)
        off = torch.where(dx == 0, 0, err * scale + 3 * ref.E32 * dx.abs())
        check(dX, dx, rounded(dx, dtype, off), "dX")
        assert bool((around(dX) == 77.0).all())
    if dw is not None:
        check(dw, dw64, rounded(dw64, dwtype, ew), "dw")
    if db is not None:
        check(db, db64, rounded(db64, dwtype, eb), "db")


# every width on either side of a change of kernel or of work to a thread
WIDTHS = [1, 2, 7, 8, 9, 63, 64, 250, 256, 257, 512, 513, 777, 1000, 1024, 1025, 2048, 2050, 4096,
          4104, 8192, 8193, 12000, 16384, 16392, 28672, 28680, 40008, 70001]


@pytest.mark.parametrize("N", WIDTHS)
def test_forward_widths(N):
    dtype, stream = TYPES[WIDTHS.index(N) % len(TYPES)]
    for M in (1, 7):
        forward(M, N, dtype, stream, True, 0.25)
    forward(5, N, BF16, BF16, False, 0.0, store=False)


@pytest.mark.parametrize("N", WIDTHS)
def test_backward_widths(N):
    dtype, stream = TYPES[WIDTHS.index(N) % len(TYPES)]
    for M in (1, 7):
        backward(M, N, dtype, stream, True, 0.25)
    backward(37, N, BF16, BF16, False, 0.0)


@pytest.mark.parametrize("M", [2, 3, 4, 5, 33, 128, 607, 1215, 1217, 5000])
def test_row_counts(M):
    """Fewer rows than blocks, as many, and several to a block."""
    for N in (40, 300, 600, 1500):
        forward(M, N, BF16, F32, True, 0.1)
        backward(M, N, BF16, F32, True, 0.1)
    backward(M, 9000, F16, F16, True, 0.1)


# every width of work to a thread, whole units of eight columns and not, with so many rows that
# each group of threads walks down several
@pytest.mark.parametrize("M,N", [(15000, 64), (7500, 71), (15000, 250), (9000, 512), (8000, 777),
                                 (7400, 1024), (4000, 1030), (4000, 1536), (2500, 2048),
                                 (2400, 2510), (2300, 3500),
                                 (2000, 4096), (1000, 6001), (1000, 8000), (800, 8192), (700, 12001),
                                 (700, 16384), (300, 20001), (150, 32768)])
@pytest.mark.parametrize("dtype,stream", TYPES)
def test_many_rows(M, N, dtype, stream):
    forward(M, N, dtype, stream, True, 0.1)
    forward(M, N, dtype, stream, False, 0.0)
    backward(M, N, dtype, stream, True, 0.1)
    backward(M, N, dtype, stream, False, 0.0, outputs=("dS", "dw"))


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_types(dtype, stream, residual, p):
    for N in (200, 4096, 17000):
        forward(19, N, dtype, stream, residual, p)
        backward(19, N, dtype, stream, residual, p)
        forward(19, N, dtype, stream, residual, p, affine=False)
        backward(19, N, dtype, stream, residual, p, affine=False)
        forward(19, N, dtype, stream, residual, p, wtype=dtype)
        backward(19, N, dtype, stream, residual, p, wtype=dtype, dwtype=dtype)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (8, 1), (0, 5)])
def test_any_stride_and_alignment(dtype, stream, pad, shift):
    for N in (9, 255, 1027, 9001, 17001):
        forward(6, N, dtype, stream, True, 0.1, pad, shift)
        backward(6, N, dtype, stream, True, 0.1, pad, shift)


@pytest.mark.parametrize("M,N", [(1, 9), (2048, 64), (2049, 64), (512, 250), (513, 250), (128, 510),
                                 (129, 510), (64, 1000), (65, 1000), (40, 1530), (41, 1530),
                                 (16, 4096), (17, 4096), (7, 8191), (8, 8192), (9, 8192)])
def test_few_rows_joined_in_a_cluster(M, N):
    """On either side of the rows up to which one cluster adds its blocks' column sums."""
    backward(M, N, BF16, BF16, False, 0.0, wtype=BF16, dwtype=BF16)
    backward(M, N, F16, F32, True, 0.1, outputs=("dX", "db"))
    backward(M, N, F32, F32, True, 0.1, outputs=("dw",))


@pytest.mark.parametrize("outputs", [("dS",), ("dX",), ("dw",), ("db",), ("dS", "db"),
                                     ("dX", "dw", "db")])
def test_some_of_the_gradients(outputs):
    for N in (100, 2000, 9000):
        backward(11, N, BF16, F32, True, 0.1, outputs=outputs)


def test_defaults_and_no_rows():
    X = torch.randn(6, 96, device="cuda").half()
    y = igc.layer_norm(X)
    m, r = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    assert torch.equal(igc.layer_norm(X, mean=m, rstd=r), y) and y.dtype == F16
    dS, dX, dw, db = igc.layer_norm_backward(y, X, m, r)
    assert dX is None and dS.dtype == F16 and dw.dtype == db.dtype == F32
    ds, err, dw64, ew, db64, eb = ref.norm_backward64(y, X, m, r, None, None)
    check(dS, ds, rounded(ds, F16, err))
    check(dw, dw64, rounded(dw64, F32, ew))
    e = torch.empty((0, 96), device="cuda", dtype=F16)
    assert igc.layer_norm(e).shape == (0, 96)
    dw, db = (torch.full((96,), 5.0, device="cuda") for _ in range(2))
    v = torch.empty(0, device="cuda")
    igc.layer_norm_backward(e, e, v, v, dw=dw, db=db)
    check_device_ok()
    assert not bool(dw.any()) and not bool(db.any())


def test_in_place_streams():
    """S over the residual, dS over the gradient that is added: the bits of separate buffers."""
    for N in (100, 4096, 9000, 40000):
        gen = generator(N)
        X, R = (matrix(gen, 9, N, BF16) for _ in range(2))
        S, Y = torch.empty_like(R), torch.empty(9, N, device="cuda", dtype=BF16)
        m, r = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        drop = dict(p=0.1, seed=3)
        igc.layer_norm(X, residual=R, Y=Y, S=S, mean=m, rstd=r, **drop)
        R2 = matrix(gen, 9, N, BF16)
        R2.copy_(R)
        Y2 = igc.layer_norm(X, residual=R2, S=R2, **drop)
        assert torch.equal(R2, S) and torch.equal(Y2, Y)
        A = matrix(gen, 9, N, BF16)
        dS, dX = torch.empty_like(S), torch.empty_like(X)
        igc.layer_norm_backward(Y, S, m, r, dS_add=A, dS=dS, dX=dX, **drop)
        dX2 = torch.empty_like(X)
        igc.layer_norm_backward(Y, S, m, r, dS_add=A, dS=A, dX=dX2, **drop)
        check_device_ok()
        assert torch.equal(A, dS) and torch.equal(dX2, dX)


@pytest.mark.parametrize("N,pad,shift", [(100, 0, 1), (777, 0, 0), (4097, 3, 5), (12001, 0, 3),
                                         (20003, 2, 7)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_in_place_streams_off_boundaries(N, pad, shift, stream):
    """The same where a 16-byte piece holds what two lanes, warps or rows write."""
    gen = generator(N, str(stream))
    X, R = matrix(gen, 65, N, BF16, pad=pad, shift=shift), \
        matrix(gen, 65, N, stream, pad=pad, shift=shift)
    S, Y = (matrix(gen, 65, N, t, pad=pad, shift=shift) for t in (stream, BF16))
    m, r = torch.empty(65, device="cuda"), torch.empty(65, device="cuda")
    drop = dict(p=0.1, seed=3)
    igc.layer_norm(X, residual=R, Y=Y, S=S, mean=m, rstd=r, **drop)
    Y2 = matrix(gen, 65, N, BF16, pad=pad, shift=shift)
    igc.layer_norm(X, residual=R, S=R, Y=Y2, **drop)
    assert torch.equal(R, S) and torch.equal(Y2, Y)
    assert bool((around(R) == 77.0).all()) and bool((around(Y2) == 77.0).all())
    A, dS = (matrix(gen, 65, N, stream, pad=pad, shift=shift) for _ in range(2))
    dX, dX2 = (matrix(gen, 65, N, BF16, pad=pad, shift=shift) for _ in range(2))
    igc.layer_norm_backward(Y, S, m, r, dS_add=A, dS=dS, dX=dX, **drop)
    igc.layer_norm_backward(Y, S, m, r, dS_add=A, dS=A, dX=dX2, **drop)
    check_device_ok()
    assert torch.equal(A, dS) and torch.equal(dX2, dX)
    assert bool((around(A) == 77.0).all()) and bool((around(dX2) == 77.0).all())


def test_rows_far_from_zero_and_constant_rows():
    """A mean that is 4096 times the spread cancels nothing but its own rounding; a row of one
    value has variance 0 and gives b."""
    forward(5, 4096, F32, F32, False, 0.0, mean=6000.0)
    forward(5, 20000, F32, F32, True, 0.0, mean=6000.0)
    X = torch.full((3, 512), 0.75, device="cuda", dtype=BF16)
    b = torch.randn(512, device="cuda")
    rstd = torch.empty(3, device="cuda")
    y = igc.layer_norm(X, b=b, eps=2.0 ** -20, rstd=rstd)
    check_device_ok()
    assert torch.equal(y, b.bfloat16().expand(3, -1)) and bool((rstd == 1024.0).all())


def test_nan_and_infinities_stay_in_their_rows():
    X = torch.randn(8, 1000, device="cuda")
    good = igc.layer_norm(X)
    bad = X.clone()
    bad[2, 17] = float("nan")
    bad[5, 999] = float("inf")
    y = igc.layer_norm(bad)
    rows = [0, 1, 3, 4, 6, 7]
    check_device_ok()
    assert bool(y[[2, 5]].isnan().all()) and torch.equal(y[rows], good[rows])
    # a dropped NaN is gone
    drop = dict(p=0.5, seed=1)
    gone = ~ref.keep(8, 1000, 0.5, 1, 0).cuda()
    hidden = torch.where(gone, float("nan"), X)
    assert torch.equal(igc.layer_norm(hidden, **drop), igc.layer_norm(X, **drop))
    m, r = torch.zeros(8, device="cuda"), torch.ones(8, device="cuda")
    dS, _, dw, db = igc.layer_norm_backward(bad, X, m, r)
    check_device_ok()
    # with an infinite element both means of its row are infinite: g - inf - h inf is NaN where
    # h < 0 and -inf where h > 0
    assert bool(dS[2].isnan().all()) and bool(dS[rows].isfinite().all())
    assert bool((dS[5].isnan() | (dS[5] == float("-inf"))).all())
    assert int(dw.isnan().sum()) == 1 and int(db.isnan().sum()) == 1 and bool(db[999].isinf())


def test_gradients_against_differences():
    """dS, dX, dw and db against central differences of the fp32 forward pass's 64-bit form."""
    M, N, p, seed = 3, 24, 0.25, 9
    gen = generator(1)
    X, R = (torch.randn(M, N, generator=gen, device="cuda") for _ in range(2))
    w, b = (torch.randn(N, generator=gen, device="cuda") for _ in range(2))
    dY, dSnext = (torch.randn(M, N, generator=gen, device="cuda") for _ in range(2))
    S, m, r = torch.empty_like(X), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    igc.layer_norm(X, w, b, residual=R, p=p, seed=seed, S=S, mean=m, rstd=r)
    dS, dX, dw, db = igc.layer_norm_backward(dY, S, m, r, w, dS_add=dSnext, p=p, seed=seed,
                                             dS=torch.empty_like(X), dX=torch.empty_like(X),
                                             dw=torch.empty_like(w), db=torch.empty_like(b))
    check_device_ok()

    def loss(x, rr, ww, bb):
        s = rr + ref.drop64(x, p, seed, 0)
        zero = torch.zeros_like(s)
        return float((ref.norm64(s, zero, ww, bb, 1e-5)[0] * dY.double()).sum() +
                     (s * dSnext.double()).sum())

    args = [t.double() for t in (X, R, w, b)]
    for k, grad in enumerate((dX, dS, dw, db)):
        for i in range(0, grad.numel(), 5):
            step, vals = 1e-5, []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += sign * step
                vals.append(loss(*moved))
            want = (vals[0] - vals[1]) / (2 * step)
            # third derivatives of a norm of 24 values times step^2, and fp32 values of size ~10
            assert abs(float(grad.view(-1)[i]) - want) <= 2e-5 * (1 + abs(want))


def test_repeatable_streams_and_graphs():
    """The same bits on another stream and from a captured graph, whose step moves the dropout."""
    M, N = 700, 1000
    gen = generator(2)
    X, R, dY = (matrix(gen, M, N, BF16) for _ in range(3))
    w = torch.randn(N, generator=gen, device="cuda")

    def step_of(counter, stream=None):
        S, dX = torch.empty_like(R), torch.empty_like(R)
        Y = torch.empty(M, N, device="cuda", dtype=BF16)
        m, r = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        drop = dict(p=0.2, seed=5, offset=11, step=counter, stream=stream)
        igc.layer_norm(X, w, residual=R, S=S, Y=Y, mean=m, rstd=r, **drop)
        igc.layer_norm_backward(dY, S, m, r, w, dX=dX, dw=dw, db=db, **drop)
        return S, Y, m, r, dX, dw, db

    counter = torch.tensor(4, device="cuda")
    first = step_of(counter)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step_of(counter, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step_of(counter)
        counter.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out)) and int(counter) == 5
    graph.replay()
    torch.cuda.synchronize()
    s, err = ref.dropout64(X, 0.2, 5, 16, R)
    check(out[0], s, rounded(s, BF16, err))
    dx = ref.drop64(torch.ones(M, N), 0.2, 5, 16).cuda()
    assert bool((out[4][dx == 0] == 0).all())
    check_device_ok()


def test_offsets_past_32_bits():
    """Rows that start past 2^31 elements and 2^32 bytes into their matrices."""
    M, N, ld = 9, 64, (1 << 28) + 64
    buf = torch.empty(M * ld, device="cuda", dtype=BF16)
    X = buf.view(M, ld)[:, :N]
    S, dY, A, dX = (buf.view(M, ld)[:, k * N:(k + 1) * N] for k in range(1, 5))
    gen = generator(3)
    vals = torch.randn(3, M, N, generator=gen, device="cuda").bfloat16()
    X.copy_(vals[0])
    dY.copy_(vals[1])
    A.copy_(vals[2])
    m, r = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    y = igc.layer_norm(X, p=0.1, seed=1, S=S, mean=m, rstd=r)
    dS, dXs, Ss = (torch.empty(M, N, device="cuda", dtype=BF16) for _ in range(3))
    y2 = igc.layer_norm(vals[0], p=0.1, seed=1, S=Ss)
    assert torch.equal(y, y2) and torch.equal(S, Ss)
    igc.layer_norm_backward(vals[1], Ss, m, r, dS_add=vals[2], p=0.1, seed=1, dS=dS, dX=dXs)
    igc.layer_norm_backward(dY, S, m, r, dS_add=A, p=0.1, seed=1, dS=A, dX=dX)
    check_device_ok()
    assert torch.equal(A, dS) and torch.equal(dX, dXs)
