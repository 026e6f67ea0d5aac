"""linear_act and linear_act_backward against their 64-bit forms."""

import pytest
import torch

import ffn_reference as ref
import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def matrix(gen, rows, cols, dtype, scale=1.0, pad=0, fill=float("nan")):
    """rows x cols of N(0, scale^2) in a buffer whose rows are padded to a multiple of 8
    elements and by `pad` more; the padding holds `fill`."""
    buf = torch.full((max(rows, 1), -(-max(cols, 1) // 8) * 8 + pad), fill, device="cuda",
                     dtype=dtype)
    t = buf[:rows, :cols]
    t.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
    return t


def generator(*key):
    return torch.Generator(device="cuda").manual_seed(abs(hash(key)) % (1 << 31))


@pytest.fixture(params=[0, 128, 256], ids=["auto", "tiles128", "tiles256"])
def width(request):
    """The schedule chosen per problem, and the 256-row tiles of either width forced."""
    igc.igc_set_tile_width(request.param)
    yield request.param
    igc.igc_set_tile_width(0)


def d(t):
    return None if t is None else t.double()


def make(M, N, K, dtype, bias, residual, seed, pad=0):
    gen = generator(M, N, K, seed)
    x = matrix(gen, M, K, dtype, pad=pad)
    w = matrix(gen, N, K, dtype, K ** -0.5 if K else 1.0, pad=pad)
    b = matrix(gen, 1, N, dtype)[0].clone() if bias else None
    r = matrix(gen, M, N, dtype, pad=pad) if residual else None
    return x, w, b, r


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 777), (2, 5, 8), (3, 129, 200), (15, 128, 1024),
          (16, 64, 4096), (17, 300, 72), (64, 640, 520), (127, 257, 130), (128, 384, 2048),
          (129, 300, 72), (200, 1, 64), (256, 256, 256), (257, 513, 1000), (333, 1000, 2056),
          (640, 2304, 192), (1, 20000, 64), (5, 256, 16384),
          (2000, 1300, 200), (1800, 1501, 264)]   # the last two take 192-wide tiles


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_shapes(M, N, K, dtype, width):
    i = SHAPES.index((M, N, K))
    name = ref.ACTS[i % 5]
    x, w, b, r = make(M, N, K, dtype, i % 2 == 0, i % 3 != 0, i, pad=8 * (i % 2))
    Y = torch.full((M, N), 7.0, device="cuda", dtype=dtype)
    Z = torch.full((M, N), 7.0, device="cuda", dtype=dtype)
    assert igc.linear_act(x, w, bias=b, act=name, residual=r, Y=Y, Z=Z) is Y
    check_device_ok()
    want_y, want_z = ref.linear(d(x), d(w), d(b), name, d(r), dtype, dtype)
    ref.check(Z, want_z, "Z")
    ref.check(Y, want_y, "Y")


@pytest.mark.parametrize("M", [7, 300])
@pytest.mark.parametrize("name", ref.ACTS)
def test_forward_activations_and_types(M, name, width):
    N, K = 200, 192
    for dtype in (BF16, F16):
        for out, bt in ((dtype, F32), (F32, dtype), (F32, F32)):
            x, w, b, r = make(M, N, K, dtype, True, True, 3)
            x = x * 4  # pre-activations out to where the activations are flat
            Y = torch.empty((M, N), device="cuda", dtype=out)
            igc.linear_act(x, w, bias=b.to(bt), act=name, residual=r, Y=Y)
            check_device_ok()
            want, _ = ref.linear(d(x), d(w), d(b), name, d(r), out, dtype)
            ref.check(Y, want, f"{name} {dtype} -> {out}")


@pytest.mark.parametrize("M", [4, 300])
def test_forward_unaligned_outputs_and_guard_columns(M, width):
    """Outputs at any alignment; nothing outside them is written."""
    N, K = 131, 96
    x, w, b, r = make(M, N, K, BF16, True, False, 5)
    rbuf = torch.randn((M, N + 6), device="cuda").to(BF16)
    r = rbuf[:, 3:3 + N]
    for out in (BF16, F32):
        ybuf = torch.full((M + 2, N + 5), 9.0, device="cuda", dtype=out)
        zbuf = torch.full((M + 2, N + 5), 9.0, device="cuda", dtype=BF16)
        Y, Z = ybuf[1:M + 1, 1:N + 1], zbuf[1:M + 1, 3:N + 3]
        igc.linear_act(x, w, bias=b, act="gelu", residual=r, Y=Y, Z=Z)
        check_device_ok()
        want_y, want_z = ref.linear(d(x), d(w), d(b), "gelu", d(r), out, BF16)
        ref.check(Y, want_y, "Y")
        ref.check(Z, want_z, "Z")
        for buf, lo in ((ybuf, 1), (zbuf, 3)):
            keep = torch.ones_like(buf, dtype=torch.bool)
            keep[1:M + 1, lo:lo + N] = False
            assert bool((buf[keep] == 9.0).all())


@pytest.mark.parametrize("M", [1, 20, 400])
def test_forward_residual_in_place(M, width):
    x, w, b, r = make(M, 520, 264, BF16, True, True, 6)
    want, _ = ref.linear(d(x), d(w), d(b), "none", d(r), BF16, BF16)
    igc.linear_act(x, w, bias=b, residual=r, Y=r)
    check_device_ok()
    ref.check(r, want, "Y over its residual")


@pytest.mark.parametrize("M", [3, 300])
def test_forward_nan_and_infinity_stay_in_their_rows(M, width):
    x, w, _, _ = make(M, 96, 128, F16, False, False, 7)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    Y = igc.linear_act(x, w)
    check_device_ok()
    assert bool(Y[1].isnan().all())
    assert not bool(Y[2].isfinite().any())
    rest = [i for i in range(M) if i not in (1, 2)]
    want, _ = ref.linear(d(x[rest]), d(w), None, "none", None, F16, F16)
    ref.check(Y[rest], want, "other rows")


@pytest.mark.parametrize("M", [2, 200])
def test_forward_empty(M):
    """An empty contraction leaves the bias; an empty output is a no-op."""
    N = 37
    b = torch.randn(N, device="cuda")
    r = torch.randn((M, N), device="cuda").to(F16)
    e = torch.empty((M, 0), device="cuda", dtype=F16)
    Z = torch.empty((M, N), device="cuda", dtype=F16)
    Y = igc.linear_act(e, e[:1].expand(N, 0).contiguous(), bias=b, act="silu", residual=r, Z=Z)
    check_device_ok()
    z = d(b).expand(M, N)
    y = ref.act("silu", z) + d(r)
    ref.check(Z, (z, ref.rounded(z, 0 * z, F16)), "Z")
    ref.check(Y, (y, ref.rounded(y, 1e-5 * z.abs() + 2.0 ** -23 * y.abs(), F16)), "Y")
    x = torch.randn((M, 64), device="cuda").to(F16)
    assert igc.linear_act(x[:0], x).shape == (0, M)
    assert igc.linear_act(x, x[:0]).shape == (M, 0)


@pytest.mark.parametrize("M,N", [(5, 40), (300, 300)])
def test_forward_offsets_past_32_bits(M, N, width):
    """Rows of every matrix lie further apart than 2^31 bytes allow in all."""
    gen = generator(M, N, 8)
    stride = (1 << 31) // M + 1024 - ((1 << 31) // M) % 8   # M rows pass 2^31 elements
    K = 72
    buf = torch.empty(stride * M, device="cuda", dtype=BF16)
    view = buf.view(M, stride)
    x, Y, Z, r = (view[:, o:o + n] for o, n in ((0, K), (512, N), (1024, N), (1536, N)))
    x.copy_(torch.randn((M, K), generator=gen, device="cuda"))
    r.copy_(torch.randn((M, N), generator=gen, device="cuda"))
    w = matrix(gen, N, K, BF16, K ** -0.5)
    igc.linear_act(x, w, act="gelu_tanh", residual=r, Y=Y, Z=Z)
    check_device_ok()
    want_y, want_z = ref.linear(d(x), d(w), None, "gelu_tanh", d(r), BF16, BF16)
    ref.check(Y, want_y, "Y")
    ref.check(Z, want_z, "Z")


@pytest.mark.parametrize("M,N,K", [(9, 1000, 4096), (400, 500, 1100)])
def test_forward_is_repeatable_and_runs_on_other_streams_and_in_graphs(M, N, K):
    x, w, b, r = make(M, N, K, BF16, True, True, 9)
    first = igc.linear_act(x, w, bias=b, act="silu", residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = igc.linear_act(x, w, bias=b, act="silu", residual=r, stream=side)
    raw = igc.linear_act(x, w, bias=b, act="silu", residual=r, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, raw)
    Y = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        igc.linear_act(x, w, bias=b, act="silu", residual=r, Y=Y)
    for _ in range(2):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, Y)
    x2 = x.clone()
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = ref.linear(2 * d(x2), d(w), d(b), "silu", d(r), BF16, BF16)
    ref.check(Y, want, "replay on new inputs")
    check_device_ok()


# ------------------------------------------------------------------------------ gradients

BWD_SHAPES = [(1, 1, 1), (1, 64, 64), (2, 5, 8), (7, 300, 40), (100, 129, 200), (129, 64, 520),
              (300, 257, 300), (509, 1001, 777), (640, 256, 1030), (2000, 72, 96), (33, 2048, 2300)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", BWD_SHAPES)
def test_backward_shapes(M, N, K, dtype, width):
    i = BWD_SHAPES.index((M, N, K))
    name = ref.ACTS[i % 5]
    gen = generator(M, N, K, 20)
    x = matrix(gen, M, K, dtype, pad=8 * (i % 2))
    w = matrix(gen, N, K, dtype, K ** -0.5)
    # the pre-activation and the incoming gradient may have any alignment
    dy = matrix(gen, M, N, dtype, 0.5, pad=i % 3)
    z = matrix(gen, M, N, dtype, 2.0, pad=i % 2)
    dX = torch.full((M, K), 7.0, device="cuda", dtype=dtype)
    dW = torch.full((N, K), 7.0, device="cuda", dtype=dtype if i % 2 else F32)
    db = torch.full((N,), 7.0, device="cuda", dtype=F32 if i % 2 else dtype)
    got = igc.linear_act_backward(dy, x, w, act=name, Z=z, dX=dX, dW=dW, dbias=db)
    assert got[0] is dX and got[1] is dW and got[2] is db
    check_device_ok()
    dz, ez = ref.linear_dz(d(dy), d(z), name)
    wx, ww, wb = ref.grads([dz], [ez], d(x), [d(w)], dtype, dW.dtype, db.dtype)
    ref.check(dX, wx[0], "dX")
    ref.check(dW, ww[0], "dW")
    ref.check(db, wb[0], "db")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_backward_small_integers_bit_exact(dtype):
    """Every product and sum is a small integer: any wrong element shows."""
    gen = generator(21)
    M, N, K = 384, 520, 328

    def ints(r, c):
        return torch.randint(-2, 3, (r, c), generator=gen, device="cuda").to(dtype)

    x, w, dy = ints(M, K), ints(N, K), ints(M, N)
    for width in (0, 128, 256):
        dX = torch.empty((M, K), device="cuda", dtype=dtype)
        dW = torch.empty((N, K), device="cuda", dtype=F32)
        db = torch.empty(N, device="cuda")
        igc.igc_set_tile_width(width)
        try:
            igc.linear_act_backward(dy, x, w, dX=dX, dW=dW, dbias=db)
        finally:
            igc.igc_set_tile_width(0)
        check_device_ok()
        assert torch.equal(dX, (d(dy) @ d(w)).to(dtype))
        assert torch.equal(dW.double(), d(dy).t() @ d(x))
        assert torch.equal(db.double(), d(dy).sum(0))


def test_backward_each_gradient_alone():
    gen = generator(22)
    M, N, K = 150, 131, 200
    x, w = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, 0.1)
    z = torch.randn((M, N), generator=gen, device="cuda").to(BF16)
    dy = torch.randn((M, N), generator=gen, device="cuda").to(BF16)   # rows not 16-byte aligned
    for name in ("none", "gelu"):
        dz, ez = ref.linear_dz(d(dy), d(z), name)
        wx, ww, wb = ref.grads([dz], [ez], d(x), [d(w)], BF16, BF16, F32)
        dX = torch.empty((M, K), device="cuda", dtype=BF16)
        assert igc.linear_act_backward(dy, None, w, act=name, Z=z, dX=dX)[1:] == (None, None)
        dW = torch.empty((N, K), device="cuda", dtype=BF16)
        igc.linear_act_backward(dy, x, None, act=name, Z=z, dW=dW)
        db = torch.empty(N, device="cuda")
        igc.linear_act_backward(dy, None, None, act=name, Z=z, dbias=db)
        aX, aW, none = igc.linear_act_backward(dy, x, w, act=name, Z=z)
        check_device_ok()
        ref.check(dX, wx[0], "dX")
        ref.check(dW, ww[0], "dW")
        ref.check(db, wb[0], "db")
        assert none is None and torch.equal(aX, dX) and torch.equal(aW, dW)


def test_backward_empty():
    x = torch.randn((0, 40), device="cuda").to(F16)
    w = torch.randn((24, 40), device="cuda").to(F16)
    dy = torch.randn((0, 24), device="cuda").to(F16)
    dW = torch.full((24, 40), 5.0, device="cuda")
    db = torch.full((24,), 5.0, device="cuda")
    igc.linear_act_backward(dy, x, w, dW=dW, dbias=db)      # no rows: zero gradients
    x5 = torch.randn((5, 40), device="cuda").to(F16)
    dX = torch.full((5, 40), 5.0, device="cuda", dtype=F16)
    igc.linear_act_backward(x5[:, :0], None, w[:0], dX=dX)  # no outputs: zero gradient
    check_device_ok()
    assert not bool(dW.any()) and not bool(db.any()) and not bool(dX.any())


@pytest.mark.parametrize("name", ref.ACTS)
def test_backward_against_differences(name):
    """The gradients' inner product with a direction equals the central difference of
    sum(C * Y) along it, Y in 64 bits."""
    gen = generator(23)
    M, N, K = 60, 72, 96
    x, w = matrix(gen, M, K, F16), matrix(gen, N, K, F16, K ** -0.5)
    c = matrix(gen, M, N, F16)
    b = torch.randn(N, generator=gen, device="cuda").to(F16)
    Z = torch.empty((M, N), device="cuda", dtype=F16)
    igc.linear_act(x, w, bias=b, act=name, Z=Z)
    dX = torch.empty((M, K), device="cuda", dtype=F16)
    dW = torch.empty((N, K), device="cuda")
    db = torch.empty(N, device="cuda")
    igc.linear_act_backward(c, x, w, act=name, Z=Z, dX=dX, dW=dW, dbias=db)
    check_device_ok()

    def loss(px, pw, pb):
        return float((d(c) * ref.act(name, px @ pw.t() + pb)).sum())

    for at, grad in enumerate((dX, dW, db)):
        base = [d(x), d(w), d(b)]
        step = torch.randn(base[at].shape, generator=gen, device="cuda").double()
        h = 1e-6
        hi, lo = list(base), list(base)
        hi[at] = base[at] + h * step
        lo[at] = base[at] - h * step
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        got = float((grad.double() * step).sum())
        # Z and dZ are rounded to fp16 (2^-11 each; slopes' slopes are at most 1.6) and the
        # result too: a random walk of the terms, held to 40 u of the terms' 2-norm
        terms = (grad.double() * step).square().sum().sqrt()
        dz, _ = ref.linear_dz(d(c), d(Z), name)
        spread = dz.abs().max() * base[at].numel() ** 0.5
        assert abs(got - want) <= 40 * 2.0 ** -11 * float(terms + spread), (at, got, want)


def test_backward_is_repeatable_on_a_side_stream():
    gen = generator(24)
    M, N, K = 700, 400, 300
    x, w = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, 0.1)
    z, dy = matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)
    db = [torch.empty(N, device="cuda") for _ in range(2)]
    outs = [torch.empty((M, K), device="cuda", dtype=BF16) for _ in range(2)]
    igc.linear_act_backward(dy, x, w, act="silu", Z=z, dX=outs[0], dbias=db[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    igc.linear_act_backward(dy, x, w, act="silu", Z=z, dX=outs[1], dbias=db[1], stream=side)
    torch.cuda.synchronize()
    check_device_ok()
    assert torch.equal(outs[0], outs[1]) and torch.equal(db[0], db[1])


def test_backward_offsets_past_32_bits():
    """Every matrix's rows lie further apart than 2^31 elements allow in all."""
    gen = generator(25)
    M, N, K = 6, 40, 72
    stride = (1 << 31) // M + 1024 - ((1 << 31) // M) % 8
    view = torch.empty(stride * M, device="cuda", dtype=BF16).view(M, stride)
    dy, z, x, dX = (view[:, o:o + n] for o, n in ((0, N), (512, N), (1024, K), (1536, K)))
    for t, n in ((dy, N), (z, N), (x, K)):
        t.copy_(torch.randn((M, n), generator=gen, device="cuda"))
    w = matrix(gen, N, K, BF16, K ** -0.5)
    dW = torch.empty((N, K), device="cuda")
    db = torch.empty(N, device="cuda")
    igc.linear_act_backward(dy, x, w, act="gelu", Z=z, dX=dX, dW=dW, dbias=db)
    check_device_ok()
    dz, ez = ref.linear_dz(d(dy), d(z), "gelu")
    wx, ww, wb = ref.grads([dz], [ez], d(x), [d(w)], BF16, F32, F32)
    ref.check(dX, wx[0], "dX")
    ref.check(dW, ww[0], "dW")
    ref.check(db, wb[0], "db")


@pytest.mark.parametrize("own_streams", [False, True])
def test_backward_from_threads(own_streams):
    """Calls of several host threads interleave on one stream, or run on streams of their
    own; each thread has its own workspace."""
    import threading
    gen = generator(26)
    shapes = [(300, 200, 136), (70, 520, 264), (600, 72, 328), (128, 300, 200)]
    cases, results = [], {}
    for M, N, K in shapes:
        x, w = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, K ** -0.5)
        dy, z = matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)
        alone = igc.linear_act_backward(dy, x, w, act="silu", Z=z)[:2]
        cases.append((x, w, dy, z, [t.clone() for t in alone]))
    torch.cuda.synchronize()

    def work(i):
        x, w, dy, z, _ = cases[i]
        stream = torch.cuda.Stream() if own_streams else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            results[i] = [igc.linear_act_backward(dy, x, w, act="silu", Z=z)[:2]
                          for _ in range(30)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    check_device_ok()
    for i, case in enumerate(cases):
        for dX, dW in results[i]:
            assert torch.equal(dX, case[4][0]) and torch.equal(dW, case[4][1])


def test_backward_replays_in_a_graph_beside_eager_calls():
    """A captured call keeps its own workspace: eager calls in between, larger ones among
    them, do not disturb its replays."""
    gen = generator(27)
    M, N, K = 200, 136, 264
    x, w = matrix(gen, M, K, F16), matrix(gen, N, K, F16, K ** -0.5)
    dy, z = matrix(gen, M, N, F16), matrix(gen, M, N, F16)
    dX, dW = (torch.empty(s, device="cuda", dtype=F16) for s in ((M, K), (N, K)))
    db = torch.empty(N, device="cuda")
    igc.linear_act_backward(dy, x, w, act="gelu", Z=z, dX=dX, dW=dW, dbias=db)
    want = [t.clone() for t in (dX, dW, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        igc.linear_act_backward(dy, x, w, act="gelu", Z=z, dX=dX, dW=dW, dbias=db)
    big = [matrix(gen, 900, n, F16) for n in (700, 520)]
    wbig = matrix(gen, 700, 520, F16, 0.05)
    for _ in range(3):
        for t in (dX, dW, db):
            t.zero_()
        igc.linear_act_backward(big[0], big[1], wbig, act="gelu", Z=big[0])
        graph.replay()
        igc.linear_act_backward(big[0], big[1], wbig, act="gelu", Z=big[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dX, dW, db), want))
    check_device_ok()


@pytest.mark.parametrize("M", [3, 300])
def test_forward_overflow_is_infinite(M):
    x = torch.full((M, 64), 200.0, device="cuda", dtype=F16)
    w = torch.full((40, 64), 200.0, device="cuda", dtype=F16)
    Y = torch.empty((M, 40), device="cuda", dtype=F32)
    Z = torch.empty((M, 40), device="cuda", dtype=F16)
    igc.linear_act(x, w, Y=Y, Z=Z)
    check_device_ok()
    assert bool((Y == 64 * 40000.0).all()) and bool(torch.isposinf(Z).all())


def padded_out(rows, cols, dtype):
    """An output whose rows are padded to 16 bytes and a little more, and the buffer."""
    buf = torch.full((rows, -(-cols // 8) * 8 + 8), 9.0, device="cuda", dtype=dtype)
    return buf[:, :cols], buf


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("n", [1, 3, 67, 129, 130, 133, 260])
def test_padding_of_outputs_is_kept(M, n, width):
    """Outputs with 16-byte aligned rows whose last columns do not fill 16 bytes: nothing
    past them is written, in either direction's outputs."""
    for dtype in (BF16, F32):
        x, w, b, _ = make(M, n, 96, BF16, True, False, 30)
        (Y, yb), (Z, zb) = padded_out(M, n, dtype), padded_out(M, n, BF16)
        igc.linear_act(x, w, bias=b, act="silu", Y=Y, Z=Z)
        gen = generator(M, n, 31)
        x2, w2 = matrix(gen, M, n, BF16), matrix(gen, 72, n, BF16)
        dy = matrix(gen, M, 72, BF16)
        (dX, xb), (dW, wb) = padded_out(M, n, BF16), padded_out(72, n, dtype)
        igc.linear_act_backward(dy, x2, w2, dX=dX, dW=dW)
        check_device_ok()
        want_y, want_z = ref.linear(d(x), d(w), d(b), "silu", None, dtype, BF16)
        wx, ww, _ = ref.grads([d(dy)], [0 * d(dy)], d(x2), [d(w2)], BF16, dtype, F32)
        for got, want, buf, what in ((Y, want_y, yb, "Y"), (Z, want_z, zb, "Z"),
                                     (dX, wx[0], xb, "dX"), (dW, ww[0], wb, "dW")):
            ref.check(got, want, what)
            assert bool((buf[:, n:] == 9.0).all()), what
