"""Host-side checks of embedding, layer norm and dropout that need no GPU: declared and exported
entry points, refusals of the C entries before any device call, refusals of the binding,
workspace sizes, the reference form's generator."""

import ctypes

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref

INVALID, MISALIGNED, WORKSPACE, UNSUPPORTED, OK = (
    igc.IGC_ERR_INVALID_ARG, igc.IGC_ERR_MISALIGNED, igc.IGC_ERR_WORKSPACE,
    igc.IGC_ERR_UNSUPPORTED, igc.IGC_OK)
F32, F16, BF16 = igc.IGC_F32, igc.IGC_F16, igc.IGC_BF16
A, B, C, D, E, F, G, H, K, L = (ctypes.c_void_p(1 << s) for s in range(16, 26))
ODD = ctypes.c_void_p((1 << 26) + 1)
HALF = ctypes.c_void_p((1 << 26) + 2)       # a boundary of 16-bit elements alone
NAN = float("nan")
BIG = 0x7fffff00


def test_header_declares_the_operators_and_the_library_exports_them():
    names = {"dropout_add", "layer_norm", "layer_norm_backward",
             "layer_norm_backward_workspace_size", "embedding_lookup", "embedding_backward",
             "embedding_backward_workspace_size"}
    found = set(igc.declared_functions(igc.LAYERS_HEADER))
    assert found == names
    for n in names:
        assert ctypes.cast(getattr(igc.lib(), n), ctypes.c_void_p).value
        assert callable(getattr(igc, n))


def dropout(M=4, N=8, X=A, ldx=8, xt=BF16, R=B, ldr=8, p=0.1, seed=1, offset=0, step=None, Y=C,
            ldy=8, yt=BF16):
    return igc.lib().dropout_add(M, N, X, ldx, xt, R, ldr, p, seed, offset, step, Y, ldy, yt, None)


def test_dropout_refusals():
    for bad in (dict(M=-1), dict(N=-1), dict(xt=3), dict(yt=-1), dict(yt=F16), dict(xt=F16),
                dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(X=None), dict(Y=None), dict(ldx=7),
                dict(ldr=7), dict(ldy=7), dict(step=C), dict(Y=A, ldy=9), dict(Y=A, xt=F32),
                dict(Y=B, ldy=9)):
        assert dropout(**bad) == INVALID, bad
    for bad in (dict(X=ODD), dict(R=ODD), dict(Y=ODD), dict(X=HALF, xt=F32), dict(step=HALF),
                dict(R=HALF, yt=F32), dict(Y=HALF, yt=F32)):
        assert dropout(**bad) == MISALIGNED, bad
    assert dropout(M=1 << 31) == UNSUPPORTED
    assert dropout(N=1 << 31, ldx=1 << 31, ldr=1 << 31, ldy=1 << 31) == UNSUPPORTED
    assert dropout(M=0, X=None, Y=None) == OK and dropout(N=0, X=None, Y=None) == OK


def norm(M=4, N=8, dt=BF16, X=A, ldx=8, R=B, ldr=8, st=BF16, p=0.0, seed=1, offset=0, step=None,
         w=C, b=D, wt=F32, eps=1e-5, S=E, lds=8, Y=F, ldy=8, mean=G, rstd=H):
    return igc.lib().layer_norm(M, N, dt, X, ldx, R, ldr, st, p, seed, offset, step, w, b, wt, eps,
                                S, lds, Y, ldy, mean, rstd, None)


def test_layer_norm_refusals():
    for bad in (dict(M=-1), dict(N=-1), dict(N=0), dict(dt=3), dict(st=F16), dict(wt=F16),
                dict(dt=F32), dict(p=-1e-9), dict(p=2.0), dict(p=NAN), dict(eps=-1.0),
                dict(eps=NAN), dict(X=None, R=None), dict(Y=None), dict(ldx=7), dict(ldr=7),
                dict(lds=7), dict(ldy=7)):
        assert norm(**bad) == INVALID, bad
    # an output that is an input or another output; a residual in place of another stride
    for bad in (dict(Y=A), dict(Y=B), dict(Y=E), dict(Y=C), dict(Y=D), dict(Y=G), dict(Y=H),
                dict(S=A), dict(S=C), dict(S=D), dict(S=G), dict(S=H), dict(S=B, lds=9),
                dict(mean=H), dict(mean=A), dict(mean=B), dict(mean=C), dict(rstd=A), dict(rstd=B),
                dict(rstd=D), dict(p=0.1, step=F), dict(p=0.1, step=E), dict(p=0.1, step=G),
                dict(p=0.1, step=H)):
        assert norm(**bad) == INVALID, bad
    for name in ("X", "R", "S", "Y", "w", "b", "mean", "rstd", "step"):
        assert norm(**{name: ODD}) == MISALIGNED, name
    for bad in (dict(R=HALF, st=F32), dict(S=HALF, st=F32), dict(w=HALF), dict(mean=HALF)):
        assert norm(**bad) == MISALIGNED, bad
    assert norm(M=1 << 31) == UNSUPPORTED
    assert norm(M=0, X=None, R=None, Y=None) == OK


def norm_bwd(M=4, N=8, dt=BF16, dY=A, lddy=8, S=B, lds=8, st=BF16, mean=C, rstd=D, w=E, wt=F32,
             add=F, lda=8, p=0.0, seed=1, offset=0, step=None, dS=G, ldds=8, dX=H, lddx=8, dw=K,
             db=L, dwt=F32, ws=None, n=0):
    return igc.lib().layer_norm_backward(M, N, dt, dY, lddy, S, lds, st, mean, rstd, w, wt, add,
                                         lda, p, seed, offset, step, dS, ldds, dX, lddx, dw, db,
                                         dwt, ws, n, None)


def test_layer_norm_backward_refusals():
    for bad in (dict(M=-1), dict(N=0), dict(dt=3), dict(st=F16), dict(wt=F16), dict(dwt=F16),
                dict(p=-0.1), dict(p=NAN), dict(dY=None), dict(S=None), dict(mean=None),
                dict(rstd=None), dict(lddy=7), dict(lds=7), dict(lda=7), dict(ldds=7),
                dict(lddx=7)):
        assert norm_bwd(**bad) == INVALID, bad
    for out in ("dS", "dX", "dw", "db"):
        for other in (A, B, C, D, E):
            assert norm_bwd(**{out: other}) == INVALID, (out, other)
    for bad in (dict(dS=F, ldds=9), dict(dX=F), dict(dw=F), dict(db=F), dict(dX=G), dict(dw=G),
                dict(db=G), dict(dw=H), dict(db=H), dict(db=K), dict(step=G), dict(step=L)):
        assert norm_bwd(**bad) == INVALID, bad
    for name in ("dY", "S", "mean", "rstd", "w", "add", "dS", "dX", "dw", "db", "step"):
        assert norm_bwd(**{name: ODD}) == MISALIGNED, name
    assert norm_bwd(M=1 << 31) == UNSUPPORTED
    # nothing asked for
    assert norm_bwd(dS=None, dX=None, dw=None, db=None, dY=None) == OK


def lookup(M=4, V=10, N=8, tokens=A, size=8, W=B, ldw=8, wt=BF16, scale=1.0, Y=C, ldy=8, yt=BF16):
    return igc.lib().embedding_lookup(M, V, N, tokens, size, W, ldw, wt, scale, Y, ldy, yt, None)


def test_embedding_lookup_refusals():
    for bad in (dict(M=-1), dict(V=-1), dict(N=-1), dict(size=2), dict(wt=3), dict(yt=F16),
                dict(tokens=None), dict(W=None), dict(Y=None), dict(ldw=7), dict(ldy=7),
                dict(Y=A), dict(Y=B)):
        assert lookup(**bad) == INVALID, bad
    for bad in (dict(W=ODD), dict(Y=ODD), dict(Y=HALF, yt=F32), dict(tokens=HALF),
                dict(tokens=ctypes.c_void_p(68), size=8)):
        assert lookup(**bad) == MISALIGNED, bad
    for bad in (dict(M=1 << 31), dict(V=1 << 31), dict(N=1 << 31, ldw=1 << 31, ldy=1 << 31)):
        assert lookup(**bad) == UNSUPPORTED, bad
    assert lookup(M=0, Y=None) == OK and lookup(N=0, Y=None) == OK


def lookup_bwd(M=4, V=10, N=8, tokens=A, size=8, dY=B, lddy=8, yt=BF16, scale=1.0, acc=0, dW=C,
               lddw=8, wt=BF16, ws=None, n=0):
    return igc.lib().embedding_backward(M, V, N, tokens, size, dY, lddy, yt, scale, acc, dW, lddw,
                                        wt, ws, n, None)


def test_embedding_backward_refusals():
    for bad in (dict(M=-1), dict(V=-1), dict(N=-1), dict(size=1), dict(yt=3), dict(wt=F16),
                dict(tokens=None), dict(dY=None), dict(dW=None), dict(lddy=7), dict(lddw=7),
                dict(dW=A), dict(dW=B)):
        assert lookup_bwd(**bad) == INVALID, bad
    for bad in (dict(dY=ODD), dict(dW=ODD), dict(dW=HALF, wt=F32), dict(tokens=HALF)):
        assert lookup_bwd(**bad) == MISALIGNED, bad
    for bad in (dict(M=1 << 31), dict(V=1 << 31), dict(N=1 << 31, lddy=1 << 31, lddw=1 << 31)):
        assert lookup_bwd(**bad) == UNSUPPORTED, bad
    assert lookup_bwd(V=0, dW=None) == OK and lookup_bwd(N=0, dW=None) == OK
    assert lookup_bwd(M=0, acc=1, dW=None) == OK


def test_workspace_sizes():
    size = igc.layer_norm_backward_workspace_size
    assert size(-1, 8) == 0 and size(8, -1) == 0 and size(0, 100) == 0
    # two rows of fp32 sums (dw and db) for each row of the input at most
    assert size(3, 100) == 2 * 3 * 100 * 4
    assert 0 < size(1 << 20, 4096) <= 2 * 512 * 4096 * 4
    size = igc.embedding_backward_workspace_size
    assert size(-1, 8, 8) == 0 and size(8, -1, 8) == 0 and size(8, 8, -1) == 0
    assert size(1, 100000, 4096) == 0 and size(5000, 0, 8) == 0 and size(5000, 8, 0) == 0
    # tokens and positions twice, a byte for each row of the table, the counts of 512 digits in 64
    # blocks, two rows of fp32 sums for 32 positions
    most = 4 * 4 * 8192 + 100000 + 64 * 512 * 4 + 2 * 256 * 64 * 4 + 8 * 256
    assert 4 * 4 * 8192 < size(8192, 100000, 64) <= most


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    X, v = t(4, 16), t(16, dtype=torch.float32)
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        igc.dropout_add(X, 0.1, seed=1)
    for p in (-0.1, 1.5, NAN):
        with pytest.raises(ValueError, match="a probability"):
            igc.dropout_add(X, p, seed=1)
        with pytest.raises(ValueError, match="a probability"):
            igc.layer_norm(X, p=p, seed=1)
    with pytest.raises(ValueError, match="seed is needed"):
        igc.dropout_add(X, 0.1)
    with pytest.raises(ValueError, match="seed is needed"):
        igc.layer_norm(X, p=0.1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1)):
        with pytest.raises(ValueError, match="seed and offset"):
            igc.dropout_add(X, 0.1, **kw)
    with pytest.raises(ValueError, match="step must be"):
        igc.dropout_add(X, 0.1, seed=1, step=t(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="X has dtype"):
        igc.dropout_add(X.double(), 0.1, seed=1)
    with pytest.raises(TypeError, match="the output"):
        igc.dropout_add(X, 0.1, seed=1, residual=X.half())
    with pytest.raises(TypeError, match="residual has dtype"):
        igc.dropout_add(X, 0.1, seed=1, residual=X, Y=X.float())
    with pytest.raises(ValueError, match="residual has shape"):
        igc.dropout_add(X, 0.1, seed=1, residual=t(4, 8))
    with pytest.raises(ValueError, match="Y must be row-major"):
        igc.dropout_add(X, 0.1, seed=1, Y=t(16, 4).t())
    with pytest.raises(ValueError, match="Y must be row-major"):
        igc.dropout_add(X, 0.1, seed=1, Y=t(1, 16).expand(4, 16))
    with pytest.raises(ValueError, match="X must be a matrix"):
        igc.layer_norm(t(2, 4, 16))
    with pytest.raises(ValueError, match="w must be"):
        igc.layer_norm(X, v[:8])
    with pytest.raises(ValueError, match="one type"):
        igc.layer_norm(X, v, t(16))
    with pytest.raises(TypeError, match="residual has dtype"):
        igc.layer_norm(X, residual=X.half())
    with pytest.raises(TypeError, match="X has dtype"):
        igc.layer_norm(X, residual=X.float(), Y=X.half())
    with pytest.raises(TypeError, match="S has dtype"):
        igc.layer_norm(X, residual=X.float(), S=X)
    with pytest.raises(ValueError, match="mean must be"):
        igc.layer_norm(X, mean=v)
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        igc.layer_norm(X)
    m = v[:4].contiguous()
    with pytest.raises(ValueError, match="mean and rstd are needed"):
        igc.layer_norm_backward(X, X, m, None)
    with pytest.raises(TypeError, match="dS_add has dtype"):
        igc.layer_norm_backward(X, X.float(), m, m, dS_add=X, dS=X.float())
    with pytest.raises(TypeError, match="dX has dtype"):
        igc.layer_norm_backward(X, X.float(), m, m, dX=X.float())
    with pytest.raises(ValueError, match="dw and db must have one type"):
        igc.layer_norm_backward(X, X, m, m, dw=v, db=t(16))
    with pytest.raises(ValueError, match="dY must be a CUDA tensor"):
        igc.layer_norm_backward(X, X, m, m, dX=X)
    tok = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="tokens has dtype"):
        igc.embedding_lookup(tok.short(), X)
    with pytest.raises(ValueError, match="contiguous vector"):
        igc.embedding_lookup(tok.view(2, 2), X)
    with pytest.raises(ValueError, match="contiguous vector"):
        igc.embedding_lookup(torch.zeros(8, dtype=torch.int64)[::2], X)
    with pytest.raises(TypeError, match="Y has dtype"):
        igc.embedding_lookup(tok, X, Y=X.half())
    with pytest.raises(ValueError, match="W must be a CUDA tensor"):
        igc.embedding_lookup(tok, X)
    with pytest.raises(ValueError, match="tokens has 4 elements, dY 3 rows"):
        igc.embedding_backward(tok, X[:3], V=9)
    with pytest.raises(ValueError, match="V, the rows of dW"):
        igc.embedding_backward(tok, X)
    with pytest.raises(ValueError, match="dW is needed"):
        igc.embedding_backward(tok, X, V=9, accumulate=True)
    with pytest.raises(ValueError, match="dW has 5 rows"):
        igc.embedding_backward(tok, X, V=9, dW=t(5, 16))
    with pytest.raises(TypeError, match="dW has dtype"):
        igc.embedding_backward(tok, X, dW=t(5, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="dY must be a CUDA tensor"):
        igc.embedding_backward(tok, X, V=9)


def test_known_answers_of_the_reference_generator():
    """Philox4x32-10's published answers for all zeros and all ones."""
    got = ref.philox((0, 0, 0, 0), (0, 0))
    assert [int(v) for v in got] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = [0xFFFFFFFF] * 4
    got = ref.philox(ones, ones[:2])
    assert [int(v) for v in got] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
