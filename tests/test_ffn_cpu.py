"""Host-side checks of the feed-forward operators that need no GPU: declared and exported
entry points, refusals of the C entries before any device call, refusals of the binding,
workspace sizes."""

import ctypes

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc

INVALID, MISALIGNED, WORKSPACE, OK = (igc.IGC_ERR_INVALID_ARG, igc.IGC_ERR_MISALIGNED,
                                      igc.IGC_ERR_WORKSPACE, igc.IGC_OK)
P, Q, S = (ctypes.c_void_p(v) for v in (4096, 8192, 12288))
A, B, C, D = (ctypes.c_void_p(v) for v in (1 << 16, 1 << 17, 1 << 18, 1 << 19))
ODD = ctypes.c_void_p(4098)


def test_header_declares_the_operators_and_the_library_exports_them():
    names = {"linear_act", "linear_act_backward", "linear_act_backward_workspace_size", "gated_ffn",
             "gated_ffn_backward", "gated_ffn_backward_workspace_size", "grad_norm_clip",
             "grad_norm_clip_workspace_size", "igc_plan_ffn"}
    assert set(igc.declared_functions(igc.FFN_HEADER)) == names
    for n in names:
        assert ctypes.cast(getattr(igc.lib(), n), ctypes.c_void_p).value


def linear(M=4, N=8, K=16, dt=1, X=P, ldx=16, W=Q, ldw=16, b=None, bt=0, act=0, R=None, ldr=8,
           Z=None, ldz=8, Y=S, ldy=8, yt=1):
    return igc.lib().linear_act(M, N, K, dt, X, ldx, W, ldw, b, bt, act, R, ldr, Z, ldz, Y, ldy,
                                yt, None)


def test_linear_act_refusals():
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(dt=0), dict(dt=3), dict(yt=2),
                dict(b=P, bt=2), dict(act=5), dict(act=-1), dict(Y=None), dict(ldy=7),
                dict(R=P, ldr=7), dict(Z=P, ldz=7), dict(X=None), dict(W=None), dict(ldx=15),
                dict(ldw=15)):
        assert linear(**bad) == INVALID, bad
    # an output that is an input or another output; a residual in place of another shape
    for bad in (dict(Y=P), dict(Y=Q), dict(b=S), dict(Z=S), dict(Z=P), dict(Z=A, R=A),
                dict(R=S, ldr=9), dict(R=S, yt=0)):
        assert linear(**bad) == INVALID, bad
    for bad in (dict(X=ODD), dict(W=ODD), dict(ldx=17), dict(ldw=20)):
        assert linear(**bad) == MISALIGNED, bad
    assert linear(M=1 << 31) == igc.IGC_ERR_UNSUPPORTED
    assert linear(M=0, X=None, Y=None) == OK and linear(N=0, W=None, Y=None) == OK


def linear_bwd(M=4, N=8, K=16, dt=2, dY=P, lddy=8, Z=None, ldz=8, act=0, X=Q, ldx=16, W=S, ldw=16,
               dX=A, lddx=16, dW=B, lddw=16, dwt=2, db=None, dbt=0, ws=None, n=0):
    return igc.lib().linear_act_backward(M, N, K, dt, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX,
                                         lddx, dW, lddw, dwt, db, dbt, ws, n, None)


def test_linear_act_backward_refusals():
    for bad in (dict(M=-1), dict(dt=0), dict(act=9), dict(dwt=1), dict(db=P, dbt=1), dict(lddx=15),
                dict(lddw=15), dict(dY=None), dict(lddy=7), dict(act=2), dict(act=2, Z=P, ldz=7),
                dict(X=None), dict(W=None), dict(ldx=15), dict(ldw=15), dict(dX=P), dict(dX=Q),
                dict(dW=S), dict(dW=A), dict(db=A), dict(db=P), dict(act=2, Z=B)):
        assert linear_bwd(**bad) == INVALID, bad
    for bad in (dict(X=ODD), dict(W=ODD), dict(ldx=17), dict(ldw=20)):
        assert linear_bwd(**bad) == MISALIGNED, bad
    # nothing asked for, or nothing to compute: no operand is looked at
    assert linear_bwd(dX=None, dW=None, dY=None, X=None, W=None) == OK
    assert linear_bwd(M=0, dW=None, dY=None) == OK


def gated(M=4, F=8, K=16, dt=1, X=P, ldx=16, Wg=Q, Wu=S, ldw=16, bg=None, bu=None, bt=0, act=4,
          G=None, U=None, ldgu=8, H=A, ldh=8):
    return igc.lib().gated_ffn(M, F, K, dt, X, ldx, Wg, Wu, ldw, bg, bu, bt, act, G, U, ldgu, H, ldh,
                               None)


def test_gated_ffn_refusals():
    for bad in (dict(M=-1), dict(F=-1), dict(K=-1), dict(dt=0), dict(bg=P, bt=2), dict(bu=P, bt=2),
                dict(act=5), dict(H=None), dict(ldh=7), dict(G=P), dict(U=P),
                dict(G=B, U=C, ldgu=7), dict(H=P), dict(H=Q), dict(H=S), dict(bg=A),
                dict(G=B, U=B), dict(G=A, U=B), dict(G=P, U=B), dict(X=None), dict(Wg=None), dict(Wu=None), dict(ldx=15),
                dict(ldw=15)):
        assert gated(**bad) == INVALID, bad
    for bad in (dict(X=ODD), dict(Wg=ODD), dict(Wu=ODD), dict(ldx=17), dict(ldw=20)):
        assert gated(**bad) == MISALIGNED, bad
    assert gated(M=0, H=None) == OK and gated(F=0, H=None) == OK


E, F_, G_ = (ctypes.c_void_p(v) for v in (1 << 20, 1 << 21, 1 << 22))


def gated_bwd(M=4, F=8, K=16, dt=2, dH=P, lddh=8, G=Q, U=S, ldgu=8, act=4, X=A, ldx=16, Wg=B, Wu=C,
              ldw=16, dX=D, lddx=16, dWg=E, dWu=F_, lddw=16, dwt=2, dbg=None, dbu=None, dbt=0,
              ws=None, n=0):
    return igc.lib().gated_ffn_backward(M, F, K, dt, dH, lddh, G, U, ldgu, act, X, ldx, Wg, Wu, ldw,
                                        dX, lddx, dWg, dWu, lddw, dwt, dbg, dbu, dbt, ws, n, None)


def test_gated_ffn_backward_refusals():
    for bad in (dict(M=-1), dict(dt=0), dict(act=9), dict(dWg=None), dict(dWu=None), dict(dbg=G_),
                dict(dbu=G_), dict(dwt=1), dict(dbg=G_, dbu=G_), dict(dX=P), dict(dX=A), dict(dWg=D),
                dict(dWu=E), dict(dWg=Q), dict(lddx=15), dict(lddw=15),
                dict(dH=None), dict(lddh=7), dict(G=None), dict(U=None), dict(ldgu=7), dict(X=None),
                dict(Wg=None), dict(Wu=None), dict(ldx=15), dict(ldw=15)):
        assert gated_bwd(**bad) == INVALID, bad
    for bad in (dict(X=ODD), dict(Wg=ODD), dict(Wu=ODD), dict(ldx=17), dict(ldw=20)):
        assert gated_bwd(**bad) == MISALIGNED, bad


def clip(n=2, grads=(4096, 8192), sizes=(5, 7), types=(0, 1), out=None, max_norm=1.0, eps=0.0,
         norm=P, ws=P, nbytes=1 << 20):
    g = (ctypes.c_void_p * max(len(grads), 1))(*grads)
    s = (ctypes.c_int64 * max(len(sizes), 1))(*sizes)
    t = (ctypes.c_int32 * max(len(types), 1))(*types)
    o = None if out is None else (ctypes.c_void_p * len(out))(*out)
    return igc.lib().grad_norm_clip(n, g, s, t, o, max_norm, eps, norm, ws, nbytes, None)


def test_grad_norm_clip_refusals():
    for bad in (dict(n=-1), dict(norm=None), dict(max_norm=-1.0), dict(max_norm=float("nan")),
                dict(eps=-1.0), dict(eps=float("nan")), dict(sizes=(5, -7)), dict(types=(0, 3)),
                dict(grads=(4096, None)), dict(out=(None, 4096))):
        assert clip(**bad) == INVALID, bad
    assert igc.lib().grad_norm_clip(1, None, None, None, None, 1.0, 0.0, P, P, 1 << 20,
                                    None) == INVALID
    for bad in (dict(grads=(4098, 8192)), dict(grads=(4096, 8193)), dict(out=(4097, 8192))):
        assert clip(**bad) == MISALIGNED, bad


def test_workspace_sizes():
    def up(v):
        return -(-v // 256) * 256

    # dZ with rows padded to 8 columns, then one row of partial sums per chunk of rows
    assert igc.linear_act_backward_workspace_size(3, 5, 7) == up(3 * 8 * 2) + up(5 * 4)
    assert igc.gated_ffn_backward_workspace_size(3, 5, 7) == 2 * up(3 * 8 * 2) + up(2 * 5 * 4)
    assert igc.linear_act_backward_workspace_size(-1, 5, 7) == 0
    assert igc.gated_ffn_backward_workspace_size(1, -5, 7) == 0
    assert igc.grad_norm_clip_workspace_size(-1) == 0
    one = igc.grad_norm_clip_workspace_size(1)
    assert one == igc.grad_norm_clip_workspace_size(0) == igc.grad_norm_clip_workspace_size(1024)
    assert igc.grad_norm_clip_workspace_size(1025) == 2 * one


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    X, W = t(4, 16), t(8, 16)
    with pytest.raises(TypeError, match="X has dtype"):
        igc.linear_act(X.float(), W)
    with pytest.raises(TypeError, match="W has dtype"):
        igc.linear_act(X, W.half())
    with pytest.raises(ValueError, match="W has shape"):
        igc.linear_act(X, t(8, 15))
    with pytest.raises(ValueError, match="act is"):
        igc.linear_act(X, W, act="tanh")
    with pytest.raises(ValueError, match="bias must be"):
        igc.linear_act(X, W, bias=t(9))
    with pytest.raises(ValueError, match="bias must be"):
        igc.linear_act(X, W, bias=t(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="rows apart"):      # a broadcast view has no rows
        igc.linear_act(X, W, residual=t(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="unit inner stride"):
        igc.linear_act(t(16, 4).t(), W)
    with pytest.raises(ValueError, match="Y has shape"):
        igc.linear_act(X, W, Y=t(4, 9))
    with pytest.raises(ValueError, match="X must be a matrix"):
        igc.linear_act(t(16), W)
    with pytest.raises(ValueError, match="CUDA"):
        igc.linear_act(X, W)
    dY = t(4, 8)
    with pytest.raises(ValueError, match="pre-activation"):
        igc.linear_act_backward(dY, X, W, act="gelu", dX=t(4, 16))
    with pytest.raises(ValueError, match="dX needs W"):
        igc.linear_act_backward(dY, X, None, dX=t(4, 16))
    with pytest.raises(ValueError, match="rows apart"):
        igc.linear_act_backward(t(1, 8).expand(4, 8), X, W, dX=t(4, 16))
    with pytest.raises(TypeError, match="dX has dtype"):
        igc.linear_act_backward(dY, X, W, dX=t(4, 16, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        igc.linear_act_backward(dY, X, W, dX=t(4, 16))
    with pytest.raises(ValueError, match="one row stride"):
        igc.gated_ffn(X, W, t(8, 24)[:, :16])
    with pytest.raises(ValueError, match="go together"):
        igc.gated_ffn(X, W, W, G=t(4, 8))
    with pytest.raises(ValueError, match="one type"):
        igc.gated_ffn(X, W, W, bg=t(8), bu=t(8, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        igc.gated_ffn(X, W, W)
    with pytest.raises(ValueError, match="go together"):
        igc.gated_ffn_backward(dY, dY, dY, X, W, W, dWg=t(8, 16))
    with pytest.raises(ValueError, match="CUDA"):
        igc.gated_ffn_backward(dY, dY, dY, X, W, W, dX=t(4, 16))
    with pytest.raises(TypeError, match="a gradient has dtype"):
        igc.grad_norm_clip([t(4, dtype=torch.float64)], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        igc.grad_norm_clip([t(4, 8).t()], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        igc.grad_norm_clip([t(4)], 1.0)
    with pytest.raises(ValueError, match="as many"):
        igc.grad_norm_clip([t(4)], 1.0, out=[])


def test_plans():
    """The schedule rules on a GPU of 152 SMs, at cases on either side of them."""
    lin, gat, gx, gw = (igc.PLAN_FFN_LINEAR, igc.PLAN_FFN_GATED, igc.PLAN_FFN_GRAD_X,
                        igc.PLAN_FFN_GRAD_W)
    # one token through 32 column blocks of long rows: eight CTAs share a block
    p = igc.igc_plan_ffn(lin, 1, 4096, 16384)
    assert (p["small"], p["rows"], p["row_blocks"], p["split"]) == (1, 16, 1, 8)
    # the gated pair has twice the blocks (64 columns each): 128 of them, two CTAs each
    p = igc.igc_plan_ffn(gat, 1, 8192, 4096)
    assert (p["small"], p["rows"], p["split"]) == (1, 16, 2)
    # enough blocks to fill the GPU: no split
    assert igc.igc_plan_ffn(gat, 48, 16384, 4096)["split"] == 1
    # large outputs take the 256-row tiles, in every direction
    for op, count in ((lin, 1), (gat, 1), (gx, 1), (gx, 2), (gw, 1), (gw, 2)):
        p = igc.igc_plan_ffn(op, 8192, 8192, 8192, count)
        assert (p["small"], p["rows"], p["row_blocks"], p["split"]) == (0, 256, 32, 1)
        assert p["tiles_ns"] < p["small_ns"]
    # GradW's blocks of rows are multiples of 64 (atoms contiguous along them)
    assert igc.igc_plan_ffn(gw, 64, 100, 100)["rows"] % 64 == 0
    # 15 x 3 tiles of 256 columns and 15 x 4 of 192 are one round on 76 pairs either way:
    # the narrower ones are done sooner; many rounds take the wider ones
    for shape in ((3630, 702, 2944), (2000, 1300, 200), (1800, 1501, 264)):
        assert igc.igc_plan_ffn(lin, *shape)["columns"] == 192
    assert igc.igc_plan_ffn(lin, 8192, 8192, 8192)["columns"] == 256
    # a forced tile width is always the tiles
    igc.igc_set_tile_width(128)
    try:
        assert igc.igc_plan_ffn(lin, 1, 4096, 16384)["small"] == 0
    finally:
        igc.igc_set_tile_width(0)
    for bad in ((4, 1, 1, 1, 1, 152), (0, 0, 1, 1, 1, 152), (0, 1, 1, 1, 3, 152),
                (0, 1, 1, 1, 1, 1)):
        with pytest.raises(igc.IGCError):
            igc.igc_plan_ffn(*bad)
