"""A matrix or vector that does not start on a boundary of its elements is refused before
anything is launched (on the GPU its first access would be a fault)."""

import ctypes

import pytest

import implicit_gemm_conv_tcgen05_gb300 as igc
from test_ffn_cpu import clip, gated, gated_bwd, linear, linear_bwd

MISALIGNED = igc.IGC_ERR_MISALIGNED
F32, F16 = igc.IGC_F32, igc.IGC_F16
P, Q = (ctypes.c_void_p((1 << 24) * i) for i in (1, 2))


def off(p, by):
    return ctypes.c_void_p(p.value + by)


@pytest.mark.parametrize("by", [1, 3, 5])
def test_half_way_into_a_16_bit_element(by):
    p = off(P, by)
    for bad in (dict(Y=p), dict(Z=p), dict(R=p), dict(b=p, bt=F16), dict(b=p, bt=F32),
                dict(Y=p, yt=F32), dict(Y=p, K=0), dict(b=p, bt=F16, K=0)):
        assert linear(**bad) == MISALIGNED, bad
    for bad in (dict(dY=p), dict(Z=p, act=2), dict(dX=p), dict(dW=p), dict(db=p, dbt=2),
                dict(db=p, dbt=F32), dict(dX=p, N=0, dW=None), dict(dW=p, M=0)):
        assert linear_bwd(**bad) == MISALIGNED, bad
    for bad in (dict(H=p), dict(G=p, U=Q), dict(G=Q, U=p), dict(bg=p, bt=F16), dict(bu=p, bt=F16)):
        assert gated(**bad) == MISALIGNED, bad
    for bad in (dict(dH=p), dict(G=p), dict(U=p), dict(dX=p), dict(dWg=p), dict(dWu=p),
                dict(dbg=p, dbu=Q, dbt=2), dict(dbg=Q, dbu=p, dbt=2)):
        assert gated_bwd(**bad) == MISALIGNED, bad
    assert clip(norm=p) == MISALIGNED


def test_half_way_into_an_fp32_element():
    p = off(P, 2)
    for bad in (dict(Y=p, yt=F32), dict(b=p, bt=F32)):
        assert linear(**bad) == MISALIGNED, bad
    for bad in (dict(dW=p, dwt=F32), dict(db=p, dbt=F32)):
        assert linear_bwd(**bad) == MISALIGNED, bad
    for bad in (dict(bg=p, bt=F32), dict(bu=p, bt=F32)):
        assert gated(**bad) == MISALIGNED, bad
    for bad in (dict(dWg=p, dwt=F32), dict(dWu=p, dwt=F32), dict(dbg=p, dbu=Q, dbt=F32),
                dict(dbg=Q, dbu=p, dbt=F32)):
        assert gated_bwd(**bad) == MISALIGNED, bad
    assert clip(norm=p) == MISALIGNED
