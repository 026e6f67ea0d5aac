"""Outputs whose rows start on 16-byte boundaries but are padded: nothing past their last column
is written, whatever 16-byte piece it falls into (bulk tensor stores clip in pieces of 16
bytes).  The padding may be the neighbouring columns of a wider matrix."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import oracle
import synth
from gpu_helpers import assert_fp16_bound, check_device_ok, dev, host

pytestmark = pytest.mark.gpu

# columns: each residue modulo 16 once, below, at and past the tiles' and boxes' widths
COLUMNS = [1, 18, 67, 100, 133, 150, 199, 232, 265, 314, 331, 380, 429, 494, 607, 720]


def padded(M, N, dtype):
    """An M x N view with rows of whole 16 bytes and 16 more, and its buffer."""
    es = torch.empty(0, dtype=dtype).element_size()
    per = 16 // es
    buf = torch.full((M, -(-N // per) * per + per), 77, device="cuda", dtype=dtype)
    return buf[:, :N], buf


def untouched(buf, N, what):
    assert bool((buf[:, N:] == 77).all()), f"{what}: written past column {N}"


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("N", COLUMNS)
def test_float_gemms(M, N):
    K = 72
    A, Bt = synth.uniform_f16(300 + M, 1, (M, K)), synth.uniform_f16(400 + N, 2, (N, K))
    ref, sabs = oracle.gemm_f16(A, Bt)
    for gemm, t16 in ((igc.gemm_f16, torch.float16), (igc.gemm_bf16, torch.bfloat16)):
        a, b = dev(A), dev(Bt)
        if t16 is torch.bfloat16:   # operands exact in bf16 as well
            a, b = (t.bfloat16().half() for t in (a, b))
            ref, sabs = oracle.gemm_f16(host(a), host(b))
            a, b = a.bfloat16(), b.bfloat16()
        for out in (torch.float32, t16):
            (C, cbuf), (C32, buf32) = padded(M, N, out), padded(M, N, torch.float32)
            gemm(a, b, C, C32)
            check_device_ok()
            assert_fp16_bound(host(C32), ref, sabs, "fp32 copy")
            assert torch.equal(C, C32.to(out))
            untouched(cbuf, N, f"{gemm.__name__} {out}")
            untouched(buf32, N, f"{gemm.__name__} fp32 copy")


@pytest.mark.parametrize("path", [0, 1, 2, 3],
                         ids=["tcgen05", "mma_sync", "fused", "convert"])
@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("N", COLUMNS)
def test_int8_gemm(M, N, path):
    K = 64
    rng = np.random.default_rng(M * 1000 + N)
    A = rng.integers(0, 256, size=(M, K)).astype(np.uint8)
    Bt = rng.integers(-128, 128, size=(N, K)).astype(np.int8)
    want32, want8, _, _ = oracle.gemm_s8_zp(A, Bt, a_signed=0, b_signed=1, zA=3, zB=-5,
                                            scale=2.0 ** -9)
    a, b = dev(A), dev(Bt)
    (C32, buf32), (C8, buf8) = padded(M, N, torch.int32), padded(M, N, torch.int8)
    (Y, ybuf) = padded(M, N, torch.float32)
    igc.igc_set_int8_path(path)
    try:
        igc.gemm_s8_zp(a, b, zA=3, zB=-5, C32=C32, C8=C8, scale=2.0 ** -9)
        igc.gemm_s8_zp_dequant(a, b, zA=3, zB=-5, Y=Y)
    finally:
        igc.igc_set_int8_path(0)
    check_device_ok()
    assert np.array_equal(host(C32), want32) and np.array_equal(host(C8), want8)
    assert np.array_equal(host(Y), want32.astype(np.float32))
    for buf, what in ((buf32, "C32"), (buf8, "C8"), (ybuf, "Y")):
        untouched(buf, N, what)


@pytest.mark.parametrize("N", [67, 133, 232, 720])
def test_int8_gemm_noalloc(N):
    M, K = 200, 128
    rng = np.random.default_rng(N)
    A = rng.integers(-128, 128, size=(M, K)).astype(np.int8)
    Bt = rng.integers(-128, 128, size=(N, K)).astype(np.int8)
    want32, want8, _, _ = oracle.gemm_s8_zp(A, Bt, a_signed=1, b_signed=1, zA=0, zB=0,
                                            scale=2.0 ** -9)
    (C32, buf32), (C8, buf8) = padded(M, N, torch.int32), padded(M, N, torch.int8)
    igc.gemm_s8_zp_noalloc(dev(A), dev(Bt), C32=C32, C8=C8, scale=2.0 ** -9)
    check_device_ok()
    assert np.array_equal(host(C32), want32) and np.array_equal(host(C8), want8)
    untouched(buf32, N, "C32")
    untouched(buf8, N, "C8")
