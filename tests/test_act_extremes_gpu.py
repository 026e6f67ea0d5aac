"""Activations and their derivatives where the sigmoids have long saturated: at |z| of 1e4
and more act(z) is z or 0 and act'(z) is 1 or 0 to every bit of fp32, up to the largest finite
values of the types."""

import pytest
import torch

import ffn_reference as ref
import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LARGE = {BF16: [1e4, 1e10, 1e20, 1e27, 1.5e27, 1.7e27, 2e27, 1e30, 1e38, 3.3e38],
         F16: [1e4, 3e4, 65504.0]}
ROWS = [1, 40, 600]   # column sums within a block, in a cluster, over chunks


def extremes(dtype, name):
    """z and, in fp32, act(z) and act'(z)."""
    pos = torch.tensor(LARGE[dtype], device="cuda").to(dtype)
    z = torch.cat([pos, -pos])
    up = torch.cat([torch.ones_like(pos), torch.zeros_like(pos)]).float()
    if name == "none":
        up = torch.ones_like(up)
    return z, z.float() * up, up


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", ROWS)
def test_linear_derivative(M, dtype, name):
    z, _, up = extremes(dtype, name)
    N, K = z.numel(), 24
    Z = z.expand(M, N).contiguous()
    dy = torch.ones((M, N), device="cuda", dtype=dtype)
    x = torch.ones((M, K), device="cuda", dtype=dtype)
    w = torch.ones((N, K), device="cuda", dtype=dtype)
    dX, dW = torch.empty_like(x), torch.empty((N, K), device="cuda")
    db = torch.empty(N, device="cuda")
    igc.linear_act_backward(dy, x, w, act=name, Z=Z, dX=dX, dW=dW, dbias=db)
    check_device_ok()
    assert torch.equal(db, M * up)
    assert torch.equal(dW, (M * up)[:, None].expand(N, K))
    assert bool((dX == up.sum()).all())


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", ROWS)
def test_gated_derivative(M, dtype, name):
    """One row counts (dH is 0 in the others), so that no sum leaves the range."""
    z, value, up = extremes(dtype, name)
    F = z.numel()
    G = z.expand(M, F).contiguous()
    U = torch.full((M, F), 2.0, device="cuda", dtype=dtype)
    dh = torch.zeros((M, F), device="cuda", dtype=dtype)
    dh[M // 2] = 1.0
    dbg, dbu = (torch.empty(F, device="cuda") for _ in range(2))
    igc.gated_ffn_backward(dh, G, U, None, None, None, act=name, dbg=dbg, dbu=dbu)
    check_device_ok()
    assert torch.equal(dbg, 2 * up)
    assert torch.equal(dbu, value)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [1, 300])
def test_forward(M, dtype, name):
    z, value, _ = extremes(dtype, name)
    N = z.numel()
    x = torch.zeros((M, 8), device="cuda", dtype=dtype)
    x[:, 0] = 1.0
    w = torch.zeros((N, 8), device="cuda", dtype=dtype)
    w[:, 0] = z
    Y = torch.empty((M, N), device="cuda", dtype=F32)
    igc.linear_act(x, w, act=name, Y=Y)
    H = igc.gated_ffn(x, w, torch.ones_like(w), act=name)
    check_device_ok()
    assert torch.equal(Y, value.expand(M, N))
    assert torch.equal(H, value.to(dtype).expand(M, N))


@pytest.mark.parametrize("name", ref.ACTS)
def test_nan_stays_nan(name):
    """But for ReLU, whose derivative is 1 where z > 0 and else 0."""
    Z = torch.tensor([[float("nan"), 1.0]], device="cuda", dtype=BF16)
    dy = torch.ones((1, 2), device="cuda", dtype=BF16)
    if name == "none":
        dy[0, 0] = float("nan")
    db = torch.empty(2, device="cuda")
    igc.linear_act_backward(dy, None, None, act=name, Z=Z, dbias=db)
    check_device_ok()
    assert float(db[0]) == 0.0 if name == "relu" else bool(db[0].isnan())
    assert bool(db[1].isfinite())
