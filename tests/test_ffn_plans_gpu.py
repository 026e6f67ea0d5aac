"""igc_plan_ffn answers what the backward passes run: where it says 256-row tiles, the gradients
have the bits that these tiles give when they are forced; where it says a contraction shared by
several CTAs (another order of the sums), they do not."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from test_linear_act_gpu import BF16, F32, generator, matrix

pytestmark = pytest.mark.gpu

SIZES = [(900, 1000, 1000), (900, 1024, 1024), (1500, 1001, 777), (509, 1001, 777),
         (900, 2000, 1000), (2000, 1000, 1000), (64, 2000, 1030), (301, 1111, 650), (3000, 1001, 777),
         (1100, 1024, 768)]


def gradients(count, dy, u, x, w):
    M, K = x.shape
    N = dy.shape[1]
    dX = torch.empty((M, K), device="cuda", dtype=BF16)
    dW, dWu = (torch.empty((N, K), device="cuda", dtype=F32) for _ in range(2))
    if count == 1:
        igc.linear_act_backward(dy, x, w, dX=dX, dW=dW)
    else:
        igc.gated_ffn_backward(dy, u, u, x, w, w, dX=dX, dWg=dW, dWu=dWu)
    return dX, dW


@pytest.mark.parametrize("count", [1, 2])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_plan_is_what_runs(M, N, K, count):
    gen = generator(M, N, K, 95)
    x, w = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, K ** -0.5)
    dy, u = matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)
    got = gradients(count, dy, u, x, w)
    forced = {}
    for width in (128, 256):
        igc.igc_set_tile_width(width)
        try:
            forced[width] = gradients(count, dy, u, x, w)
        finally:
            igc.igc_set_tile_width(0)
    check_device_ok()
    seen = 0
    for i, op in enumerate((igc.PLAN_FFN_GRAD_X, igc.PLAN_FFN_GRAD_W)):
        p = igc.igc_plan_ffn(op, M, N, K, count,
                             sms=torch.cuda.get_device_properties(0).multi_processor_count)
        if not p["small"]:
            assert torch.equal(got[i], forced[p["columns"]][i]), (op, p)
            seen += 1
        elif p["split"] > 1:
            assert all(not torch.equal(got[i], f[i]) for f in forced.values()), (op, p)
            seen += 1
    assert seen
