"""Memory that the binding holds between calls, over many streams and after a release."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok

pytestmark = pytest.mark.gpu


def test_many_streams_hold_nothing_and_release_gives_back():
    M, N, K = 700, 264, 136
    dy, z = (torch.randn((M, N), device="cuda").bfloat16() for _ in range(2))
    x, w = torch.randn((M, K), device="cuda").bfloat16(), torch.randn((N, K), device="cuda").bfloat16()

    def call(dX, dW, db):
        igc.linear_act_backward(dy, x, w, act="silu", Z=z, dX=dX, dW=dW, dbias=db)

    outs = [(torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda"))
            for _ in range(24)]
    igc.release_workspaces()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    call(*outs[0])
    held = torch.cuda.memory_allocated() - before
    need = igc.linear_act_backward_workspace_size(M, N, K)
    assert need <= held < need + 4096
    streams = [torch.cuda.Stream() for _ in outs]
    for s, out in zip(streams, outs):
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            call(*out)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before == held
    igc.release_workspaces()
    assert torch.cuda.memory_allocated() == before
    call(*outs[1])
    check_device_ok()
    for out in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, outs[0]))
    igc.release_workspaces()
