"""Products of different shapes on streams of their own, so that CTAs that want different
amounts of tensor memory share SMs: the same bits as alone."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok
from test_linear_act_gpu import BF16, generator, matrix

pytestmark = pytest.mark.gpu


def make(kind, M, N, K, gen):
    x, w, w2 = matrix(gen, M, K, BF16), matrix(gen, N, K, BF16, K ** -0.5), matrix(gen, N, K, BF16)
    dy, z = matrix(gen, M, N, BF16), matrix(gen, M, N, BF16)
    if kind == "linear":
        return lambda: [igc.linear_act(x, w, act="silu", residual=dy)]
    if kind == "gated":
        return lambda: [igc.gated_ffn(x, w, w2)]
    if kind == "linear_bwd":
        return lambda: list(igc.linear_act_backward(dy, x, w, act="silu", Z=z)[:2])
    return lambda: list(igc.gated_ffn_backward(dy, z, z, x, w, w2)[:3])


MIXES = [
    # 256 columns in clusters of 5 beside 32 columns, alone and in clusters
    [("gated", 139, 1690, 637), ("linear", 1, 1000, 777), ("linear", 1, 4096, 2048),
     ("gated", 139, 1690, 637)],
    # 192-wide tiles (512 columns) beside one-stage blocks
    [("linear", 2000, 1300, 200), ("linear", 1, 5000, 64), ("linear", 16, 700, 64),
     ("linear", 1800, 1501, 264)],
    # 64, 128 and 256 columns, forward and backward
    [("linear", 50, 900, 3000), ("linear", 120, 700, 2000), ("gated_bwd", 301, 1111, 650),
     ("linear_bwd", 70, 800, 1500), ("gated", 250, 640, 900)],
]


@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_streams_of_different_shapes(mix):
    gen = generator(mix, 97)
    calls = [make(*c, gen) for c in MIXES[mix]]
    alone = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    results = [[] for _ in calls]
    for _ in range(60):
        for call, stream, kept in zip(calls, streams, results):
            with torch.cuda.stream(stream):
                kept.append(call())
    torch.cuda.synchronize()
    check_device_ok()
    for kept, want in zip(results, alone):
        for got in kept:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
