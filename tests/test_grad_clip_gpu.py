"""grad_norm_clip against its 64-bit form."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
from gpu_helpers import check_device_ok

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


def tensors(sizes, dtypes, seed, scale=0.1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(dt)
            for n, dt in zip(sizes, dtypes)]


def norm64(grads):
    return float(sum(g.double().square().sum() for g in grads)) ** 0.5


def check(got_norm, outs, grads, max_norm, eps=1e-6):
    want = norm64(grads)
    # squares and per-thread sums in fp32: each term is added at most 2^12 times before it
    # reaches fp64, so the norm is off by less than half of 2^12 2^-24
    tol = 2.0 ** -13
    assert abs(float(got_norm) - want) <= tol * want
    coef = min(1.0, max_norm / (want + eps))
    for o, g in zip(outs, grads):
        ref = g.double() * coef
        bound = ref.abs() * (tol + 2 * UNIT[o.dtype]) + (2.0 ** -24 if o.dtype == F16 else 0.0)
        assert bool(((o.double() - ref).abs() <= bound).all())


CASES = [[1], [0], [7], [4096], [4097, 1, 0, 65536], [100003], [3, 5, 1000, 0, 70001, 12],
         [17] * 65, [1000 + i for i in range(200)], [3] * 1100, [300001, 5000000]]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_clips_lists_of_tensors(i):
    sizes = CASES[i]
    dtypes = [(F32, BF16, F16)[(i + j) % 3] for j in range(len(sizes))]
    for max_norm in (0.01, 1e6):
        grads = tensors(sizes, dtypes, i)
        out = [torch.full_like(g, 7.0) for g in grads]
        norm = igc.grad_norm_clip(grads, max_norm, out=out)
        alone = igc.grad_norm_clip(grads, max_norm, out=False)
        check_device_ok()
        assert norm.shape == () and torch.equal(norm, alone)
        check(norm, out, grads, max_norm)
        if max_norm > 1:
            assert all(torch.equal(o, g) for o, g in zip(out, grads))
        kept = [g.clone() for g in grads]
        again = igc.grad_norm_clip(grads, max_norm)          # in place
        check_device_ok()
        assert torch.equal(norm, again)
        assert all(torch.equal(o, g) for o, g in zip(out, grads))
        del kept


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_unaligned_tensors(dtype):
    """Views at every element offset, inputs and outputs shifted against one another."""
    buf = tensors([40000], [dtype], 3)[0]
    for a in range(8):
        for b in (0, a, 3):
            g = buf[a:a + 9001]
            obuf = torch.full((9100,), 9.0, device="cuda", dtype=dtype)
            norm = igc.grad_norm_clip([g], 0.5, out=[obuf[b:b + 9001]])
            check_device_ok()
            check(norm, [obuf[b:b + 9001]], [g], 0.5)
            assert bool((obuf[:b] == 9.0).all()) and bool((obuf[b + 9001:] == 9.0).all())


def test_nothing_and_zeros():
    norm = torch.full((1,), 5.0, device="cuda")
    assert igc.grad_norm_clip([], 1.0, norm=norm) is norm
    z = torch.zeros(1000, device="cuda")
    nz = igc.grad_norm_clip([z], 1.0)
    check_device_ok()
    assert float(norm) == 0.0 and float(nz) == 0.0 and not bool(z.any())


def test_nan_and_infinity_as_the_formula_has_them():
    g = tensors([5000, 300], [F32, BF16], 4)
    bad = [t.clone() for t in g]
    bad[1][7] = float("nan")
    out = [torch.empty_like(t) for t in bad]
    norm = igc.grad_norm_clip(bad, 1.0, out=out)
    check_device_ok()
    assert bool(norm.isnan()) and all(bool(o.isnan().all()) for o in out)
    bad = [t.clone() for t in g]
    bad[0][4321] = float("-inf")
    norm = igc.grad_norm_clip(bad, 1.0, out=out)
    check_device_ok()
    assert float(norm) == float("inf")
    assert bool(out[0][4321].isnan()) and int(out[0].isnan().sum()) == 1
    assert not bool(out[0].nan_to_num(nan=0.0).any()) and not bool(out[1].any())


def test_sizes_past_32_bits():
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, device="cuda", dtype=BF16)
    g[-1] = 3.0
    want = (0.25 * (n - 1) + 9.0) ** 0.5
    norm = igc.grad_norm_clip([g], want / 2)
    check_device_ok()
    assert abs(float(norm) - want) <= 2.0 ** -13 * want
    assert float(g[-1]) == 1.5 and float(g[0]) == 0.25 and float(g[n // 2]) == 0.25
    assert bool((g[-100000:-1] == 0.25).all())


def test_repeatable_side_stream_and_graph():
    grads = tensors([70001, 300, 123456], [BF16, F32, F16], 5)
    out = [torch.empty_like(g) for g in grads]
    first = igc.grad_norm_clip(grads, 1.0, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(g) for g in grads]
    second = igc.grad_norm_clip(grads, 1.0, out=out2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and all(torch.equal(a, b) for a, b in zip(out, out2))
    norm = torch.zeros((), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        igc.grad_norm_clip(grads, 1.0, out=out, norm=norm)
    grads[1].mul_(3)
    graph.replay()
    check_device_ok()
    check(norm, out, grads, 1.0)
