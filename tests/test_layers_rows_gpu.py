"""Where the rows of the layer operators start: those of results that the binding allocates, and
single rows, whose stride says nothing."""

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc
import layers_reference as ref
from gpu_helpers import check_device_ok
from layers_reference import BF16, F16, F32, generator, matrix

pytestmark = pytest.mark.gpu


def results(X, S, W, tok):
    """The matrices that each operator allocates by itself."""
    M, N = X.shape
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    return {"dropout_add": igc.dropout_add(X, 0.2, seed=3),
            "dropout_add f32": igc.dropout_add(X, 0.2, seed=3, residual=S),
            "layer_norm": igc.layer_norm(X, residual=S),
            "layer_norm_backward": igc.layer_norm_backward(X, S, mean, rstd)[0],
            "embedding_lookup": igc.embedding_lookup(tok, W),
            "embedding_backward": igc.embedding_backward(tok, X, V=W.shape[0])}


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N", [1001, 9, 64])
def test_results_have_padded_rows_where_the_inputs_have(dtype, N):
    def made(pad):
        gen = generator(N, str(dtype))
        X, S, W = (matrix(gen, 30, N, t, pad=pad) for t in (dtype, F32, dtype))
        return results(X, S, W, torch.arange(30, device="cuda") % 7)

    padded, close = made(None), made(0)
    check_device_ok()
    for name, y in padded.items():
        assert y.stride(0) * y.element_size() % 16 == 0 and y.stride(0) - N < 8, name
        assert y.stride(1) == 1 and y.shape == (30, N)
        assert close[name].is_contiguous(), name
    # dropout and lookups are the same to the bit however rows lie
    for name in ("dropout_add", "dropout_add f32", "embedding_lookup", "embedding_backward"):
        assert torch.equal(padded[name], close[name]), name


@pytest.mark.parametrize("N", [1, 9, 1001, 4097, 9001, 20003])
def test_a_single_row_may_have_any_stride(N):
    """The bits of a single row do not go by its stride."""
    gen = generator(N)
    X, S = (torch.randn((2, N + 3), generator=gen, device="cuda").to(t)[:1, :N]
            for t in (BF16, F32))
    wide = results(X.as_strided((1, N), (-(-N // 8) * 8, 1)), S, X,
                   torch.zeros(1, device="cuda", dtype=torch.int64))
    mean, rstd = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    outs = []
    for ld in (-(-N // 8) * 8, N, N + 3):      # through the C entry, which sees the stride
        Y, dS = torch.empty(N, device="cuda", dtype=BF16), torch.empty(N, device="cuda")
        assert igc.lib().layer_norm(1, N, igc.IGC_BF16, X.data_ptr(), ld, S.data_ptr(), ld,
                                    igc.IGC_F32, 0.0, 0, 0, None, None, None, igc.IGC_F32, 1e-5,
                                    None, 0, Y.data_ptr(), ld, mean.data_ptr(), rstd.data_ptr(),
                                    None) == igc.IGC_OK
        assert igc.lib().layer_norm_backward(1, N, igc.IGC_BF16, X.data_ptr(), ld, S.data_ptr(),
                                             ld, igc.IGC_F32, mean.data_ptr(), rstd.data_ptr(),
                                             None, igc.IGC_F32, None, 0, 0.0, 0, 0, None,
                                             dS.data_ptr(), ld, None, 0, None, None, igc.IGC_F32,
                                             None, 0, None) == igc.IGC_OK
        check_device_ok()
        outs.append((Y, dS))
    for Y, dS in outs[1:]:
        assert torch.equal(Y, outs[0][0]) and torch.equal(dS, outs[0][1])
    assert torch.equal(outs[0][0], wide["layer_norm"][0])
    y, err = ref.dropout64(X, 0.0, 0, 0, S)
    want, dy = ref.norm64(y, err, None, None, 1e-5)[:2]
    ref.check(outs[0][0], want[0], ref.rounded(want, BF16, dy)[0])
