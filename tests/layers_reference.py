"""64-bit forms of the layer operators (embedding, layer norm, dropout) and the bounds that their
fp32 arithmetic and one rounding keep, shared by the tests."""

import zlib

import numpy as np
import torch

E32 = 2.0 ** -24                      # half a step of fp32, relative
DEPTH = 64                            # additions between a row's element and its sum, at most
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the step of the type's subnormals."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def threshold(p):
    return round((1.0 - p) * 65536)


def philox(counter, key):
    """Philox4x32-10 on four arrays of 32-bit words (uint64 arrays)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def keep(M, N, p, seed, offset):
    """M x N truth values (CPU)."""
    i, j = np.meshgrid(np.arange(M), np.arange((N + 7) // 8), indexing="ij")
    zero = np.zeros_like(i)
    w = philox((j, i, zero + offset % 2 ** 32, zero + offset // 2 ** 32),
               (seed % 2 ** 32, seed // 2 ** 32))
    halves = [h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))]
    bits = np.stack(halves, axis=2).reshape(M, -1)[:, :N]
    return torch.from_numpy(bits < threshold(p))


def drop64(x, p, seed, offset):
    x = x.double()
    T = threshold(p)
    if T == 65536:
        return x
    mask = keep(x.shape[0], x.shape[1], p, seed, offset).to(x.device)
    return torch.where(mask, x * (65536.0 / T if T else 0.0), torch.zeros_like(x))


def check(got, want, bound, what=""):
    """Every element within its bound; NaN and infinities where they are wanted."""
    got = got.double()
    finite = want.isfinite()
    assert bool((got.isnan() == want.isnan()).all()), f"{what}: NaN"
    inf = want.isinf()
    assert bool((got[inf] == want[inf]).all()), f"{what}: infinities"
    off = (got - want).abs()
    over = finite & ~(off <= bound)
    if bool(over.any()):
        at = int(torch.where(over.flatten())[0][0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside, first at {at}: "
                             f"{float(got.flatten()[at])} for {float(want.flatten()[at])}, bound "
                             f"{float(bound.expand_as(want).flatten()[at]):.3g}")


def rounded(want, dtype, err):
    """The bound of a value that is off by err before it is rounded to dtype."""
    return err + (want.abs() + err) * unit(dtype) + least(dtype)


def dropout64(X, p, seed, offset, R):
    """(Y, its fp32 error): a product with a scale that is itself rounded, and a sum."""
    d = drop64(X, p, seed, offset)
    if R is None:
        return d, 2.1 * E32 * d.abs()
    y = R.double() + d
    return y, 2.1 * E32 * d.abs() + 1.1 * E32 * (y.abs() + d.abs() * 2 * E32)


def norm64(S, err, w, b, eps):
    """(Y, its fp32 error, mean, its error, rstd, its error) of rows S that are off by err."""
    mean = S.mean(1, keepdim=True)
    d = S - mean
    var = d.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    worst = err.amax(1, keepdim=True)
    dm = (DEPTH + 2) * E32 * S.abs().mean(1, keepdim=True) + worst
    dd = dm + worst + E32 * (d.abs() + dm)                      # of d
    dmax = dd.amax(1, keepdim=True)
    dvar = 2 * var.sqrt() * dmax + dmax.square() + (DEPTH + 2) * E32 * var
    rho = 0.5 * dvar / (var + eps) * 1.1 + 4 * E32              # of rstd, relative
    w = torch.ones_like(S[0]) if w is None else w.double()
    b = torch.zeros_like(S[0]) if b is None else b.double()
    h = d * rstd
    y = h * w + b
    dy = w.abs() * (rstd * (1 + rho) * dd + h.abs() * (rho + 3 * E32)) + 2 * E32 * y.abs()
    return y, dy, mean[:, 0], dm[:, 0], rstd[:, 0], (rstd * rho)[:, 0]


def norm_backward64(dY, S, mean, rstd, w, A):
    """(dS, its fp32 error, dw, its error, db, its error) for the statistics given."""
    dY, S = dY.double(), S.double()
    M, N = dY.shape
    m, r = mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(N, dtype=torch.float64, device=dY.device) if w is None else w.double()
    h = (S - m) * r
    g = dY * w
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    inner = g - c1 - h * c2
    dS = r * inner + (0 if A is None else A.double())
    size = g.abs() + c1.abs() + (h * c2).abs()
    e1 = (DEPTH + 3) * E32 * g.abs().mean(1, keepdim=True)
    e2 = (DEPTH + 6) * E32 * (g * h).abs().mean(1, keepdim=True)
    err = r * (e1 + h.abs() * e2 * 1.01 + 7 * E32 * size) + 2 * E32 * dS.abs()
    # a sum of M terms in any order: at most M - 1 roundings on the way of each
    t = dY * h
    return (dS, err, t.sum(0), (M + 4) * E32 * t.abs().sum(0), dY.sum(0),
            M * E32 * dY.abs().sum(0))


def lookup64(tokens, W, scale):
    inside = (tokens >= 0) & (tokens < W.shape[0])
    y = torch.zeros((tokens.numel(), W.shape[1]), dtype=torch.float64, device=W.device)
    y[inside] = W.double()[tokens[inside].long()] * scale
    return y


def lookup_backward64(tokens, dY, V, scale):
    """(dW, its fp32 error)."""
    inside = (tokens >= 0) & (tokens < V)
    at = tokens[inside].long()
    rows = dY.double()[inside]
    dW = torch.zeros((V, dY.shape[1]), dtype=torch.float64, device=dY.device)
    size, count = torch.zeros_like(dW), torch.zeros((V, 1), dtype=torch.float64, device=dY.device)
    dW.index_add_(0, at, rows)
    size.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones((at.numel(), 1), dtype=torch.float64, device=dY.device))
    return dW * scale, (count + 1) * E32 * size * abs(scale) * 1.01


def generator(*key):
    """A generator of values on the GPU, seeded by what it is for."""
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def matrix(gen, rows, cols, dtype, scale=1.0, mean=0.0, pad=None, shift=0, device="cuda"):
    """rows x cols of normal values, as a view of rows that are padded to a multiple of 8
    (pad=None) or by `pad` elements, starting `shift` elements into its buffer."""
    ld = -(-cols // 8) * 8 if pad is None else cols + pad
    buf = torch.full((rows * ld + shift + 8,), 77.0, device=device, dtype=dtype)
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.randn((rows, cols), generator=gen, device=device) * scale + mean)
    return view


def around(view):
    """The elements between the rows of a view made by matrix (its padding)."""
    rows, cols = view.shape
    ld = view.stride(0)
    return view.as_strided((rows - 1, ld - cols), (ld, 1), view.storage_offset() + cols) \
        if rows > 1 and ld > cols else view.new_empty((0,))
