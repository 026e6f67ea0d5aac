"""64-bit forms of the feed-forward operators and the error bounds of the kernels, shared
by their tests.

Bounds.  u is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16; fp16 values
below 2^-14 have spacing 2^-24).  A product sum of K terms in fp32 with truncating
additions is off by at most gamma = (K + 8) 2^-23 of sum |x w|.  The activations use
approximate exponentials (2^-22, and |x| 2^-23 from the rounded argument), reciprocals
(2^-23) and erff (2 ulp): their value is off by at most 1e-5 |z|, their derivative by at
most 1e-5 (1 + |z|), where the sigmoid exceeds 1e-17; below that both are far under the
other terms.  The slopes of
the activations are at most 1.13.
"""

import math

import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
SLOPE = 1.13
ACT_ERR = 1e-5


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + \
            z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def gamma(k):
    return (k + 8) * 2.0 ** -23


def rounded(ref, err, dtype):
    """The bound after rounding a value within err of ref to dtype."""
    return err + UNIT[dtype] * (ref.abs() + err) + TINY[dtype]


def preact(x, w, b):
    """Z = x w^T + b in 64 bits and the bound of its fp32 sum."""
    z = x @ w.t()
    err = gamma(x.shape[1]) * (x.abs() @ w.abs().t())
    if b is not None:
        z = z + b
        err = err + 2.0 ** -24 * (z.abs() + err)
    return z, err


def linear(x, w, b, name, r, out_dtype, z_dtype):
    """(Y, bound), (Z, bound)."""
    z, ez = preact(x, w, b)
    y = act(name, z)
    ey = SLOPE * ez + ACT_ERR * z.abs()
    if r is not None:
        y = y + r
        ey = ey + 2.0 ** -23 * (y.abs() + r.abs())
    return (y, rounded(y, ey, out_dtype)), (z, rounded(z, ez, z_dtype))


def gated(x, wg, wu, bg, bu, name, dtype):
    """(H, bound), (G, bound), (U, bound)."""
    g, eg = preact(x, wg, bg)
    u, eu = preact(x, wu, bu)
    f = act(name, g)
    ef = SLOPE * eg + ACT_ERR * g.abs()
    h = f * u
    eh = ef * u.abs() + (f.abs() + ef) * eu + 2.0 ** -23 * h.abs()
    return (h, rounded(h, eh, dtype)), (g, rounded(g, eg, dtype)), (u, rounded(u, eu, dtype))


def grads(ds, es, x, ws, in_dtype, dw_dtype, db_dtype):
    """From the pre-activation gradients ds (64 bits, off by at most es in fp32): the
    lists [(dX, bound)], [(dW, bound)], [(db, bound)].  The products take ds rounded to
    in_dtype; the sums of db take them in fp32."""
    rows = ds[0].shape[0]
    eds = [e + UNIT[in_dtype] * (d.abs() + e) + TINY[in_dtype] for d, e in zip(ds, es)]
    dx = sum(d @ w for d, w in zip(ds, ws))
    k = sum(d.shape[1] for d in ds)
    ex = sum(e @ w.abs() + gamma(k) * ((d.abs() + e) @ w.abs()) for d, e, w in zip(ds, eds, ws))
    dws, dbs = [], []
    for d, e0, e in zip(ds, es, eds):
        dw = d.t() @ x
        ew = e.t() @ x.abs() + gamma(rows) * ((d.abs() + e).t() @ x.abs())
        dws.append((dw, rounded(dw, ew, dw_dtype)))
        db = d.sum(0)
        eb = e0.sum(0) + gamma(rows) * d.abs().sum(0)
        dbs.append((db, rounded(db, eb, db_dtype)))
    return [(dx, rounded(dx, ex, in_dtype))], dws, dbs


def linear_dz(dy, z, name):
    """dZ and the bound of its fp32 value."""
    dz = dy * act_grad(name, z)
    return dz, dy.abs() * ACT_ERR * (1 + z.abs()) * (name != "none") + 2.0 ** -23 * dz.abs()


def gated_dgu(dh, g, u, name):
    """[dG, dU] and the bounds of their fp32 values."""
    du = dh * act(name, g)
    dg = dh * u * act_grad(name, g)
    eu = dh.abs() * ACT_ERR * g.abs() + 2.0 ** -23 * du.abs()
    eg = (dh * u).abs() * ACT_ERR * (1 + g.abs()) + 2.0 ** -22 * dg.abs()
    return [dg, du], [eg, eu]


def check(got, want, what):
    ref, bound = want
    got = got.double()
    assert got.shape == ref.shape, what
    off = (got - ref).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = int(torch.argmax((off / bound).nan_to_num(nan=float("inf"))).item())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst "
                             f"at {i}: {got.flatten()[i].item()} for {ref.flatten()[i].item()}, "
                             f"bound {bound.flatten()[i].item()}")
