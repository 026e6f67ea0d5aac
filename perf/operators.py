"""The feed-forward operators' cases: inputs, a plain form in elementary torch operations, and
the calls of this package that compute the same.

Five kinds of pass:
  linear      Y = act(X W^T + b) + R, optionally also the pre-activation Z
  linear_bwd  its gradients dX, dW and db
  gated       H = act(X Wg^T + bg) * (X Wu^T + bu), optionally also G and U (the two pre-activations)
  gated_bwd   its gradients dX, dWg, dWu, dbg and dbu
  clip        the global 2-norm of many gradient tensors, and the tensors scaled by
              min(1, max_norm / (norm + eps))

`own` chooses between the plain form (False) and the package's kernels (True).  Operands whose
rows are not a multiple of 16 bytes are views of a buffer with padded rows, as the package's
matrix products ask for.
"""

import math

import torch

own = False

CLIP_EPS = 1e-6
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_GELU_C = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token through a down projection back onto the residual stream
        dict(name="linear decode 1", op="linear", M=1, N=4096, K=16384, dtype="bf16", act="none",
             bias=False, residual=True, save=False),
        # a short ragged prompt through a narrow layer whose sizes fill no tile
        dict(name="linear ragged 333", op="linear", M=333, N=1000, K=2056, dtype="f16", act="gelu",
             bias=True, residual=True, save=False),
        # a training batch through a square layer, pre-activation kept for the backward pass
        dict(name="linear train 8192", op="linear", M=8192, N=8192, K=8192, dtype="bf16",
             act="gelu_tanh", bias=True, residual=True, save=True),
        # gradients of a small fine-tuning batch; odd sizes
        dict(name="linear_bwd odd 509", op="linear_bwd", M=509, N=1001, K=777, dtype="f16",
             act="relu", bias=True),
        # gradients of an ordinary training batch
        dict(name="linear_bwd train 4096", op="linear_bwd", M=4096, N=8192, K=4096, dtype="bf16",
             act="gelu_tanh", bias=True),
        # one token through the gated projections
        dict(name="gated decode 1", op="gated", M=1, F=8192, K=4096, dtype="bf16", act="silu",
             bias=False, save=False),
        # a decode batch of 48 sequences
        dict(name="gated decode 48", op="gated", M=48, F=16384, K=4096, dtype="f16",
             act="gelu_tanh", bias=True, save=False),
        # a training batch, pre-activations kept
        dict(name="gated train 8192", op="gated", M=8192, F=16384, K=4096, dtype="bf16",
             act="silu", bias=False, save=True),
        # gradients of a small batch; odd sizes
        dict(name="gated_bwd odd 301", op="gated_bwd", M=301, F=1111, K=650, dtype="f16",
             act="gelu", bias=True),
        # gradients of the training batch
        dict(name="gated_bwd train 8192", op="gated_bwd", M=8192, F=16384, K=4096, dtype="bf16",
             act="silu", bias=False),
        # gradients of a small model: many little tensors of both widths
        dict(name="clip small", op="clip", tensors=48, elements=2_000_003, dtype="mixed"),
        # gradients of a block-sized shard in 16 bits
        dict(name="clip large", op="clip", tensors=24, elements=1_200_000_000, dtype="bf16"),
    ]


def _log_size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 64, of 8, or any."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((64, 8, 1, 1))
    if step > 1 and v >= 2 * step:
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    most_flops = max(work(c)["flops"] for c in listed())
    most_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd", "clip"))
        if op == "clip":
            case = dict(op=op, tensors=rng.randint(1, 60),
                        elements=int(math.exp(rng.uniform(math.log(1e4), math.log(1.2e9)))),
                        dtype=rng.choice(("mixed", "bf16", "f16", "f32")))
        else:
            case = dict(op=op, M=_log_size(rng, 1, 8192))
            case["N" if op.startswith("linear") else "F"] = _log_size(rng, 64, 16384)
            case["K"] = _log_size(rng, 64, 16384)
            case["dtype"] = rng.choice(("bf16", "f16"))
            case["act"] = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")
                                     if op.startswith("linear")
                                     else ("silu", "gelu", "gelu_tanh", "relu"))
            case["bias"] = rng.random() < 0.5
            if op == "linear":
                case["residual"] = rng.random() < 0.5
            if op in ("linear", "gated"):
                case["save"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] <= most_flops and w["bytes"] <= most_bytes:
            return case


def _clip_sizes(case):
    """Sizes of the case's tensors: a few large ones and many small ones, odd ones among them."""
    n, total = case["tensors"], case["elements"]
    weights = [1.0 / (1 + (7 * i) % n) for i in range(n)]
    s = sum(weights)
    sizes = [max(1, int(total * w / s)) for w in weights]
    sizes[0] = max(1, sizes[0] + total - sum(sizes))
    return sizes


def _clip_dtypes(case):
    if case["dtype"] == "mixed":
        return [(torch.float32, torch.bfloat16, torch.float16)[i % 3]
                for i in range(case["tensors"])]
    return [_DTYPES[case["dtype"]]] * case["tensors"]


def _normal(gen, rows, cols, dtype, scale=1.0):
    """rows x cols of N(0, scale^2), rows padded to 16 bytes."""
    pad = -(-cols // 8) * 8
    t = torch.randn((rows, pad), generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(scale).to(dtype)[:, :cols]


def _padded(rows, cols, dtype):
    return torch.empty((rows, -(-cols // 8) * 8), device="cuda", dtype=dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "clip":
        s["grads"] = []
        for i, (n, dt) in enumerate(zip(_clip_sizes(case), _clip_dtypes(case))):
            g = torch.empty(n, device="cuda", dtype=dt)
            g.normal_(0.0, 0.02 * (1 + i % 5), generator=gen)
            s["grads"].append(g)
        s["max_norm"] = 1.0
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        return s
    dt = _DTYPES[case["dtype"]]
    M, K = case["M"], case["K"]
    N = case["N"] if op.startswith("linear") else case["F"]
    s["X"] = _normal(gen, M, K, dt)
    weights = ("W",) if op.startswith("linear") else ("Wg", "Wu")
    for name in weights:
        s[name] = _normal(gen, N, K, dt, 1.0 / math.sqrt(K))
    if op in ("linear", "gated"):
        for name in (("b",) if op == "linear" else ("bg", "bu")):
            s[name] = _normal(gen, 1, N, dt, 0.5)[0].contiguous() if case["bias"] else None
        if op == "linear":
            s["R"] = _normal(gen, M, N, dt) if case["residual"] else None
            s["Y"] = _padded(M, N, dt)
            s["Z"] = _padded(M, N, dt) if case["save"] else None
        else:
            s["H"] = _padded(M, N, dt)
            s["G"] = _padded(M, N, dt) if case["save"] else None
            s["U"] = _padded(M, N, dt) if case["save"] else None
        return s
    # gradients arrive at the scale that a loss scale leaves them at
    s["dO"] = _normal(gen, M, N, dt, 0.25)
    for name in (("Z",) if op == "linear_bwd" else ("G", "U")):
        s[name] = _normal(gen, M, N, dt)
    s["dX"] = _padded(M, K, dt)
    for name in weights:
        s["d" + name] = _padded(N, K, dt)
        s["db" + name[1:]] = (torch.empty(N, device="cuda", dtype=torch.float32)
                              if case["bias"] else None)
    return s


# ---------------------------------------------------------------------------------- plain form


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(_GELU_C * (z + 0.044715 * z * z * z)))


def _dact(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) +
                z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    t = torch.tanh(_GELU_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _GELU_C * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    op = s["op"]
    if op == "clip":
        norm = torch.sqrt(sum((g.float() * g.float()).sum() for g in s["grads"]))
        coef = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
        return {"norm": norm, "grads": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}
    dt = s["X"].dtype
    X = s["X"].float()
    if op == "linear":
        Z = X @ s["W"].float().t()
        if s["b"] is not None:
            Z = Z + s["b"].float()
        Y = _act(s["act"], Z)
        if s["R"] is not None:
            Y = Y + s["R"].float()
        return {"Y": Y.to(dt), "Z": Z.to(dt) if s["Z"] is not None else None}
    if op == "gated":
        G = X @ s["Wg"].float().t()
        U = X @ s["Wu"].float().t()
        if s["bg"] is not None:
            G = G + s["bg"].float()
            U = U + s["bu"].float()
        H = _act(s["act"], G) * U
        keep = s["G"] is not None
        return {"H": H.to(dt), "G": G.to(dt) if keep else None, "U": U.to(dt) if keep else None}
    dO = s["dO"].float()
    if op == "linear_bwd":
        dZ = dO * _dact(s["act"], s["Z"].float())
        out = {"dX": (dZ @ s["W"].float()).to(dt), "dW": (dZ.t() @ X).to(dt)}
        out["db"] = dZ.sum(0) if s["db"] is not None else None
        return out
    G, U = s["G"].float(), s["U"].float()
    dU = dO * _act(s["act"], G)
    dG = dO * U * _dact(s["act"], G)
    out = {"dX": (dG @ s["Wg"].float() + dU @ s["Wu"].float()).to(dt),
           "dWg": (dG.t() @ X).to(dt), "dWu": (dU.t() @ X).to(dt)}
    out["dbg"] = dG.sum(0) if s["dbg"] is not None else None
    out["dbu"] = dU.sum(0) if s["dbu"] is not None else None
    return out


# ---------------------------------------------------------------------------- package's kernels


def _own(s):
    import implicit_gemm_conv_tcgen05_gb300 as igc
    op = s["op"]
    if op == "linear":
        igc.linear_act(s["X"], s["W"], bias=s["b"], act=s["act"], residual=s["R"], Y=s["Y"],
                       Z=s["Z"])
        return {"Y": s["Y"], "Z": s["Z"]}
    if op == "gated":
        igc.gated_ffn(s["X"], s["Wg"], s["Wu"], bg=s["bg"], bu=s["bu"], act=s["act"], H=s["H"],
                      G=s["G"], U=s["U"])
        return {"H": s["H"], "G": s["G"], "U": s["U"]}
    if op == "linear_bwd":
        igc.linear_act_backward(s["dO"], s["X"], s["W"], act=s["act"], Z=s["Z"], dX=s["dX"],
                                dW=s["dW"], dbias=s["db"])
        return {k: s[k] for k in ("dX", "dW", "db")}
    if op == "gated_bwd":
        igc.gated_ffn_backward(s["dO"], s["G"], s["U"], s["X"], s["Wg"], s["Wu"], act=s["act"],
                               dX=s["dX"], dWg=s["dWg"], dWu=s["dWu"], dbg=s["dbg"],
                               dbu=s["dbu"])
        return {k: s[k] for k in ("dX", "dWg", "dWu", "dbg", "dbu")}
    norm = igc.grad_norm_clip(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"])
    return {"norm": norm, "grads": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- 64-bit definition


def _act64(name, z):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[name](z)


def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = torch.zeros((), device="cuda", dtype=torch.float64)
        for g in s["grads"]:
            total += torch.linalg.vector_norm(g, dtype=torch.float64).square()
        norm = total.sqrt()
        coef = min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
        return {"norm": norm, "grads": [g.double() * coef for g in s["grads"]]}
    X = s["X"].double()
    if case["op"] == "linear":
        Z = torch.nn.functional.linear(X, s["W"].double(),
                                       None if s["b"] is None else s["b"].double())
        Y = _act64(case["act"], Z)
        return {"Y": Y if s["R"] is None else Y + s["R"].double(),
                "Z": Z if case["save"] else None}
    if case["op"] == "gated":
        G, U = (torch.nn.functional.linear(X, s["W" + c].double(),
                                           None if s["b" + c] is None else s["b" + c].double())
                for c in "gu")
        return {"H": _act64(case["act"], G) * U, "G": G if case["save"] else None,
                "U": U if case["save"] else None}
    dO = s["dO"].double()
    if case["op"] == "linear_bwd":
        Z = s["Z"].double().requires_grad_()
        _act64(case["act"], Z).backward(dO)
        dZ = Z.grad if case["act"] != "none" else dO
        return {"dX": torch.mm(dZ, s["W"].double()), "dW": torch.mm(dZ.t(), X),
                "db": dZ.sum(0) if case["bias"] else None}
    G, U = s["G"].double().requires_grad_(), s["U"].double().requires_grad_()
    (_act64(case["act"], G) * U).backward(dO)
    return {"dX": torch.mm(G.grad, s["Wg"].double()).addmm_(U.grad, s["Wu"].double()),
            "dWg": torch.mm(G.grad.t(), X), "dWu": torch.mm(U.grad.t(), X),
            "dbg": G.grad.sum(0) if case["bias"] else None,
            "dbu": U.grad.sum(0) if case["bias"] else None}


def work(case):
    op = case["op"]
    if op == "clip":
        size = {"f32": 4, "bf16": 2, "f16": 2}
        if case["dtype"] == "mixed":
            nbytes = sum(n * (4, 2, 2)[i % 3] for i, n in enumerate(_clip_sizes(case)))
        else:
            nbytes = case["elements"] * size[case["dtype"]]
        return {"bytes": 2 * nbytes, "flops": 3 * case["elements"]}
    M, K = case["M"], case["K"]
    if op == "linear":
        N = case["N"]
        elems = M * K + N * K + M * N * (1 + case["residual"] + case["save"]) + N * case["bias"]
        return {"bytes": 2 * elems, "flops": 2 * M * N * K}
    if op == "gated":
        F = case["F"]
        elems = M * K + 2 * F * K + M * F * (3 if case["save"] else 1) + 2 * F * case["bias"]
        return {"bytes": 2 * elems, "flops": 4 * M * F * K}
    if op == "linear_bwd":
        N = case["N"]
        elems = M * N * (1 if case["act"] == "none" else 2) + 2 * (M * K + N * K)
        return {"bytes": 2 * elems + 4 * N * case["bias"], "flops": 4 * M * N * K}
    F = case["F"]
    elems = 3 * M * F + 2 * (M * K + 2 * F * K)
    return {"bytes": 2 * elems + 8 * F * case["bias"], "flops": 8 * M * F * K}
