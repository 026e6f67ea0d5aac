"""Cases of the operators around the feed-forward products in a training step (embedding, layer
norm, dropout): inputs, a plain form in elementary torch operations, and the calls of this package
that compute the same.

Five kinds of pass:
  norm        S = R + drop(X) and Y = (S - mean) rstd w + b over the rows of S
  norm_bwd    dS (with the gradient that reaches S past the norm added), dX through the dropout,
              dw and db
  dropout     Y = R + drop(X), or drop(X) alone
  lookup      Y[i] = scale W[token[i]]; a token outside the table gives a row of zeros
  lookup_bwd  dW[v] = scale * sum of dY[i] over the positions i that hold token v

drop(X) keeps an element with probability T / 65536, T = (1 - p) 65536 rounded to an integer, and
scales what it keeps by 65536 / T.  Which ones it keeps follows from (seed, offset, row, column)
by the counter-based generator Philox4x32-10, so no mask is an input or an output.

`own` chooses between the plain form (False) and the package's kernels (True).  Rows are padded to
a multiple of 16 bytes, as the package's matrix products ask for.
"""

import math

import torch

own = False

EPS = 1e-5
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token of a generated text: the branch joins the residual stream and is normalised
        dict(name="norm decode 1", op="norm", M=1, N=4096, dtype="bf16", stream="bf16",
             residual=True, p=0.0, train=False),
        # a short ragged prompt, odd width, residual stream kept in fp32
        dict(name="norm ragged 333", op="norm", M=333, N=1001, dtype="f16", stream="f32",
             residual=True, p=0.0, train=True),
        # a training batch: dropout on the branch, sum, norm, statistics kept
        dict(name="norm train 16384", op="norm", M=16384, N=4096, dtype="bf16", stream="bf16",
             residual=True, p=0.1, train=True),
        # gradients of a small fine-tuning batch; odd sizes
        dict(name="norm_bwd odd 509", op="norm_bwd", M=509, N=777, dtype="f16", stream="f16",
             add=False, p=0.0),
        # gradients of the training batch
        dict(name="norm_bwd train 16384", op="norm_bwd", M=16384, N=4096, dtype="bf16",
             stream="bf16", add=True, p=0.1),
        # gradients of a narrow model's long batch, residual stream in fp32
        dict(name="norm_bwd narrow 65536", op="norm_bwd", M=65536, N=512, dtype="bf16",
             stream="f32", add=True, p=0.0),
        # the branch of a small batch onto its residual stream
        dict(name="dropout small 48", op="dropout", M=48, N=4096, dtype="bf16", stream="bf16",
             residual=True, p=0.1),
        # a training batch through a wide layer
        dict(name="dropout train 16384", op="dropout", M=16384, N=8192, dtype="bf16",
             stream="bf16", residual=True, p=0.1),
        # one token for each of 64 sequences that are being generated
        dict(name="lookup decode 64", op="lookup", M=64, V=131072, D=4096, dtype="bf16",
             stream="bf16", pad=False),
        # a training batch
        dict(name="lookup train 32768", op="lookup", M=32768, V=131072, D=4096, dtype="bf16",
             stream="bf16", pad=True),
        # gradients of a small fine-tuning batch; odd sizes
        dict(name="lookup_bwd odd 509", op="lookup_bwd", M=509, V=5003, D=777, dtype="f16",
             dw="f32", pad=True),
        # gradients of the training batch
        dict(name="lookup_bwd train 32768", op="lookup_bwd", M=32768, V=131072, D=4096,
             dtype="bf16", dw="bf16", pad=False),
    ]


def _log_size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 64, of 8, or any."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((64, 8, 1, 1))
    if step > 1 and v >= 2 * step:
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("norm", "norm_bwd", "norm_bwd", "dropout", "lookup", "lookup_bwd"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        case = dict(op=op, M=_log_size(rng, 1, 65536))
        if op.startswith("lookup"):
            case.update(V=_log_size(rng, 1000, 200000), D=_log_size(rng, 64, 8192))
        else:
            case.update(N=_log_size(rng, 64, 16384), p=rng.choice((0.0, 0.1, 0.25)))
        case["dtype"] = dtype
        if op == "lookup_bwd":
            case["dw"] = rng.choice((dtype, "f32"))
        else:
            case["stream"] = rng.choice((dtype, "f32"))
        if op.startswith("lookup"):
            case["pad"] = rng.random() < 0.5
        elif op == "norm_bwd":
            case["add"] = rng.random() < 0.5
        else:
            case["residual"] = rng.random() < 0.7
            if op == "norm":
                case["train"] = rng.random() < 0.5
            elif case["p"] == 0.0:
                case["p"] = 0.1
        if work(case)["bytes"] <= most:
            return case


def _padded(rows, cols, dtype):
    return torch.empty((rows, -(-cols // 8) * 8), device="cuda", dtype=dtype)[:, :cols]


def _normal(gen, rows, cols, dtype, scale=1.0, mean=0.0):
    t = _padded(rows, cols, dtype)
    t.normal_(mean, scale, generator=gen)
    return t


def _tokens(case, gen):
    """Token ids, a few of them frequent and most of them rare: id k - 1 with a probability near
    that of k = floor(exp(u log(V + 1))), u uniform, which falls as 1 / k.  With `pad`, every
    eighth sequence of 64 positions ends in 24 positions of padding (-1)."""
    M, V = case["M"], case["V"]
    u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
    tok = (torch.exp(u * math.log(V + 1)).long() - 1).clamp_(0, V - 1)
    if case["pad"]:
        at = torch.arange(M, device="cuda")
        tok = torch.where(((at // 64) % 8 == 0) & (at % 64 >= 40), -1, tok)
    return tok


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op, M = case["op"], case["M"]
    dt = _DTYPES[case["dtype"]]
    if op == "lookup":
        s["tokens"] = _tokens(case, gen)
        s["scale"] = math.sqrt(case["D"])
        s["W"] = _normal(gen, case["V"], case["D"], dt, 1.0 / s["scale"])
        s["Y"] = _padded(M, case["D"], _DTYPES[case["stream"]])
        return s
    if op == "lookup_bwd":
        s["tokens"] = _tokens(case, gen)
        s["scale"] = math.sqrt(case["D"])
        s["dY"] = _normal(gen, M, case["D"], dt, 0.25)
        s["dW"] = _padded(case["V"], case["D"], _DTYPES[case["dw"]])
        return s
    N = case["N"]
    st = _DTYPES[case["stream"]]
    s["seed"] = 0x9E3779B97F4A7C15 * (int(seed) + 1) & (2**64 - 1)   # of the dropout
    s["offset"] = 7 * int(seed) + 5                                  # (a step of the training)
    if op == "dropout":
        s["X"] = _normal(gen, M, N, dt)
        s["R"] = _normal(gen, M, N, st, 2.0) if case["residual"] else None
        s["Y"] = _padded(M, N, st)
        return s
    s["w"] = torch.empty(N, device="cuda").normal_(1.0, 0.2, generator=gen)
    if op == "norm":
        # without a residual the input is the stream itself, unless dropout comes first
        s["X"] = _normal(gen, M, N, dt if case["residual"] or case["p"] else st, 1.0, 0.1)
        s["b"] = torch.empty(N, device="cuda").normal_(0.0, 0.2, generator=gen)
        s["R"] = _normal(gen, M, N, st, 2.0) if case["residual"] else None
        joined = case["residual"] or case["p"] > 0
        s["S"] = _padded(M, N, st if case["residual"] else s["X"].dtype) if joined else None
        s["Y"] = _padded(M, N, dt)
        for name in ("mean", "rstd"):
            s[name] = torch.empty(M, device="cuda") if case["train"] else None
        return s
    s["dY"] = _normal(gen, M, N, dt, 0.25)
    s["S"] = _normal(gen, M, N, st, 2.0, 0.3)
    # the statistics that the forward pass kept
    rows = s["S"].float()
    s["mean"] = rows.mean(1)
    s["rstd"] = 1.0 / torch.sqrt((rows - s["mean"][:, None]).square().mean(1) + EPS)
    s["add_to"] = _normal(gen, M, N, st, 0.25) if case["add"] else None
    s["dS"] = _padded(M, N, st)
    s["dX"] = _padded(M, N, dt) if case["p"] > 0 or st != dt else None
    s["dw"], s["db"] = (torch.empty(N, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------------------------- plain form


def _threshold(p):
    return round((1.0 - p) * 65536.0)


def _keep(M, N, p, seed, offset):
    """M x N truth values: Philox4x32-10 on the counter (column / 8, row, offset), keyed by the
    seed; the eight 16-bit halves of its four words, low half first, for eight columns."""
    mask = 0xFFFFFFFF
    c = [torch.arange(-(-N // 8), device="cuda").expand(M, -1),
         torch.arange(M, device="cuda")[:, None].expand(-1, -(-N // 8)),
         torch.full((1, 1), offset & mask, device="cuda"),
         torch.full((1, 1), offset >> 32, device="cuda")]
    k0, k1 = seed & mask, seed >> 32
    for _ in range(10):
        a = c[0] * 0xD2511F53          # (wraps past 2^63: the bits are those of the product)
        b = c[2] * 0xCD9E8D57
        c = [((b >> 32) & mask) ^ c[1] ^ k0, b & mask, ((a >> 32) & mask) ^ c[3] ^ k1, a & mask]
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    T = _threshold(p)
    bits = [h for word in c for h in (word & 0xFFFF, word >> 16)]
    keep = [(h < T).expand(M, -(-N // 8)) for h in bits]
    return torch.stack(keep, dim=2).reshape(M, -1)[:, :N]


def _drop(x, s):
    """drop(x) in fp32."""
    if s["p"] == 0.0:
        return x
    T = _threshold(s["p"])
    keep = _keep(x.shape[0], x.shape[1], s["p"], s["seed"], s["offset"])
    return torch.where(keep, x * (65536.0 / T), torch.zeros_like(x))


def _plain(s):
    op = s["op"]
    if op in ("lookup", "lookup_bwd"):
        tok = s["tokens"]
        inside = (tok >= 0) & (tok < s["V"])
        if op == "lookup":
            rows = s["W"][torch.where(inside, tok, 0)].float() * s["scale"]
            return torch.where(inside[:, None], rows, torch.zeros_like(rows)).to(s["Y"].dtype)
        dW = torch.zeros((s["V"], s["D"]), device="cuda")
        dW.index_add_(0, tok[inside], s["dY"][inside].float())
        return (dW * s["scale"]).to(s["dW"].dtype)
    if op == "dropout":
        Y = _drop(s["X"].float(), s)
        return (Y if s["R"] is None else s["R"].float() + Y).to(s["Y"].dtype)
    w = s["w"]
    if op == "norm":
        S = _drop(s["X"].float(), s)
        if s["R"] is not None:
            S = s["R"].float() + S
        mean = S.mean(1)
        rstd = 1.0 / torch.sqrt((S - mean[:, None]).square().mean(1) + EPS)
        Y = (S - mean[:, None]) * rstd[:, None] * w + s["b"]
        return {"Y": Y.to(s["Y"].dtype), "S": None if s["S"] is None else S.to(s["S"].dtype),
                "mean": mean if s["train"] else None, "rstd": rstd if s["train"] else None}
    rstd = s["rstd"][:, None]
    h = (s["S"].float() - s["mean"][:, None]) * rstd
    dY = s["dY"].float()
    g = dY * w
    dS = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if s["add_to"] is not None:
        dS = dS + s["add_to"].float()
    out = {"dS": dS.to(s["dS"].dtype), "dw": (dY * h).sum(0), "db": dY.sum(0)}
    out["dX"] = None if s["dX"] is None else _drop(dS, s).to(s["dX"].dtype)
    return out


# ---------------------------------------------------------------------------- package's kernels


def _own(s):
    import implicit_gemm_conv_tcgen05_gb300 as igc
    op = s["op"]
    if op == "lookup":
        return igc.embedding_lookup(s["tokens"], s["W"], scale=s["scale"], Y=s["Y"])
    if op == "lookup_bwd":
        return igc.embedding_backward(s["tokens"], s["dY"], scale=s["scale"], dW=s["dW"])
    if op == "dropout":
        return igc.dropout_add(s["X"], s["p"], seed=s["seed"], offset=s["offset"],
                               residual=s["R"], Y=s["Y"])
    if op == "norm":
        igc.layer_norm(s["X"], s["w"], s["b"], eps=EPS, residual=s["R"], p=s["p"],
                       seed=s["seed"], offset=s["offset"], Y=s["Y"], S=s["S"], mean=s["mean"],
                       rstd=s["rstd"])
        return {k: s[k] for k in ("Y", "S", "mean", "rstd")}
    igc.layer_norm_backward(s["dY"], s["S"], s["mean"], s["rstd"], s["w"], dS_add=s["add_to"],
                            p=s["p"], seed=s["seed"], offset=s["offset"], dS=s["dS"], dX=s["dX"],
                            dw=s["dw"], db=s["db"])
    return {k: s[k] for k in ("dS", "dw", "db", "dX")}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- 64-bit definition


def _mul32(a, m):
    """High and low 32 bits of a * m for tensors a of 32-bit values, by 16-bit halves."""
    al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = ah * ml + ((al * ml) >> 16)
    cross = al * mh + (mid & 0xFFFF)
    high = ah * mh + (mid >> 16) + (cross >> 16)
    return high, ((cross & 0xFFFF) << 16) | ((al * ml) & 0xFFFF)


def _factors64(case, s, M, N):
    """What drop multiplies by: 0 or 65536 / T, in 64 bits, row block by row block."""
    T = _threshold(case["p"])
    if T == 65536:
        return torch.ones((1, 1), device="cuda", dtype=torch.float64)
    out = torch.empty((M, N), device="cuda", dtype=torch.float64)
    blocks = (N + 7) // 8
    step = max(1, (1 << 24) // blocks)
    for r0 in range(0, M, step):
        rows = torch.arange(r0, min(M, r0 + step), device="cuda").repeat_interleave(blocks)
        x0 = torch.arange(blocks, device="cuda").repeat(rows.numel() // blocks)
        x1 = rows
        x2 = torch.full_like(x0, s["offset"] % 2**32)
        x3 = torch.full_like(x0, s["offset"] // 2**32)
        for r in range(10):
            key0 = (s["seed"] % 2**32 + r * 0x9E3779B9) % 2**32
            key1 = (s["seed"] // 2**32 + r * 0xBB67AE85) % 2**32
            h0, l0 = _mul32(x0, 0xD2511F53)
            h1, l1 = _mul32(x2, 0xCD9E8D57)
            x0, x1, x2, x3 = h1 ^ x1 ^ key0, l1, h0 ^ x3 ^ key1, l0
        n = rows.numel() // blocks
        for i, word in enumerate((x0, x1, x2, x3)):
            for half in range(2):
                col = 2 * i + half
                if col < N:
                    v = ((word >> (16 * half)) % 65536).view(n, blocks) < T
                    cols = out[r0:r0 + n, col::8]
                    cols.copy_(v[:, :cols.shape[1]])
    return out.mul_(65536.0 / T)


def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    f = torch.nn.functional
    if op == "lookup":
        table = torch.cat([s["W"].double() * s["scale"],
                           torch.zeros((1, case["D"]), device="cuda", dtype=torch.float64)])
        tok = s["tokens"]
        return table[torch.where((tok < 0) | (tok >= case["V"]), case["V"], tok)]
    if op == "lookup_bwd":
        tok = s["tokens"]
        order = torch.argsort(torch.where((tok < 0) | (tok >= case["V"]), case["V"], tok),
                              stable=True)
        ids, counts = torch.unique_consecutive(tok[order], return_counts=True)
        dW = torch.zeros((case["V"], case["D"]), device="cuda", dtype=torch.float64)
        rows = s["dY"][order].double()
        sums = torch.segment_reduce(rows, "sum", lengths=counts, axis=0)
        good = (ids >= 0) & (ids < case["V"])
        dW[ids[good]] = sums[good] * s["scale"]
        return dW
    N = case["N"]
    if op == "dropout":
        Y = s["X"].double() * _factors64(case, s, M, N)
        return Y if s["R"] is None else Y.add_(s["R"].double())
    if op == "norm":
        S = s["X"].double() * _factors64(case, s, M, N)
        if s["R"] is not None:
            S += s["R"].double()
        var, mean = torch.var_mean(S, dim=1, correction=0)
        return {"Y": f.layer_norm(S, (N,), s["w"].double(), s["b"].double(), EPS),
                "S": S if s["S"] is not None else None,
                "mean": mean if case["train"] else None,
                "rstd": torch.rsqrt(var + EPS) if case["train"] else None}
    # The statistics are inputs: dS is the derivative of the norm with what they depend on, written
    # with them.  The rows' products are taken by matrix products here.
    D = torch.float64
    dY = s["dY"].to(D)
    h = torch.addcmul(torch.zeros((), device="cuda", dtype=D),
                      s["S"].to(D) - s["mean"].to(D).unsqueeze(1), s["rstd"].to(D).unsqueeze(1))
    ones = torch.ones(max(M, N), device="cuda", dtype=D)
    out = {"db": dY.t() @ ones[:M], "dw": torch.einsum("ij,ij->j", dY, h)}
    g = dY * s["w"].to(D)
    dS = (g - (g @ ones[:N] / N).unsqueeze(1) -
          h * (torch.einsum("ij,ij->i", g, h) / N).unsqueeze(1)) * s["rstd"].to(D).unsqueeze(1)
    if s["add_to"] is not None:
        dS += s["add_to"].to(D)
    out["dX"] = None if s["dX"] is None else dS * _factors64(case, s, M, N)
    return {"dS": dS, "dw": out["dw"], "db": out["db"], "dX": out["dX"]}


def _distinct(case):
    """Expected number of different tokens among a lookup's positions."""
    V, M = case["V"], case["M"]
    total, k, log_v = 0.0, 1, math.log(V + 1)
    while k <= V:
        # runs of ids grow with k: their probabilities differ little
        n = min(max(1, k // 64), V + 1 - k)
        prob = math.log((k + n) / k) / log_v / n
        total += n * -math.expm1(M * math.log1p(-min(prob, 0.999999)))
        k += n
    return min(total, float(M))


def work(case):
    op, M = case["op"], case["M"]
    own_size = _SIZE[case["dtype"]]
    if op == "lookup":
        rows = _distinct(case) * own_size + M * _SIZE[case["stream"]]
        return {"bytes": int(8 * M + rows * case["D"]), "flops": M * case["D"]}
    if op == "lookup_bwd":
        return {"bytes": 8 * M + M * case["D"] * own_size + case["V"] * case["D"] * _SIZE[case["dw"]],
                "flops": M * case["D"]}
    N, st = case["N"], _SIZE[case["stream"]]
    if op == "dropout":
        return {"bytes": M * N * (own_size + st * (1 + case["residual"])), "flops": 2 * M * N}
    if op == "norm":
        if case["residual"]:
            per = 2 * own_size + 2 * st
        else:
            per = own_size + (2 * own_size if case["p"] > 0 else st)
        return {"bytes": M * N * per + 8 * N + 8 * M * case["train"], "flops": 8 * M * N}
    extra = case["p"] > 0 or case["stream"] != case["dtype"]
    per = own_size * (1 + extra) + st * (2 + case["add"])
    return {"bytes": M * N * per + 12 * N + 8 * M, "flops": 14 * M * N}
