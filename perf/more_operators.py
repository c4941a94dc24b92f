"""The dense operators around the experts and the attention as measured workloads: root-mean-square norm with the
residual's addition and 8-bit rows, the product of 8-bit integers with scales for each token and channel, and log
probabilities of given tokens with entropy and top alternatives.

Every case is run in two forms on the same inputs: `own` false computes it with elementary torch operations in fp32,
`own` true calls this package.  Rows held in 8 bits are int8 (rows, d) with an fp32 scale per row; they are returned as the
values they stand for.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases


def listed():
    return [
        # norm --------------------------------------------------------------------------------
        # a decode step of 8 sequences: add the layer's output, normalise, 8-bit rows for the next projection
        dict(name="norm_step", op="norm", dtype="bf16", T=8, d=4096, residual=True, q8=True, pad=0),
        # the same for a prompt
        dict(name="norm_prompt", op="norm", dtype="bf16", T=8192, d=4096, residual=True, q8=True, pad=0),
        # what the router and the experts read: 16-bit rows, an odd count, the input inside a wider tensor
        dict(name="norm_experts", op="norm", dtype="f16", T=2501, d=2048, residual=True, q8=False, pad=1024),
        # products ----------------------------------------------------------------------------
        # q, k and v of one token (latency)
        dict(name="linear_one", op="linear", dtype="bf16", M=1, N=6144, K=4096, quantize=False, bias=False),
        # a batch's attention output: 8-bit rows, then the output projection
        dict(name="linear_batch", op="linear", dtype="f16", M=24, N=4096, K=4096, quantize=True, bias=True),
        # trees of drafted tokens
        dict(name="linear_tree", op="linear", dtype="bf16", M=300, N=6144, K=2048, quantize=False, bias=False),
        # a prompt's q, k and v (compute)
        dict(name="linear_prompt", op="linear", dtype="bf16", M=8192, N=6144, K=4096, quantize=False, bias=False),
        # odd sizes, fp32 results
        dict(name="linear_odd", op="linear", dtype="f32", M=1111, N=5001, K=1408, quantize=False, bias=True),
        # scores ------------------------------------------------------------------------------
        # one row: a sampler's step (latency)
        dict(name="score_one", op="score", dtype="f32", T=1, V=32000, ids=1, k=8, pad=0),
        # verification of drafted trees: a row's children in the tree, and what the model would have taken
        dict(name="score_trees", op="score", dtype="bf16", T=320, V=131072, ids=3, k=8, pad=0),
        # a prompt's own tokens, a vocabulary of odd size inside padded rows
        dict(name="score_prompt", op="score", dtype="bf16", T=4096, V=65521, ids=1, k=5, pad=15),
        # the end of a step: logits of 8-bit hidden rows, then their scores
        dict(name="head", op="head", dtype="f32", M=40, N=32768, K=2048, ids=1, k=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "score", "score", "head"])
    if op == "norm":
        d = rng.choice([64, 128, 256, 1024, 1408, 2048, 2560, 4096, 5120, 8192, _log(rng, 100, 8192)])
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "bf16", "f32"]), T=_log(rng, 1, 16000000 // d), d=d,
                    residual=rng.random() < 0.7, q8=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 512]))
    if op == "linear":
        M, N = _log(rng, 1, 8192), rng.choice([256, 1024, 2048, 4096, 6144, _log(rng, 16, 8192)])
        K = rng.choice([256, 1024, 1408, 2048, 4096, 16 * rng.randint(4, 256), rng.randint(64, 4096), 5632])
        quantize = rng.random() < 0.3           # then results are 16-bit like the rows that come in
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "bf16", "bf16" if quantize else "f32"]),
                    M=min(M, 8192 * 6144 * 4096 // (N * K)), N=N, K=K, quantize=quantize, bias=rng.random() < 0.4)
    if op == "score":
        V = rng.choice([32000, 65536, 131072, _log(rng, 1000, 131072)])
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), T=_log(rng, 1, 120000000 // V), V=V, ids=_log(rng, 1, 8),
                    k=rng.choice([0, 1, 5, 8, 20]), pad=rng.choice([0, 0, 8, 5]))
    return dict(op=op, dtype="f32", M=_log(rng, 1, 256), N=_log(rng, 2000, 40000), K=rng.choice([1024, 1408, 2048, 4096]),
                ids=rng.choice([1, 4]), k=rng.choice([1, 8, 20]))


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    c, es = case, _size(case["dtype"])
    if c["op"] == "norm":                       # x, residual, weight in; the sum and the normalised rows out
        row = es * (1 + 2 * c["residual"]) + (2 if c["q8"] else es)
        return {"bytes": c["T"] * c["d"] * row + c["d"] * es, "flops": 6 * c["T"] * c["d"]}
    if c["op"] == "score":
        return {"bytes": c["T"] * (c["V"] * es + 4 * (2 * c["ids"] + 1 + 2 * c["k"])), "flops": 6 * c["T"] * c["V"]}
    M, N, K = c["M"], c["N"], c["K"]
    bytes_ = M * K + N * K + 4 * (M + N)
    if c["op"] == "head":                       # the logits need not leave the chip
        return {"bytes": bytes_ + 4 * M * (2 * c["ids"] + 1 + 2 * c["k"]), "flops": 2 * M * N * K}
    return {"bytes": bytes_ + M * K * (es if c["quantize"] else 0) + M * N * es + 4 * N * c["bias"], "flops": 2 * M * N * K}


# ---------------------------------------------------------------- inputs


def _rows8(v):
    """fp32 rows -> (int8, fp32 scale): the largest magnitude becomes 127, ties to even."""
    top = v.abs().amax(1)
    one = torch.where(top > 0, top, 1)
    step = torch.div(torch.full_like(one, 127.0), one)
    return (v * step[:, None]).round().to(torch.int8), torch.div(top, torch.full_like(top, 127.0))


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=g, device=DEV, dtype=dtype)  # noqa: E731
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        x = randn(T, d + c["pad"], dtype=dt)[:, :d]
        residual = randn(T, d, dtype=dt) * 4 if c["residual"] else None
        return dict(case=c, x=x, residual=residual, weight=(1 + 0.2 * randn(d)).to(dt))
    if c["op"] == "score":
        T, V = c["T"], c["V"]
        x = (randn(T, V + c["pad"], dtype=dt).mul_(2.5))[:, :V]
        x[:, V - V // 50:] = -math.inf          # the vocabulary's unused tail
        ids = torch.randint(0, V - V // 50, (T, c["ids"]), generator=g, device=DEV).to(torch.int32)
        return dict(case=c, logits=x, ids=ids)
    M, N, K = c["M"], c["N"], c["K"]
    # activations with a few large channels, weights of a layer: both quantized by rows
    x = randn(M, K) * torch.exp(0.5 * randn(K))
    w, w_scale = _rows8(randn(N, K) / math.sqrt(K))
    s = dict(case=c, w=w, w_scale=w_scale)
    if c["op"] == "head":
        s["a"], s["a_scale"] = _rows8(x)
        s["ids"] = torch.randint(0, N, (M, c["ids"]), generator=g, device=DEV).to(torch.int32)
        return s
    s["bias"] = randn(N) if c["bias"] else None
    if c["quantize"]:
        s["x"] = x.to(dt)
    else:
        s["a"], s["a_scale"] = _rows8(x)
    return s


# ---------------------------------------------------------------- the package's form


def _own(s):
    from weight_only_int4_route_gb300 import dense
    c = s["case"]
    if c["op"] == "norm":
        r = dense.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], y=not c["q8"], q8=c["q8"])
        y = r.y
        if c["q8"]:
            y = torch.empty(r.q.shape, dtype=_value_type(c), device=r.q.device)
            torch.mul(r.q, r.scale[:, None], out=y)
        return {"sum": r.sum, "y": y}
    if c["op"] == "score":
        r = dense.token_logprobs(s["logits"], s["ids"], k=c["k"])
    elif c["op"] == "head":
        logits = dense.linear_w8a8(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=torch.float32)
        r = dense.token_logprobs(logits, s["ids"], k=c["k"])
    else:
        a, a_scale = dense.quantize_rows(s["x"]) if c["quantize"] else (s["a"], s["a_scale"])
        return dense.linear_w8a8(a, a_scale, s["w"], s["w_scale"], bias=s["bias"], out_dtype=DTYPES[c["dtype"]])
    return {"logprob": r.logprob, "entropy": r.entropy, "top_ids": r.top_ids, "top_logprob": r.top_logprob}


# ---------------------------------------------------------------- plain forms


def _value_type(c):
    """The type that 8-bit rows' values are returned in: the activations' 16-bit type."""
    return torch.float16 if c["dtype"] == "f16" else torch.bfloat16


def _linear(a, a_scale, w, w_scale, bias):
    out = (a.float() @ w.float().T) * a_scale[:, None] * w_scale
    return out if bias is None else out + bias


def _scores(x, ids, k):
    x = x.float()
    top = x.amax(1, keepdim=True)
    z = x - top
    lse = z.exp().sum(1, keepdim=True).log()
    z = z - lse
    entropy = torch.where(z == -math.inf, 0, -z.exp() * z).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k] if k else ids.new_empty((x.shape[0], 0)).long()
    return {"logprob": z.gather(1, ids.long()), "entropy": entropy, "top_ids": order.to(torch.int32) if k else None,
            "top_logprob": z.gather(1, order) if k else None}


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        if c["q8"]:
            q, scale = _rows8(y)
            y = q.float() * scale[:, None]
        return {"sum": None if s["residual"] is None else h.to(s["x"].dtype), "y": y.to(_value_type(c) if c["q8"] else s["x"].dtype)}
    if c["op"] == "score":
        return _scores(s["logits"], s["ids"], c["k"])
    if c["op"] == "head":
        return _scores(_linear(s["a"], s["a_scale"], s["w"], s["w_scale"], None), s["ids"], c["k"])
    a, a_scale = _rows8(s["x"].float()) if c["quantize"] else (s["a"], s["a_scale"])
    return _linear(a, a_scale, s["w"], s["w_scale"], s["bias"]).to(DTYPES[c["dtype"]])


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = h / (torch.linalg.vector_norm(h, dim=1, keepdim=True).square() / c["d"] + EPS).sqrt() * s["weight"].double()
        if c["q8"]:
            unit = y.abs().amax(1, keepdim=True) / 127
            y = torch.where(unit > 0, (y / torch.where(unit > 0, unit, 1)).round() * unit, 0)
        return {"sum": None if s["residual"] is None else h, "y": y}
    if c["op"] == "score":
        x = s["logits"].double()
    else:
        if c["op"] == "linear" and c["quantize"]:
            x = s["x"].double()
            a_scale = x.abs().amax(1) / 127
            a = torch.where(a_scale[:, None] > 0, (x / torch.where(a_scale > 0, a_scale, 1)[:, None]).round(), 0)
        else:
            a, a_scale = s["a"].double(), s["a_scale"].double()
        x = torch.einsum("mk,nk->mn", a, s["w"].double()) * torch.outer(a_scale, s["w_scale"].double())
        if c["op"] == "linear":
            return x if s["bias"] is None else x + s["bias"].double()
    lp = x.log_softmax(1)
    p = lp.exp()
    entropy = -torch.special.xlogy(p, p).sum(1)
    k = c["k"]
    return {"logprob": lp.gather(1, s["ids"].long()), "entropy": entropy, "top_ids": None,
            "top_logprob": lp.topk(k, dim=1).values if k else None}
