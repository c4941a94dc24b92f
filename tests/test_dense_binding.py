"""Which calls of the dense operators are refused, without a GPU: by the binding (host tensors that say they are on one) and by
the library's own checks (addresses that nothing reads)."""
import pytest
import torch

from test_attn_binding import Fake1, on
from weight_only_int4_route_gb300 import attn, dense, moe

I8, F32, BF16, I32 = torch.int8, torch.float32, torch.bfloat16, torch.int32


@pytest.fixture
def calls(monkeypatch):
    """The library calls made, (name, arguments) each.  GPU 0 is current."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(dense, "lib", Library)
    monkeypatch.setattr(dense, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(attn, "_current_device", lambda: 0)
    return made


def tensors(dev=0):
    z = lambda *s, dtype=BF16: on(torch.zeros(s, dtype=dtype), dev)  # noqa: E731
    return dict(x=z(3, 8), residual=z(3, 8), weight=z(8), total=z(3, 8), a=z(3, 16, dtype=I8), sa=z(3, dtype=F32),
                w=z(5, 16, dtype=I8), sw=z(5, dtype=F32), bias=z(5, dtype=F32), out=z(3, 5), logits=z(3, 40), ids=z(3, 2, dtype=I32))


CALLS = {
    "rmsnorm": (lambda t: dense.rmsnorm(t["x"], t["weight"], residual=t["residual"], q8=True, sum_out=t["total"]),
                ["x", "weight", "residual", "total"]),
    "quantize_rows": (lambda t: dense.quantize_rows(t["x"]), ["x"]),
    "linear": (lambda t: dense.linear_w8a8(t["a"], t["sa"], t["w"], t["sw"], t["bias"], out=t["out"]),
               ["a", "sa", "w", "sw", "bias", "out"]),
    "token_logprobs": (lambda t: dense.token_logprobs(t["logits"], t["ids"], k=2), ["logits", "ids"]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_on_the_current_gpu_are_taken(calls, name):
    CALLS[name][0](tensors())
    assert calls


@pytest.mark.parametrize("name,field", [(n, f) for n in sorted(CALLS) for f in CALLS[n][1] + ["all"]])
def test_tensors_on_another_gpu_are_refused(calls, name, field):
    t = tensors(1) if field == "all" else tensors()
    if field != "all":
        t[field] = t[field].as_subclass(Fake1)
    with pytest.raises(AssertionError):
        CALLS[name][0](t)
    assert not [c for c in calls if "workspace" not in c[0]]


@pytest.mark.parametrize("name,field,other", [
    ("rmsnorm", "residual", lambda t: t.float()), ("rmsnorm", "residual", lambda t: t[:2]), ("rmsnorm", "weight", lambda t: t[:7]),
    ("rmsnorm", "weight", lambda t: t.float()), ("rmsnorm", "total", lambda t: t.float()), ("rmsnorm", "x", lambda t: t.T),
    ("linear", "a", lambda t: t.to(torch.uint8)), ("linear", "w", lambda t: t[:, :15]), ("linear", "sa", lambda t: t[:2]),
    ("linear", "sw", lambda t: t.double()), ("linear", "bias", lambda t: t.to(BF16)), ("linear", "out", lambda t: t[:, :4]),
    ("linear", "out", lambda t: t.double()), ("token_logprobs", "ids", lambda t: t.long()), ("token_logprobs", "ids", lambda t: t[:2]),
    ("token_logprobs", "ids", lambda t: t.T), ("token_logprobs", "logits", lambda t: t.T)])
def test_tensors_of_another_shape_or_type_are_refused(calls, name, field, other):
    t = tensors()
    t[field] = other(t[field])
    with pytest.raises(AssertionError):
        CALLS[name][0](t)
    assert not [c for c in calls if "workspace" not in c[0]]


def test_the_stride_of_a_single_row_is_open(calls):
    t = tensors()
    for f in ("x", "residual", "total", "a", "out", "logits", "sa", "ids"):
        t[f] = t[f][:1]
    t["w"], t["sw"], t["bias"], t["out"] = t["w"][:1], t["sw"][:1], t["bias"][:1], t["out"][:, :1]
    odd = {f: v.as_strided(v.shape, (5, 1)) if v.dim() == 2 else v for f, v in t.items()}
    strides = {"moe_rmsnorm": (1, 3, 10), "moe_quantize_rows": (1,), "moe_linear_w8a8": (1, 4, 11), "moe_token_logprobs": (1,)}
    for name in CALLS:
        calls.clear()
        CALLS[name][0](t)
        plain = list(calls)
        calls.clear()
        odd["ids"] = t["ids"]
        CALLS[name][0](odd)
        for (n, a), (m, b) in zip(plain, calls):
            assert n == m and [a[i] for i in strides.get(n, ())] == [b[i] for i in strides.get(n, ())]


@pytest.fixture(scope="module")
def built():
    from weight_only_int4_route_gb300 import build
    build.build()


P, ODD = 0x1000, 0x1001          # addresses that the checks look at and nothing else does
OK, ARG, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


def norm(x=P, xs=8, r=P, rs=8, w=P, dt=1, T=3, d=8, eps=1e-6, s=P, ss=8, y=P, q=P, scale=P):
    return moe.lib().moe_rmsnorm(x, xs, r, rs, w, dt, T, d, eps, s, ss, y, q, scale, None)


@pytest.mark.parametrize("why,status,args", [
    ("dtype", ARG, dict(dt=3)), ("rows overlap", ARG, dict(xs=7)), ("rows overlap", ARG, dict(rs=7)), ("rows overlap", ARG, dict(ss=7)),
    ("out of range", ARG, dict(d=0)), ("out of range", ARG, dict(T=-1)), ("at most", UNSUPPORTED, dict(d=16385, xs=16385, rs=16385, ss=16385)),
    ("eps", ARG, dict(eps=-1e-6)), ("eps", ARG, dict(eps=float("nan"))), ("eps", ARG, dict(eps=float("inf"))),
    ("together", ARG, dict(q=None)), ("together", ARG, dict(scale=None)), ("no output", ARG, dict(s=None, y=None, q=None, scale=None)),
    ("non-null", ARG, dict(x=None)), ("start on an element", ARG, dict(x=ODD)), ("start on an element", ARG, dict(r=ODD)),
    ("start on an element", ARG, dict(s=ODD)), ("16-byte", ARG, dict(w=0x1008)), ("16-byte", ARG, dict(y=0x1008)), ("16-byte", ARG, dict(q=0x1008)),
    ("same strides", ARG, dict(s=0x2000, r=0x2000, rs=16)), ("same strides", ARG, dict(s=0x2000, x=0x2000, xs=16))])
def test_norm_refusals(built, why, status, args):
    assert norm(**args) == status and why in moe.lib().moe_last_error_string().decode()


def test_no_rows_are_taken(built):
    assert norm(T=0, x=None, r=None, y=None, q=None, scale=None, s=None, w=None) == OK
    L = moe.lib()
    assert L.moe_quantize_rows(None, 8, 0, 0, 8, None, None, None) == OK
    assert L.moe_linear_w8a8(None, 8, None, None, 8, None, None, 0, 8, 8, None, 8, 0, None, 0, None) == OK
    assert L.moe_linear_w8a8(None, 8, None, None, 8, None, None, 8, 0, 8, None, 8, 0, None, 0, None) == OK
    assert L.moe_token_logprobs(None, 8, 0, 0, 8, 1.0, None, 1, None, None, None, 2, None, None, None) == OK


def test_quantize_refusals(built):
    L = moe.lib()
    assert L.moe_quantize_rows(P, 7, 0, 3, 8, P, P, None) == ARG
    assert L.moe_quantize_rows(P, 8, 0, 3, 8, None, P, None) == ARG
    assert L.moe_quantize_rows(P, 8, 0, 3, 8, P, None, None) == ARG
    assert L.moe_quantize_rows(P, 20000, 0, 3, 20000, P, P, None) == UNSUPPORTED
    assert L.moe_quantize_rows(ODD, 8, 2, 3, 8, P, P, None) == ARG


def linear(a=P, ar=16, sa=P, w=P, wr=16, sw=P, b=P, M=3, N=5, K=16, o=P, orow=5, dt=1, ws=P, wb=1 << 30):
    return moe.lib().moe_linear_w8a8(a, ar, sa, w, wr, sw, b, M, N, K, o, orow, dt, ws, wb, None)


@pytest.mark.parametrize("why,status,args", [
    ("out of range", ARG, dict(M=-1)), ("out of range", ARG, dict(N=-1)), ("131071", ARG, dict(K=0)),
    ("131071", ARG, dict(K=131072, ar=131072, wr=131072)), ("out_dtype", ARG, dict(dt=3)), ("rows overlap", ARG, dict(ar=15)),
    ("rows overlap", ARG, dict(wr=15)), ("rows overlap", ARG, dict(orow=4)), ("null", ARG, dict(a=None)), ("null", ARG, dict(sa=None)),
    ("null", ARG, dict(w=None)), ("null", ARG, dict(sw=None)), ("null", ARG, dict(o=None)), ("16-byte", ARG, dict(sa=0x1004)),
    ("16-byte", ARG, dict(b=0x1004)), ("start on an element", ARG, dict(o=ODD)), ("workspace", WORKSPACE, dict(K=15, wb=79)),
    ("workspace", WORKSPACE, dict(wr=17, wb=0)), ("workspace", WORKSPACE, dict(w=ODD, wb=0)), ("workspace", ARG, dict(K=15, ws=None)),
    ("workspace", ARG, dict(K=15, ws=0x1008)), ("workspace", WORKSPACE, dict(M=100, wb=0)), ("workspace", ARG, dict(M=100, ws=None))])
def test_linear_refusals(built, why, status, args):
    assert linear(**args) == status and why in moe.lib().moe_last_error_string().decode()


def scores(x=P, row=40, dt=1, T=3, V=40, scale=1.0, ids=P, n=2, lp=P, h=P, lse=P, k=2, ti=P, tl=P):
    return moe.lib().moe_token_logprobs(x, row, dt, T, V, scale, ids, n, lp, h, lse, k, ti, tl, None)


@pytest.mark.parametrize("why,status,args", [
    ("dtype", ARG, dict(dt=-1)), ("out of range", ARG, dict(T=-1)), ("out of range", ARG, dict(T=1 << 27)), ("out of range", ARG, dict(V=0)),
    ("out of range", ARG, dict(V=1 << 30, row=1 << 30)), ("rows overlap", ARG, dict(row=39)), ("scale", ARG, dict(scale=0.0)),
    ("scale", ARG, dict(scale=-1.0)), ("scale", ARG, dict(scale=float("nan"))), ("scale", ARG, dict(scale=float("inf"))),
    ("n_ids", ARG, dict(n=-1)), ("k <=", UNSUPPORTED, dict(k=65)), ("k <=", UNSUPPORTED, dict(k=-1)), ("logits", ARG, dict(x=None)),
    ("logits", ARG, dict(x=ODD)), ("without logprob", ARG, dict(lp=None)), ("without logprob", ARG, dict(ids=None)),
    ("k without", ARG, dict(ti=None)), ("k without", ARG, dict(tl=None)), ("16-byte", ARG, dict(ids=0x1004)), ("16-byte", ARG, dict(h=0x1004)),
    ("16-byte", ARG, dict(tl=0x1004))])
def test_score_refusals(built, why, status, args):
    assert scores(**args) == status and why in moe.lib().moe_last_error_string().decode()


def test_linear_workspace_size(built):
    L = moe.lib()
    size = L.moe_linear_w8a8_workspace_size
    assert size(4, 8, 0) == 0 and size(-1, 8, 8) == 0 and size(4, 8, 131072) == 0
    for N, K in ((5, 15), (4096, 4096), (33, 1408), (6144, 131071)):
        got = [size(M, N, K) for M in (0, 1, 8, 16, 17, 32, 33, 64, 200, 1000, 8192, 100000)]
        assert got[0] >= N * K and got[0] == got[3] and size(16, 0, K) == 0 and size(17, 0, K) >= 34 * K and all(b >= a for a, b in zip(got, got[1:]))      # serves every call of fewer rows
