"""Router: choice, weights, counts, balance loss and its gradient, against 64 bits.

Choices and counts are whole numbers and equal.  A probability is exp(x - max) /
sum: the exponent's argument is rounded at f32 (2^-24 |x - max|, twice: once in
the difference, once in the scaling by log2 e), the exponential is within 2 ulp,
the sum of E positive terms within E 2^-24, the division 1 ulp.  With |x - max|
<= D a probability is within (2 D + E + 8) 2^-24 relative; sums of T of them add
T 2^-24 (taken as 64 + T / 64: a block adds up to a few hundred rows per lane,
the rest is a tree).  The gradient's terms are products of such values.
"""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
from helpers import ulp_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = ("ids", "weights", "counts", "rows", "mean", "loss", "lse")


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    e.close()


def outputs(t, e, k):
    def f(*s):
        return torch.full(s, float("nan"), device="cuda")
    def i(*s):
        return torch.full(s, -7, dtype=torch.int32, device="cuda")
    return dict(ids=i(t, k), weights=f(t, k), counts=i(e), rows=i(1), mean=f(e), loss=f(1), lse=f(t))


def route(eng, logits, valid, k, normalize):
    t, e = logits.shape
    o = outputs(t, e, k)
    eng.router_forward(*[o[v] for v in NAMES], logits, valid, t, e, k, normalize, logits.dtype)
    return o


def route_back(eng, logits, o, dw, dl, k, normalize):
    t, e = logits.shape
    d = torch.full_like(logits, float("nan"))
    eng.router_backward(d, logits, o["lse"], o["ids"], o["weights"], o["counts"], o["rows"], dw, dl, t, e, k, normalize,
                        logits.dtype)
    return d


def exact(x, ok, k, normalize, dw=None, dl=0.0):
    """64-bit values for finite logits and -inf; ok: rows that take part."""
    t, e = x.shape
    alive = ok & (x.max(1) > -np.inf)
    top = np.where(alive, x.max(1), 0.0)
    z = np.where(alive[:, None], np.exp(x - top[:, None]), 0.0)
    p = z / np.maximum(z.sum(1, keepdims=True), 1e-300)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    can = np.take_along_axis(x, order, 1) > -np.inf
    can &= alive[:, None]
    w = np.where(can, np.take_along_axis(p, order, 1), 0.0)
    if normalize:
        w = np.divide(w, w.sum(1, keepdims=True), out=np.zeros_like(w), where=w.sum(1, keepdims=True) > 0)
    ids = np.where(can, order, e)
    counts = np.bincount(ids.ravel(), minlength=e + 1)[:e]
    v = int(alive.sum())
    mean = p.sum(0) / max(v, 1)
    loss = e * float((counts / max(k * v, 1)) @ mean)
    out = dict(ids=ids, w=w, counts=counts, v=v, mean=mean, loss=loss, p=p, alive=alive,
               lse=np.where(alive, top + np.log(np.maximum(z.sum(1), 1e-300)), np.inf))
    if dw is not None:
        q = dl * e * counts / max(k * v * v, 1)
        dw = np.where(can, dw, 0.0)
        rows = np.arange(t)[:, None]
        if normalize:
            d = p * (q - (p @ q)[:, None])
            add = w * (dw - (w * dw).sum(1, keepdims=True))
            mag = p * (abs(q) + (p @ abs(q))[:, None])
            mag_add = w * (abs(dw) + (w * abs(dw)).sum(1, keepdims=True))
            for j in range(k):
                pick = can[:, j]
                d[rows[pick, 0], order[pick, j]] += add[pick, j]
                mag[rows[pick, 0], order[pick, j]] += mag_add[pick, j]
        else:
            dp = np.tile(q, (t, 1))
            mp = np.tile(abs(q), (t, 1))
            for j in range(k):
                pick = can[:, j]
                dp[rows[pick, 0], order[pick, j]] += dw[pick, j]
                mp[rows[pick, 0], order[pick, j]] += abs(dw[pick, j])
            d = p * (dp - (p * dp).sum(1, keepdims=True))
            mag = p * (mp + (p * mp).sum(1, keepdims=True))
        out.update(d=d, mag=mag)
    return out


CASES = [  # t, e, k
    (1, 1, 1), (1, 8, 2), (3, 4, 4), (64, 64, 6), (257, 60, 5), (1000, 8, 2), (130, 16, 16), (77, 32, 3), (300, 128, 8),
    (5000, 256, 8), (100, 160, 64), (40000, 8, 2), (9000, 64, 6), (20000, 16, 3), (700, 256, 8), (50, 500, 33), (40, 1024, 64), (33, 1000, 7)]


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t,e,k", CASES)
def test_against_64_bits(eng, t, e, k, dtype, normalize):
    rng = np.random.default_rng(t * 31 + e)
    x = torch.from_numpy(rng.standard_normal((t, e)) * 2).to(TD[dtype])
    if e >= 8:  # ties, masked experts, both zeros
        x[::3, 2] = x[::3, 5]
        x[::4, : e // 2] = float("-inf")
        x[1::5, 3], x[1::5, 1] = -0.0, 0.0
    if t >= 3:
        x[2] = float("-inf")  # a mask that leaves nothing
    ok = rng.random(t) > 0.1
    dw = rng.standard_normal((t, k)).astype(np.float32)
    logits = x.cuda()
    garbage = torch.from_numpy(~ok).cuda()
    logits[garbage] = float("nan")  # rows left out are not looked at
    valid = torch.from_numpy(ok.astype(np.uint8)).cuda()
    dl = torch.tensor([0.7], device="cuda")
    o = route(eng, logits, valid, k, normalize)
    d = route_back(eng, logits, o, torch.from_numpy(dw).cuda(), dl, k, normalize)
    x64 = np.where(ok[:, None], x.double().numpy(), 0.0)
    r = exact(x64, ok, k, normalize, dw.astype(np.float64), float(dl.item()))
    assert np.array_equal(o["ids"].cpu().numpy(), r["ids"])
    assert np.array_equal(o["counts"].cpu().numpy(), r["counts"]) and int(o["rows"]) == r["v"]
    fin = x64[np.isfinite(x64)]
    span = float(fin.max() - fin.min()) if fin.size else 0.0
    rel = (2 * span + e + 8) * U
    w = o["weights"].double().cpu().numpy()
    assert (abs(w - r["w"]) <= 2 * rel * r["w"] + 1e-38).all()
    lse = o["lse"].double().cpu().numpy()
    assert np.array_equal(np.isinf(lse), ~r["alive"])
    assert (abs(lse - r["lse"])[r["alive"]] <= rel + 8 * U * (1 + abs(r["lse"][r["alive"]]))).all()
    sums = rel + (64 + t / 64) * U
    assert (abs(o["mean"].double().cpu().numpy() - r["mean"]) <= sums * r["mean"] + 1e-38).all()
    assert abs(float(o["loss"]) - r["loss"]) <= (sums + (e + 8) * U) * r["loss"]
    got = d.double().cpu().numpy()
    # p from lse: its error is absolute in the exponent
    grel = 2 * rel + 16 * U * (1 + (abs(r["lse"][r["alive"]]).max() if r["alive"].any() else 0.0)) + e * U
    tol = 4 * grel * r["mag"] + 1e-38 + (0.5 * ulp_of(np.maximum(abs(got), abs(r["d"])), dtype) if dtype != "f32" else 0.0)
    assert (abs(got - r["d"]) <= tol).all(), float((abs(got - r["d"]) / tol).max())
    assert not d[garbage].any()
    again = route(eng, logits, valid, k, normalize)
    for v in NAMES:
        assert torch.equal(o[v], again[v])


@pytest.mark.parametrize("normalize", [0, 1])
def test_gradient_against_differences(eng, normalize):
    """Central differences of the kernels' own sum(weights * dw) + loss * dl; logits far enough apart that no choice changes."""
    rng = np.random.default_rng(4)
    t, e, k, step = 6, 16, 3, 2.0 ** -6
    x = np.stack([rng.permutation(e) for _ in range(t)]) * 0.25
    dw = rng.standard_normal((t, k)).astype(np.float32)
    dl = torch.tensor([1.5], device="cuda")
    def value(v):
        o = route(eng, torch.from_numpy(v).float().cuda(), None, k, normalize)
        return float((o["weights"].double().cpu().numpy() * dw).sum() + 1.5 * o["loss"].double().item())
    logits = torch.from_numpy(x).float().cuda()
    o = route(eng, logits, None, k, normalize)
    d = route_back(eng, logits, o, torch.from_numpy(dw).cuda(), dl, k, normalize).cpu().numpy()
    for i, j in ((0, 0), (1, 7), (2, int(x[2].argmax())), (5, int(x[5].argmin()))):
        hi, lo = x.copy(), x.copy()
        hi[i, j] += step
        lo[i, j] -= step
        diff = (value(hi) - value(lo)) / (2 * step)
        # third derivative of a softmax is at most 1 per unit of dw: step^2 / 6 of |dw| + |dl| E
        tol = step ** 2 / 6 * (abs(dw).sum() + 1.5 * e) + 64 * U * (abs(dw).sum() + 1.5 * e) / step
        assert abs(diff - d[i, j]) <= tol


def test_not_a_number_shows(eng):
    x = torch.randn(4, 8, device="cuda")
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    o = route(eng, x, None, 2, 1)
    assert torch.isfinite(o["weights"][[0, 3]]).all() and torch.isnan(o["weights"][1]).all()
    assert torch.isnan(o["loss"]).all() and int(o["rows"]) == 4
    assert 3 not in o["ids"][1].tolist() and int(o["ids"][2, 0]) == 4
    d = route_back(eng, x, o, torch.ones(4, 2, device="cuda"), None, 2, 1)
    assert torch.isnan(d[1]).all()
    # the rows beside it, whose loss gradient is not asked for, are untouched
    assert torch.isfinite(d[[0, 3]]).all()


def test_feeds_the_grouped_matmul(eng):
    t, e, k, f, n = 200, 8, 1, 64, 72
    logits = torch.randn(t, e, device="cuda")
    valid = torch.ones(t, dtype=torch.uint8, device="cuda")
    valid[::7] = 0
    o = route(eng, logits, valid, k, 0)
    x, w = torch.randn(t, f, device="cuda"), torch.randn(e, n, f, device="cuda")
    y = torch.empty(t, n, device="cuda")
    eng.grouped_forward(y, x, w, o["ids"], t, f, n, e, "f32", None, 0)
    ids = o["ids"][:, 0].long()
    keep = ids < e
    want = torch.zeros(t, n, dtype=torch.float64, device="cuda")
    want[keep] = torch.einsum("tf,tnf->tn", x[keep].double(), w[ids[keep]].double())
    assert torch.allclose(y.double(), want, rtol=0, atol=64 * U * f * 4) and not y[~keep].any()


def test_empty_and_refusals(eng):
    x = torch.randn(4, 8, device="cuda")
    o = outputs(4, 8, 2)
    eng.router_forward(*[o[v] for v in NAMES], x, None, 0, 8, 2, 1, "f32")
    assert int(o["rows"]) == 0 and float(o["loss"]) == 0 and not o["counts"].any() and not o["mean"].any()
    none = route(eng, x, torch.zeros(4, dtype=torch.uint8, device="cuda"), 2, 1)
    assert float(none["loss"]) == 0 and (none["ids"] == 8).all() and not none["weights"].any()
    def st(t=4, e=8, k=2, dt="f32", logits=x, ids=o["ids"]):
        return bi.bi_router_forward(eng.handle, ids, *[o[v] for v in NAMES[1:]], logits, None, t, e, k, 1, dt)
    assert st() == bi.BI_OK
    for bad in (dict(t=-1), dict(e=0), dict(k=0), dict(k=9), dict(dt=5), dict(logits=None), dict(ids=None)):
        assert st(**bad) == bi.BI_ERR_INVALID_ARG, bad
    assert st(e=1025) == bi.BI_ERR_UNSUPPORTED and st(e=100, k=65) == bi.BI_ERR_UNSUPPORTED
    assert bi.bi_router_backward(eng.handle, None, x, o["lse"], o["ids"], o["weights"], o["counts"], o["rows"], None, None,
                                 4, 8, 2, 1, "f32") == bi.BI_ERR_INVALID_ARG
    assert bi.bi_router_forward(None, *[16] * 9, 1, 1, 1, 1, "f32", 0) == bi.BI_ERR_INVALID_ARG
    bi.bi_engine_fail_allocations(eng.handle, 1)  # a batch of several blocks takes scratch
    q, big = outputs(50000, 8, 2), torch.randn(50000, 8, device="cuda")
    assert bi.bi_router_forward(eng.handle, *[q[v] for v in NAMES], big, None, 50000, 8, 2, 1, "f32") == bi.BI_ERR_OOM
    bi.bi_engine_fail_allocations(eng.handle, 0)
    assert (q["ids"] == -7).all()


def test_unaligned_rows(eng):
    """A view that starts off 16-byte alignment gives the same results."""
    base = torch.randn(50 * 64 + 1, device="cuda").to(torch.bfloat16)
    x = base[1:].view(50, 64)
    o, p = route(eng, x, None, 4, 1), route(eng, x.clone(), None, 4, 1)
    for v in NAMES:
        assert torch.equal(o[v], p[v])
    dw = torch.randn(50, 4, device="cuda")
    dl = torch.ones(1, device="cuda")
    assert torch.equal(route_back(eng, x, o, dw, dl, 4, 1), route_back(eng, x.clone(), p, dw, dl, 4, 1))


@pytest.mark.parametrize("e", [8, 64, 200])
def test_large_logits(eng, e):
    """Logits of 1e4 and of 3e38 apart: the softmax is that of their differences."""
    gen = torch.Generator(device="cuda").manual_seed(e)
    x = torch.randint(0, 5, (40, e), device="cuda", generator=gen).float()
    for shift in (1.0e4, -2.0e4):  # the sums are exact in f32
        o, p = route(eng, x + shift, None, 2, 0), route(eng, x, None, 2, 0)
        for v in ("ids", "counts", "weights", "mean", "loss"):
            assert torch.equal(o[v], p[v]), v
    y = torch.full((3, e), -3.0e38, device="cuda")
    y[:, 5] = 3.0e38
    y[1, 6] = 3.0e38
    o = route(eng, y, None, 2, 0)
    assert o["weights"].tolist() == [[1.0, 0.0], [0.5, 0.5], [1.0, 0.0]]
    d = route_back(eng, y, o, torch.ones(3, 2, device="cuda"), torch.ones(1, device="cuda"), 2, 0)
    assert torch.isfinite(d).all()


def _exact_gradient_check(x, valid, o, d, dw, dl, k, normalize, dtype):
    """d against 64 bits, for probabilities from differences of logits: no term grows with the logits themselves."""
    t, e = x.shape
    x64 = x.double().cpu().numpy()
    r = exact(x64, valid, k, normalize, dw.double().cpu().numpy(), float(dl.item()))
    fin = np.where(np.isfinite(x64), x64, x64.max(1, keepdims=True))
    # beyond 104 below the maximum a probability is under 2^-149 in either case
    span = float(np.minimum(fin.max(1) - fin.min(1), 104.0).max())
    grel = 2 * (2 * span + e + 8) * U + 16 * U + e * U
    got = d.double().cpu().numpy()
    tol = 4 * grel * r["mag"] + 1e-38 + (0.5 * ulp_of(np.maximum(abs(got), abs(r["d"])), dtype) if dtype != "f32" else 0.0)
    assert (abs(got - r["d"]) <= tol).all(), float((abs(got - r["d"]) / tol).max())


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("dtype,shift,step", [("f32", 1.0e4, 1.0), ("f32", -1.0e6, 1.0), ("f32", 1.0e7, 1.0),
                                              ("bf16", 1024.0, 8.0), ("f16", 8192.0, 8.0)])
@pytest.mark.parametrize("e,k", [(8, 2), (64, 6), (200, 8), (1000, 40)])
def test_gradient_does_not_depend_on_a_shift_of_the_logits(eng, e, k, dtype, shift, step, normalize):
    """Logits whose sums with the shift are exact: differences, hence probabilities and gradients, are the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(e + k)
    x = (torch.randint(0, 5, (70, e), device="cuda", generator=gen) * step).to(TD[dtype])
    y = (x.double() + shift).to(TD[dtype])
    assert torch.equal(y.double() - shift, x.double())
    dw = torch.randn(70, k, device="cuda", generator=gen)
    dl = torch.tensor([0.7], device="cuda")
    out = []
    for v in (x, y):
        o = route(eng, v, None, k, normalize)
        out.append(route_back(eng, v, o, dw, dl, k, normalize))
        _exact_gradient_check(v, np.ones(70, bool), o, out[-1], dw, dl, k, normalize, dtype)
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("e", [8, 64, 200])
def test_gradient_of_the_largest_logits(eng, e, normalize):
    """Two experts tied at 3e38 have probability 1/2 each, in the gradient too."""
    y = torch.full((3, e), -3.0e38, device="cuda")
    y[:, 5] = 3.0e38
    y[1, 6] = 3.0e38
    dw = torch.tensor([[1.0, 1.0], [1.0, -2.0], [0.5, 3.0]], device="cuda")
    dl = torch.tensor([0.5], device="cuda")
    o = route(eng, y, None, 2, normalize)
    d = route_back(eng, y, o, dw, dl, 2, normalize)
    _exact_gradient_check(y, np.ones(3, bool), o, d, dw, dl, 2, normalize, "f32")


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dloss", [-1.0, float("inf"), float("nan")])
@pytest.mark.parametrize("e,k", [(8, 2), (60, 5), (256, 8)])
def test_rows_left_out_get_plus_zero(eng, e, k, dloss, dtype, normalize):
    """Whatever the loss's gradient is (an overflowed loss scale), the gradient of a row left out is +0, bit for bit."""
    x = torch.randn(40, e, device="cuda").to(TD[dtype])
    x[7] = float("-inf")
    valid = torch.ones(40, dtype=torch.uint8, device="cuda")
    valid[::3] = 0
    o = route(eng, x, valid, k, normalize)
    d = route_back(eng, x, o, torch.randn(40, k, device="cuda"), torch.tensor([dloss], device="cuda"), k, normalize)
    out = valid == 0
    out[7] = True
    bits = d.view(torch.int32 if dtype == "f32" else torch.int16)
    assert not bits[out].any()
