"""Low-rank adapters beside a shared projection, against a 64-bit implementation.

Bounds, per element, with u = 2^-24 (f32's rounding), S the sum of the magnitudes
of all products that enter the element (the inner products' magnitudes included),
L the longest chain of additions behind it:

* scalar tier and f32 inputs: any order of f32 additions is within L u S of the
  exact value (first order); 4 more for the scale, the bias and the piece sums.
* tensor-core tier: the framework's published 2e-6 S for an f32 accumulation,
  taken twice where an inner product feeds an outer one; the inner product
  enters the outer one as two 16-bit parts, which adds 2^-16 of its own terms
  (bf16: two roundings to 8 bits; f16: 2^-22 of the value plus 2^-24 absolute).
  3xTF32 (f32 inputs with tensor cores): the same 2e-6 S for the shared product.
* a 16-bit result adds its own rounding, half an ulp.
"""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
from helpers import ulp_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    e.close()


def inputs(m, k, n, r, g, dtype, seed=0, order="runs", none=0.1, scales=True, bias=True):
    rng = np.random.default_rng(seed)
    def t(*shape, std=1.0):
        return torch.from_numpy(rng.standard_normal(shape) * std).to(TD[dtype]).cuda()
    ids = rng.integers(0, g, size=m)
    if order == "runs":
        ids = np.sort(ids)
        ids = np.roll(ids, m // 3)
    drop = rng.random(m) < none
    ids[drop] = rng.choice([g, g + 5, 0x7FFFFFFF], size=int(drop.sum()))
    return dict(x=t(m, k), w=t(k, n, std=k ** -0.5), bias=t(n) if bias else None, a=t(g, r, k, std=k ** -0.5), b=t(g, r, n, std=0.3),
                dy=t(m, n), ids=torch.from_numpy(ids.astype(np.int32)).cuda(),
                scales=torch.from_numpy((rng.integers(1, 9, size=g) / 4.0).astype(np.float32)).cuda() if scales else None,
                m=m, k=k, n=n, r=r, g=g, dtype=dtype)


def sizes(d):
    return [d[v] for v in "mknrg"] + [d["dtype"]]


def forward(eng, d, tc, stream=None):
    y = torch.full((d["m"], d["n"]), float("nan"), dtype=TD[d["dtype"]], device="cuda")
    h = torch.full((d["m"], d["r"]), float("nan"), dtype=torch.float32, device="cuda")
    eng.adapter_forward(y, h, d["x"], d["w"], d["bias"], d["a"], d["b"], d["scales"], d["ids"], *sizes(d), stream, tc)
    return y, h


def backward(eng, d, h, tc, which=("dx", "da", "db")):
    dx = torch.full((d["m"], d["k"]), float("nan"), dtype=TD[d["dtype"]], device="cuda") if "dx" in which else None
    da = torch.full((d["g"], d["r"], d["k"]), float("nan"), dtype=torch.float32, device="cuda") if "da" in which else None
    db = torch.full((d["g"], d["r"], d["n"]), float("nan"), dtype=torch.float32, device="cuda") if "db" in which else None
    eng.adapter_backward(dx, da, db, d["x"], h, d["w"], d["dy"], d["a"], d["b"], d["scales"], d["ids"], *sizes(d),
                         None, tc)
    return dx, da, db


def f64(t):
    return t.detach().double().cpu().numpy()


def exact(d, h_in=None):
    """All results and their magnitude sums in 64 bits."""
    x, w, a, b, dy = (f64(d[v]) for v in ("x", "w", "a", "b", "dy"))
    ids, g = d["ids"].cpu().numpy().view(np.uint32), d["g"]
    s = f64(d["scales"]) if d["scales"] is not None else np.ones(g)
    bias = f64(d["bias"]) if d["bias"] is not None else np.zeros(d["n"])
    m, r = d["m"], d["r"]
    o = {"h": np.zeros((m, r)), "h_s": np.zeros((m, r)), "y": x @ w + bias, "y_s": abs(x) @ abs(w) + abs(bias),
         "dx": dy @ w.T, "dx_s": abs(dy) @ abs(w).T, "u": np.zeros((m, r)),
         "da": np.zeros(a.shape), "da_s": np.zeros(a.shape), "db": np.zeros(b.shape), "db_s": np.zeros(b.shape),
         "y_in": np.zeros((m, d["n"])), "dx_in": np.zeros((m, d["k"])), "most": 0}
    for j in range(g):
        q = np.flatnonzero(ids == j)
        o["most"] = max(o["most"], len(q))
        if not len(q):
            continue
        h, hs = x[q] @ a[j].T, abs(x[q]) @ abs(a[j]).T
        o["h"][q], o["h_s"][q] = h, hs
        o["y"][q] += s[j] * (h @ b[j])
        o["y_s"][q] += s[j] * (hs @ abs(b[j]))
        o["y_in"][q] = (s[j] * abs(h)) @ abs(b[j])
        u, us = s[j] * (dy[q] @ b[j].T), s[j] * (abs(dy[q]) @ abs(b[j]).T)
        o["dx"][q] += u @ a[j]
        o["dx_s"][q] += us @ abs(a[j])
        o["dx_in"][q] = abs(u) @ abs(a[j])
        o["da"][j], o["da_s"][j] = u.T @ x[q], us.T @ abs(x[q])
        hh = h if h_in is None else f64(h_in)[q]
        o["db"][j], o["db_s"][j] = (s[j] * hh).T @ dy[q], (s[j] * abs(hh)).T @ abs(dy[q])
    return o


def close(got, want, scale, dtype, chain, tc, inner=None, floor=0.0):
    got = f64(got)
    tol = (4e-6 if tc else (chain + 4) * U) * scale + floor
    if tc and inner is not None and dtype != "f32":
        tol = tol + 2.0 ** -16 * inner
        if dtype == "f16":
            tol = tol + 2.0 ** -24 * 64
    if dtype != "f32":
        tol = tol + 0.5 * ulp_of(np.maximum(abs(got), abs(want)), dtype)
    bad = ~(abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, float((abs(got - want) / np.maximum(tol, 1e-300)).max()))


SHAPES = [  # m, k, n, r, g, order
    (1, 64, 64, 1, 1, "runs"),
    (1, 7, 5, 3, 2, "runs"),              # nothing aligned
    (5, 72, 136, 4, 3, "random"),
    (33, 1000, 200, 20, 40, "random"),    # more adapters than rows of some
    (130, 520, 264, 16, 7, "runs"),       # the narrow product's second piece is 8 long
    (300, 513, 129, 5, 6, "random"),      # odd rows: scalar tier whatever is asked
    (257, 1024, 512, 64, 2, "runs"),
    (515, 256, 320, 100, 300, "random"),  # more adapters than a tile's rows, rank over 64
    (2100, 192, 128, 8, 2, "runs"),       # more than one chunk of rows per adapter
    (1300, 64, 64, 33, 1, "random"),
    (70, 128, 96, 256, 3, "runs"),        # the largest rank
]


@pytest.mark.parametrize("tc", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k,n,r,g,order", SHAPES)
def test_against_64_bits(eng, m, k, n, r, g, order, dtype, tc):
    d = inputs(m, k, n, r, g, dtype, seed=m + k, order=order)
    y, h = forward(eng, d, tc)
    e = exact(d, h)
    dx, da, db = backward(eng, d, h, tc)
    eng.check()
    chain = k + n + r + 16
    close(h, e["h"], e["h_s"], "f32", k, tc)
    close(y, e["y"], e["y_s"], dtype, chain, tc, e["y_in"])
    close(dx, e["dx"], e["dx_s"], dtype, chain, tc, e["dx_in"])
    rows = min(e["most"], 1024) + e["most"] // 1024
    close(da, e["da"], e["da_s"], "f32", n + rows, tc)
    close(db, e["db"], e["db_s"], "f32", rows, tc)


@pytest.mark.parametrize("dtype,tc", [("f32", 0), ("f32", 1), ("bf16", 0), ("bf16", 1), ("f16", 1)])
def test_rows_do_not_depend_on_the_batch(eng, dtype, tc):
    """Every prefix, and a shuffled copy, gives each row the same bits; so does a second run."""
    d = inputs(700, 1032, 328, 24, 9, dtype, seed=3, order="random")
    y, h = forward(eng, d, tc)
    dx, da, db = backward(eng, d, h, tc)
    y2, h2 = forward(eng, d, tc)
    dx2, da2, db2 = backward(eng, d, h, tc)
    for p, q in ((y, y2), (h, h2), (dx, dx2), (da, da2), (db, db2)):
        assert torch.equal(p, q)
    for m in (1, 2, 17, 64, 65, 128, 129, 256, 300, 513):
        e = dict(d, m=m, x=d["x"][:m].contiguous(), dy=d["dy"][:m].contiguous(), ids=d["ids"][:m].contiguous())
        ye, he = forward(eng, e, tc)
        dxe = backward(eng, e, he, tc, ("dx",))[0]
        assert torch.equal(ye, y[:m]) and torch.equal(he, h[:m]) and torch.equal(dxe, dx[:m]), m
    perm = torch.randperm(700, generator=torch.Generator().manual_seed(1)).cuda()
    e = dict(d, x=d["x"][perm].contiguous(), dy=d["dy"][perm].contiguous(), ids=d["ids"][perm].contiguous())
    ye, he = forward(eng, e, tc)
    dxe = backward(eng, e, he, tc, ("dx",))[0]
    assert torch.equal(ye, y[perm]) and torch.equal(he, h[perm]) and torch.equal(dxe, dx[perm])


@pytest.mark.parametrize("dtype,tc", [("f32", 0), ("bf16", 0), ("bf16", 1), ("f16", 1)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_request_cannot_reach_another(eng, dtype, tc, bad):
    """Infinities and NaN in one adapter, its rows and their gradients stay there, and in rows without adapter they stay there too."""
    d = inputs(400, 264, 328, 16, 5, dtype, seed=5, order="random", none=0.2)
    y, h = forward(eng, d, tc)
    dx, da, db = backward(eng, d, h, tc)
    ids = d["ids"].cpu().numpy().view(np.uint32)
    hit = torch.from_numpy((ids == 2) | (ids >= 5)).cuda()
    e = dict(d, x=d["x"].clone(), dy=d["dy"].clone(), a=d["a"].clone(), b=d["b"].clone())
    e["x"][hit] = bad
    e["dy"][hit] = bad
    e["a"][2] = bad
    e["b"][2] = bad
    ye, he = forward(eng, e, tc)
    dxe, dae, dbe = backward(eng, e, he, tc)
    for p, q in ((y, ye), (h, he), (dx, dxe)):
        assert torch.equal(p[~hit], q[~hit])
    keep = torch.tensor([0, 1, 3, 4], device="cuda")
    assert torch.equal(da[keep], dae[keep]) and torch.equal(db[keep], dbe[keep])
    assert not torch.isfinite(ye[hit]).any()


def test_rows_without_adapter_are_the_shared_projection(eng):
    """No id in range: y and dx are the plain layer's, bit for bit, h, dA and dB are 0."""
    for dtype, tc in (("f32", 0), ("f32", 1), ("bf16", 0), ("bf16", 1), ("f16", 1)):
        d = inputs(200, 136, 264, 8, 4, dtype, seed=6)
        d["ids"].fill_(4)
        y, h = forward(eng, d, tc)
        dx, da, db = backward(eng, d, h, tc)
        y0, dx0 = torch.empty_like(y), torch.empty_like(dx)
        eng.forward(y0, d["x"], d["w"], d["bias"], d["m"], d["k"], d["n"], dtype, None, tc)
        eng.backward_dx(dx0, d["dy"], d["w"], d["m"], d["k"], d["n"], dtype, None, tc)
        assert torch.equal(y, y0) and torch.equal(dx, dx0)
        assert not h.any() and not da.any() and not db.any()


@pytest.mark.parametrize("dtype,tc", [("f32", 0), ("bf16", 1)])
def test_gradients_against_differences(eng, dtype, tc):
    """sum(Y * dY) is linear in A and in B each, so a central difference of any step is its derivative up to rounding."""
    d = inputs(96, 128, 192, 8, 3, dtype, seed=7, order="random")
    y, h = forward(eng, d, tc)
    e = exact(d)
    dx, da, db = backward(eng, d, h, tc)
    dy = f64(d["dy"])
    ulp = ulp_of(np.abs(e["y"]) + 2 * e["y_in"], dtype) if dtype != "f32" else 0.0
    for name, got in (("a", da), ("b", db)):
        for idx in ((0, 0, 0), (1, 3, 77), (2, 7, 127)):
            up_, dn = d[name].clone(), d[name].clone()
            up_[idx] += 1
            dn[idx] -= 1
            step = float(up_[idx].double() - dn[idx].double())
            hi, lo = f64(forward(eng, dict(d, **{name: up_}), tc)[0]), f64(forward(eng, dict(d, **{name: dn}), tc)[0])
            diff = float(((hi - lo) * dy).sum()) / step
            rows = (d["ids"] == idx[0]).cpu().numpy()
            # each of hi, lo is off by a bound of y's at that row; S grows by the perturbed term
            grow = e["y_s"] + 4 * (abs(f64(d["x"])).max() * abs(f64(d["b"])).max() + e["h_s"].max())
            tol = float((np.abs(dy) * (8e-6 * grow + 2.0 ** -15 * grow * (tc == 1) + ulp))[rows].sum()) * 2 / step
            assert abs(diff - float(got[idx])) <= tol, (name, idx, diff, float(got[idx]), tol)


def test_parts_are_optional(eng):
    for dtype, tc in (("f32", 1), ("bf16", 1), ("bf16", 0)):
        d = inputs(150, 136, 264, 8, 4, dtype, seed=8, scales=False, bias=False)
        y, h = forward(eng, d, tc)
        y2 = torch.empty_like(y)
        eng.adapter_forward(y2, None, d["x"], d["w"], None, d["a"], d["b"], None, d["ids"], *sizes(d), None, tc)
        assert torch.equal(y, y2)
        ones = dict(d, scales=torch.ones(4, device="cuda"))
        assert torch.equal(forward(eng, ones, tc)[0], y)
        full = backward(eng, d, h, tc)
        for i, name in enumerate(("dx", "da", "db")):
            got = backward(eng, d, h, tc, (name,))
            assert torch.equal(got[i], full[i]) and all(v is None for j, v in enumerate(got) if j != i)


def test_empty_batch_and_refusals(eng):
    d = inputs(4, 64, 64, 4, 2, "bf16")
    y, h = forward(eng, d, 1)
    none = dict(d, m=0)
    _, da, db = backward(eng, none, h, 1)
    assert not da.any() and not db.any()
    eng.adapter_forward(y, h, d["x"], d["w"], None, d["a"], d["b"], None, d["ids"], *sizes(none))
    def status(**change):
        q = dict(d, **change)
        return bi.bi_adapter_forward(eng.handle, y, h, q["x"], q["w"], None, q["a"], q["b"], None, q["ids"], *sizes(q))
    assert status() == bi.BI_OK
    for change in (dict(r=0), dict(g=0), dict(k=0), dict(n=0), dict(m=-1), dict(dtype=7), dict(x=None), dict(w=None),
                   dict(a=None), dict(b=None), dict(ids=None)):
        assert status(**change) == bi.BI_ERR_INVALID_ARG, change
    assert status(r=257) == bi.BI_ERR_UNSUPPORTED and status(g=65536) == bi.BI_ERR_UNSUPPORTED
    odd = torch.empty(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    assert status(x=odd) == bi.BI_ERR_MISALIGNED
    with pytest.raises(ValueError):
        status(a=d["a"].transpose(1, 2))
    with pytest.raises(bi.BiError):
        eng.adapter_backward(y, None, None, None, None, d["w"], None, d["a"], d["b"], None, d["ids"], *sizes(d))
    assert bi.bi_adapter_forward(None, *[16] * 9, 1, 1, 1, 1, 1, "bf16", 0) == bi.BI_ERR_INVALID_ARG


def test_no_scratch_leaves_outputs_alone(eng):
    for dtype, tc in (("f32", 1), ("bf16", 1), ("bf16", 0)):
        d = inputs(64, 64, 64, 4, 2, dtype)
        want, h0 = forward(eng, d, tc)
        y, h = torch.zeros_like(want), torch.zeros_like(h0)
        args = (y, h, d["x"], d["w"], d["bias"], d["a"], d["b"], d["scales"], d["ids"], *sizes(d), None, tc)
        for nth in (1, -1):
            bi.bi_engine_fail_allocations(eng.handle, nth)
            assert bi.bi_adapter_forward(eng.handle, *args) == bi.BI_ERR_OOM
            bi.bi_engine_fail_allocations(eng.handle, 0)
            assert not y.any() and not h.any()
        eng.adapter_forward(*args)
        assert torch.equal(y, want)


def test_side_stream_and_graph(eng):
    d = inputs(40, 256, 320, 16, 6, "bf16", seed=9, order="random")
    y, h = forward(eng, d, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, h2 = forward(eng, d, 1)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2)
    y3, h3 = torch.zeros_like(y), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eng.adapter_forward(y3, h3, d["x"], d["w"], d["bias"], d["a"], d["b"], d["scales"], d["ids"], *sizes(d))
    for _ in range(2):
        y3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y)


@pytest.mark.parametrize("dtype,tc", [("f32", 0), ("bf16", 0), ("bf16", 1), ("f16", 1)])
def test_nothing_is_written_outside_the_outputs(eng, dtype, tc):
    """Poisoned bands around every output of ragged shapes stay as they were."""
    d = inputs(133, 136, 200, 12, 5, dtype, seed=10, order="random")
    pad = 64
    outs = {}
    for name, shape, t in (("y", (133, 200), TD[dtype]), ("h", (133, 12), torch.float32), ("dx", (133, 136), TD[dtype]),
                           ("da", (5, 12, 136), torch.float32), ("db", (5, 12, 200), torch.float32)):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 7.0, dtype=t, device="cuda")
        outs[name] = (buf, buf[pad:pad + n].view(shape))
    eng.adapter_forward(outs["y"][1], outs["h"][1], d["x"], d["w"], d["bias"], d["a"], d["b"], d["scales"], d["ids"],
                        *sizes(d), None, tc)
    eng.adapter_backward(outs["dx"][1], outs["da"][1], outs["db"][1], d["x"], outs["h"][1], d["w"], d["dy"], d["a"], d["b"],
                         d["scales"], d["ids"], *sizes(d), None, tc)
    torch.cuda.synchronize()
    for buf, _ in outs.values():
        assert bool((buf[:pad] == 7).all() and (buf[-pad:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k,n,r,g", [(1, 512, 256, 16, 2), (37, 1032, 328, 20, 9), (64, 136, 1000, 64, 64), (65, 264, 72, 8, 3),
                                       (200, 520, 640, 100, 30), (300, 64, 64, 33, 200), (513, 768, 264, 48, 4)])
def test_small_and_paired_tiles_give_the_same_bits(eng, m, k, n, r, g, dtype):
    """The tile shape is chosen from the number of tiles; forcing the CTA pairs' width must not change a bit."""
    d = inputs(m, k, n, r, g, dtype, seed=11, order="random")
    y, h = forward(eng, d, 1)
    dx = backward(eng, d, h, 1, ("dx",))[0]
    bi.bi_engine_set_tile_cols(eng.handle, 256)
    try:
        y2, h2 = forward(eng, d, 1)
        dx2 = backward(eng, d, h2, 1, ("dx",))[0]
    finally:
        bi.bi_engine_set_tile_cols(eng.handle, 0)
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(dx, dx2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_row_tiles(eng, dtype):
    """More tiles and pieces than resident CTAs: each takes several pieces; rows equal those of a short batch."""
    d = inputs(20011, 1040, 72, 8, 5, dtype, seed=12, order="random")
    y, h = forward(eng, d, 1)
    dx = backward(eng, d, h, 1, ("dx",))[0]
    for lo in (0, 9984, 19900):
        hi = min(lo + 111, d["m"])
        e = dict(d, m=hi - lo, x=d["x"][lo:hi].contiguous(), dy=d["dy"][lo:hi].contiguous(), ids=d["ids"][lo:hi].contiguous())
        ye, he = forward(eng, e, 1)
        assert torch.equal(ye, y[lo:hi]) and torch.equal(he, h[lo:hi])
        assert torch.equal(backward(eng, e, he, 1, ("dx",))[0], dx[lo:hi])
        r = exact(e)
        close(ye, r["y"], r["y_s"], dtype, 0, 1, r["y_in"])
        close(he, r["h"], r["h_s"], "f32", 0, 1)


def test_backward_in_a_graph_and_on_a_side_stream(eng):
    d = inputs(700, 256, 320, 16, 6, "bf16", seed=13, order="random")
    _, h = forward(eng, d, 1)
    want = backward(eng, d, h, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = backward(eng, d, h, 1)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eng.adapter_backward(*out, d["x"], h, d["w"], d["dy"], d["a"], d["b"], d["scales"], d["ids"], *sizes(d))
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, out))


def test_calls_back_to_back_on_one_buffer(eng):
    """Each call reads what the one before wrote (the kernels of the next may start early): a chain of projections."""
    d = inputs(48, 256, 256, 16, 4, "bf16", seed=14, order="random", bias=False)
    x = d["x"]
    want = []
    for _ in range(6):
        y, _ = forward(eng, dict(d, x=x), 1)
        torch.cuda.synchronize()
        x = y
        want.append(y)
    bufs = [torch.empty_like(x) for _ in range(2)]
    for rep in range(20):
        src = d["x"]
        for i in range(6):
            eng.adapter_forward(bufs[i % 2], None, src, d["w"], None, d["a"], d["b"], d["scales"], d["ids"], *sizes(d))
            src = bufs[i % 2]
        assert torch.equal(src, want[-1]), rep


def far_inputs(m, k, n, r, g, seed, which):
    """f16 whose inner products s h ("y") or u ("dx") pass 65504 in many places while the results stay finite."""
    d = inputs(m, k, n, r, g, "f16", seed=seed, order="random", none=0.1)
    rng = np.random.default_rng(seed + 1)
    powers = rng.choice([0, 14, 17, 20], size=g)
    powers[0] = 20
    d["scales"] = torch.from_numpy((2.0 ** powers).astype(np.float32)).cuda()
    if which == "y":  # h about 1: s h up to some 2^22, B about 2^-11
        d["b"] = (torch.from_numpy(rng.standard_normal((g, r, n))) * 2.0 ** -11).half().cuda()
    else:  # dY B^T about 1, A about 2^-11
        d["b"] = (torch.from_numpy(rng.standard_normal((g, r, n))) * n ** -0.5).half().cuda()
        d["a"] = (torch.from_numpy(rng.standard_normal((g, r, k))) * 2.0 ** -11).half().cuda()
    return d


FAR = [(1, 512, 256, 16, 2), (37, 1032, 328, 20, 9), (65, 264, 72, 8, 3), (200, 520, 640, 100, 30), (300, 64, 64, 33, 40), (1500, 128, 2048, 16, 6)]


@pytest.mark.parametrize("which", ["y", "dx"])
@pytest.mark.parametrize("m,k,n,r,g", FAR)
def test_inner_products_beyond_f16(eng, m, k, n, r, g, which):
    """s h and u are f32 values: those that f16 cannot hold count in full, and by any tile with the same bits.

    Bound: 2e-6 S twice (the two products), 2^-21 of the inner terms and 2^-24 r max|Q|
    for the remainders' own rounding, terms beyond f16 in f32 FMAs (r roundings), half an ulp."""
    d = far_inputs(m, k, n, r, g, m + k, which)
    if which == "y":
        got, h = forward(eng, d, 1)
        e = exact(d, h)
        want, s, inner, q = e["y"], e["y_s"], e["y_in"], d["b"]
        v = abs(e["h"]) * f64(torch.cat([d["scales"], d["scales"][:1]]))[np.minimum(d["ids"].cpu().numpy().view(np.uint32), g)][:, None]
        if m > 1:
            assert v.max() > 2.0 ** 18
    else:
        got = backward(eng, d, None, 1, ("dx",))[0]
        e = exact(d)
        want, s, inner, q = e["dx"], e["dx_s"], e["dx_in"], d["a"]
    keep = abs(want) < 6.0e4
    assert keep.mean() > 0.5
    tol = 4e-6 * s + 2.0 ** -21 * inner + 2.0 ** -24 * r * float(q.abs().max()) + (r + 4) * U * inner
    tol = tol + 0.5 * ulp_of(np.maximum(abs(f64(got)), abs(want)), "f16")
    assert (abs(f64(got) - want) <= tol)[keep].all()
    bi.bi_engine_set_tile_cols(eng.handle, 256)
    try:
        other = forward(eng, d, 1)[0] if which == "y" else backward(eng, d, None, 1, ("dx",))[0]
    finally:
        bi.bi_engine_set_tile_cols(eng.handle, 0)
    assert torch.equal(got, other)
    for lo, hi in ((0, 1), (m // 2, m)):  # rows alone
        p = dict(d, m=hi - lo, x=d["x"][lo:hi].contiguous(), dy=d["dy"][lo:hi].contiguous(), ids=d["ids"][lo:hi].contiguous())
        part = forward(eng, p, 1)[0] if which == "y" else backward(eng, p, None, 1, ("dx",))[0]
        assert torch.equal(part, got[lo:hi])


def test_zeros_beside_an_inner_product_beyond_f16(eng):
    """A finite s h times 0 is 0, whatever its size."""
    m, k, n, r, g = 5, 64, 128, 4, 1
    d = inputs(m, k, n, r, g, "f16", seed=2, none=0.0)
    d["bias"] = None
    d["w"].zero_()
    d["scales"] = torch.tensor([2.0 ** 16], device="cuda")
    d["x"].fill_(0)
    d["x"][:, 0] = 100.0
    d["a"].fill_(0)
    d["a"][:, :, 0] = 1.0  # s h = 100 * 2^16
    d["b"].fill_(0)
    d["b"][0, 0, :64] = 2.0 ** -14
    y, _ = forward(eng, d, 1)
    assert torch.equal(y, torch.cat([torch.full((m, 64), 400.0, device="cuda"), torch.zeros(m, 64, device="cuda")], 1).half())


@pytest.mark.parametrize("which", ["y", "dx"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [3, 100, 300])
def test_inner_products_keep_both_parts(eng, m, dtype, which):
    """Whole numbers throughout: inner products of 22 bits (f16; bf16 16) that f32 holds exactly and that
    cancel down to 2 z, so a bit lost in the remainder shows as it is."""
    k = n = 64
    rng = np.random.default_rng(m)
    big, unit = (32.0, 2.0 ** -6) if dtype == "f16" else (256.0, 1.0)
    rows = np.zeros((m, k))
    rows[:, 0] = rng.integers(1, 2000 if dtype == "f16" else 255, size=m)
    rows[:, 1] = rng.integers(1, 2000 if dtype == "f16" else 127, size=m) * unit
    narrow, wide = np.zeros((1, 2, k)), np.zeros((1, 2, k))
    narrow[0, 0, :2], narrow[0, 1, :2] = (big, 1.0), (big, -1.0)
    wide[0, 0], wide[0, 1] = 1.0, -1.0
    t = lambda v: torch.from_numpy(v).to(TD[dtype]).cuda()
    d = dict(x=t(rows), dy=t(rows), w=t(np.zeros((k, n))), bias=None, scales=None, m=m, k=k, n=n, r=2, g=1, dtype=dtype,
             a=t(narrow if which == "y" else wide), b=t(wide if which == "y" else narrow),
             ids=torch.zeros(m, dtype=torch.int32, device="cuda"))
    want = t(np.repeat(2 * rows[:, 1:2], 64, 1))
    for cols in (0, 256):
        bi.bi_engine_set_tile_cols(eng.handle, cols)
        try:
            got = forward(eng, d, 1)[0] if which == "y" else backward(eng, d, None, 1, ("dx",))[0]
        finally:
            bi.bi_engine_set_tile_cols(eng.handle, 0)
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,tc", [("f32", 0), ("bf16", 0), ("bf16", 1), ("f16", 1)])
@pytest.mark.parametrize("m", [5, 300])
def test_an_infinite_scale_reaches_no_padding(eng, m, dtype, tc):
    """Every term of the row is the same infinity: ranks that only pad a vector (rank 4 of 16) add nothing to it."""
    k, n, r = 64, 128, 4
    d = inputs(m, k, n, r, 1, dtype, seed=2, none=0.0)
    for v, c in (("w", 0.0), ("x", 1.0), ("dy", 1.0), ("a", 1.0), ("b", -1.0)):
        d[v].fill_(c)
    d["scales"] = torch.tensor([float("inf")], device="cuda")
    y, h = forward(eng, d, tc)
    assert (y == float("-inf")).all() and (h == k).all()
    assert (backward(eng, d, h, tc, ("dx",))[0] == float("-inf")).all()  # u = -inf, A = 1
    bi.bi_engine_set_tile_cols(eng.handle, 256)
    try:
        assert torch.equal(forward(eng, d, tc)[0], y)
    finally:
        bi.bi_engine_set_tile_cols(eng.handle, 0)


def test_lengths_beyond_the_grids_are_refused(eng):
    """Rows longer than the f32-FMA kernels' grids count: refused before anything is written."""
    long = 65535 * 128 + 1
    x, w = torch.ones(1, long, device="cuda"), torch.ones(8, 8, device="cuda")
    a, dy, b = torch.ones(1, 1, long, device="cuda"), torch.ones(1, 8, device="cuda"), torch.ones(1, 1, 8, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    da = torch.full((1, 1, long), 7.0, device="cuda")
    def status(k):
        return bi.bi_adapter_backward(eng.handle, None, da, None, x, None, w, dy, a, b, None, ids, 1, k, 8, 1, 1, "f32", None, 0)
    assert status(long) == bi.BI_ERR_UNSUPPORTED and (da == 7).all()
    assert status(long - 1) == bi.BI_OK and (da[..., :-1] == 8).all() and float(da[0, 0, -1]) == 7  # u = 8, x = 1
    # y of 65535 x 256 + 1 columns (refused on the host: nothing is read)
    y = torch.full((8,), 7.0, device="cuda")
    assert bi.bi_adapter_forward(eng.handle, y, None, x, w, None, a, b, None, ids, 1, 8, 65535 * 256 + 1, 1, 1, "f32", None,
                                 0) == bi.BI_ERR_UNSUPPORTED
    assert bi.bi_adapter_forward(eng.handle, y, None, x, w, None, a, b, None, ids, 1, 65535 * 512 + 1, 8, 1, 1, "f32", None,
                                 0) == bi.BI_ERR_UNSUPPORTED
    assert (y == 7).all()
