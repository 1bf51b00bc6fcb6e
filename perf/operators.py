"""Work on which the adapter, router and gradient-clipping operators are timed.

A case names an operator (`op`) and its sizes.  `prepare` makes a user's inputs
on the GPU, `run` makes one pass: with `own` false in plain 32-bit torch
operations, with `own` true through this package's Engine.  `exact` computes the
same results in 64 bits with numpy.

* adapter_forward / adapter_backward: a shared projection x W + bias with the
  low-rank term (s_g x A_g^T) B_g of each row's adapter g (ids outside [0, G)
  have none), and its gradients dx, dA, dB (the shared W is frozen).
* route / route_train: softmax router over E experts with the k largest taken
  (ties to the lowest index), per-expert counts and the balance loss
  E * sum_e (counts_e / kV) * mean_t p_te; route_train adds the gradient of the
  logits from those of the weights and of the loss.
* clip: the global norm of a set of gradients and the set scaled to a maximum.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
# projections (in, out) of the benchmark's layers
PROJECTIONS = [(768, 2048), (2048, 1408), (4096, 4096), (4096, 12288), (4096, 11008), (11008, 4096), (1000, 1000)]


def listed():
    return [
        # one token of one request, through the attention output projection: latency
        {"name": "adapter fwd 1 token", "op": "adapter_forward", "dtype": "bf16", "m": 1, "k": 4096, "n": 4096, "r": 16,
         "g": 8, "runs": 1, "none": 0.0},
        # a decoding batch, every request with its own adapter
        {"name": "adapter fwd decode 64", "op": "adapter_forward", "dtype": "f16", "m": 64, "k": 4096, "n": 11008, "r": 16,
         "g": 64, "runs": 64, "none": 0.05},
        # prompts of several requests, one after the other in the batch, some without adapter
        {"name": "adapter fwd prompts", "op": "adapter_forward", "dtype": "bf16", "m": 8192, "k": 4096, "n": 12288, "r": 16,
         "g": 12, "runs": 20, "none": 0.1},
        # f32 rows in no order, odd sizes
        {"name": "adapter fwd f32 odd", "op": "adapter_forward", "dtype": "f32", "m": 999, "k": 1000, "n": 1000, "r": 5,
         "g": 7, "runs": 999, "none": 0.05},
        # tuning several adapters in one batch
        {"name": "adapter bwd tuning", "op": "adapter_backward", "dtype": "bf16", "m": 8192, "k": 4096, "n": 4096, "r": 32,
         "g": 3, "runs": 8, "none": 0.0},
        # many small tenants, rows in no order, a rank that is no multiple of 16
        {"name": "adapter bwd ragged f16", "op": "adapter_backward", "dtype": "f16", "m": 1333, "k": 768, "n": 2048, "r": 20,
         "g": 17, "runs": 1333, "none": 0.05},
        # a decoding batch's routing: latency
        {"name": "route decode", "op": "route", "dtype": "f32", "t": 64, "e": 64, "k": 6, "normalize": True, "pad": 0.0},
        # a training batch over the grouped workload's eight experts
        {"name": "route train 8", "op": "route_train", "dtype": "bf16", "t": 16384, "e": 8, "k": 2, "normalize": True,
         "pad": 0.05},
        # a long batch over many experts, plain probabilities as weights
        {"name": "route train 256", "op": "route_train", "dtype": "f32", "t": 131072, "e": 256, "k": 8, "normalize": False,
         "pad": 0.05},
        # one small layer's gradients, ragged vectors among them
        {"name": "clip small f32", "op": "clip", "dtype": "f32", "tensors": 24, "elements": 1500007, "limit": 1.0},
        # one adapter set's gradients: many thin tensors, below the limit
        {"name": "clip adapters, below", "op": "clip", "dtype": "f32", "tensors": 48, "elements": 40000003, "limit": 1.0e9},
        # several 7B-class layers' gradients, larger than every cache
        {"name": "clip layers bf16", "op": "clip", "dtype": "bf16", "tensors": 16, "elements": 610000013, "limit": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter_forward", "adapter_forward", "adapter_backward", "route", "route_train", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("adapter"):
        m = _log_int(rng, 1, 8192 if dtype != "f32" else 2048)
        k, n = rng.choice(PROJECTIONS)
        if op == "adapter_backward":
            k, n = rng.choice([p for p in PROJECTIONS if p[0] * p[1] <= 4096 * 4096])
        r = rng.choice([1, 4, 8, 8, 13, 16, 16, 20, 32, 48, 64])
        g = _log_int(rng, 1, min(64, 1024 // r))
        return {"op": op, "dtype": dtype, "m": m, "k": k, "n": n, "r": r, "g": g,
                "runs": rng.choice([min(m, _log_int(rng, 1, 64)), m]), "none": rng.choice([0.0, 0.05, 0.3])}
    if op.startswith("route"):
        e = rng.choice([4, 8, 16, 60, 64, 128, 160, 256])
        return {"op": op, "dtype": dtype, "t": _log_int(rng, 1, 131072), "e": e, "k": rng.randint(1, min(8, e)),
                "normalize": rng.choice([True, False]), "pad": rng.choice([0.0, 0.05])}
    return {"op": op, "dtype": dtype, "tensors": rng.randint(1, 60), "elements": _log_int(rng, 1000, 300000000),
            "limit": rng.choice([1.0e-3, 1.0, 1.0e9])}


def _ids(case, rng):
    """Row -> adapter: `runs` contiguous runs of rows, each with one adapter, or (with probability `none`) without."""
    m, g = case["m"], case["g"]
    cuts = np.sort(rng.choice(np.arange(1, m), size=min(case["runs"], m) - 1, replace=False)) if m > 1 else np.zeros(0, int)
    run = np.searchsorted(cuts, np.arange(m), side="right")
    of = rng.integers(0, g, size=len(cuts) + 1)
    if case["runs"] <= g:  # no more requests than adapters: each has its own
        of = rng.permutation(g)[: len(cuts) + 1]
    of[rng.random(len(of)) < case["none"]] = g
    return of[run].astype(np.int32)


def _sizes(case):
    """`tensors` sizes that add up to about `elements`: matrices and thin vectors, over three orders of magnitude."""
    rng = np.random.default_rng(case["tensors"])
    w = np.exp(rng.uniform(0.0, math.log(1000.0), size=case["tensors"]))
    s = np.maximum(1, (w / w.sum() * case["elements"]).astype(np.int64))
    s[0] = max(1, s[0] + case["elements"] - int(s.sum()))
    return [int(v) for v in s]


def prepare(case, seed):
    op, dt = case["op"], TYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if op.startswith("adapter"):
        m, k, n, r, g = (case[v] for v in "mknrg")
        s.update(x=normal(m, k), w=normal(k, n, std=0.02), bias=normal(n, std=0.1), a=normal(g, r, k, std=k ** -0.5),
                 b=normal(g, r, n, std=0.05), ids=torch.from_numpy(_ids(case, rng)).cuda(),
                 scales=torch.from_numpy((2.0 / rng.integers(1, 5, size=g)).astype(np.float32)).cuda())
        if op == "adapter_forward":
            s.update(y=empty(m, n), h=empty(m, r, dtype=torch.float32))
        else:
            s.update(dy=normal(m, n, std=1e-2), dx=empty(m, k), da=empty(g, r, k, dtype=torch.float32),
                     db=empty(g, r, n, dtype=torch.float32))
            # h as a forward pass leaves it: x A_g^T of each row's adapter in f32
            s["h"] = _adapter_h(s, m, g, r, k).sum(1)
    elif op.startswith("route"):
        t, e, k = case["t"], case["e"], case["k"]
        s.update(logits=normal(t, e, std=1.5), valid=torch.from_numpy((rng.random(t) >= case["pad"]).astype(np.uint8)).cuda(),
                 ids=empty(t, k, dtype=torch.int32), weights=empty(t, k, dtype=torch.float32),
                 counts=empty(e, dtype=torch.int32), rows=empty(1, dtype=torch.int32), mean=empty(e, dtype=torch.float32),
                 loss=empty(1, dtype=torch.float32), lse=empty(t, dtype=torch.float32))
        if op == "route_train":
            s.update(dweights=normal(t, k, std=1e-3, dtype=torch.float32),
                     dloss=torch.full((1,), 0.01, device="cuda"), dlogits=empty(t, e))
    else:
        grads = [normal(v, std=1e-2 * float(np.exp(rng.uniform(-2, 2)))) for v in _sizes(case)]
        out = [torch.empty_like(v) for v in grads]
        s.update(grads=grads, out=out, norm=empty(1, dtype=torch.float32))
    if own:  # the handles a program keeps: the engine, and the table of its gradient buffers
        import deterministic_invariant_gemm_fixed_gb300 as bi
        if not _ENGINE:
            _ENGINE.append(bi.Engine(torch.cuda.current_device()))
        s["eng"] = _ENGINE[0]
        if op == "clip":
            s.update(grad_set=bi.TensorSet(s["grads"]), out_set=bi.TensorSet(s["out"]))
    return s


_ENGINE = []


# ---- plain forms -----------------------------------------------------------

def _rows_of(s, g):
    """[M, G] truth: row m has adapter j."""
    return s["ids"][:, None] == torch.arange(g, device="cuda", dtype=torch.int32)


def _adapter_h(s, m, g, r, k):
    """[M, G, R]: x A_j^T at the row's own adapter, 0 elsewhere."""
    h = (s["x"].float() @ s["a"].float().reshape(g * r, k).t()).view(m, g, r)
    return torch.where(_rows_of(s, g)[:, :, None], h, 0.0)


def _plain_adapter_forward(s, c):
    m, k, n, r, g = (c[v] for v in "mknrg")
    h = _adapter_h(s, m, g, r, k)
    y = s["x"].float() @ s["w"].float() + s["bias"].float()
    y = y + (h * s["scales"][None, :, None]).view(m, g * r) @ s["b"].float().reshape(g * r, n)
    return {"y": y.to(TYPES[c["dtype"]]), "h": h.sum(1)}


def _plain_adapter_backward(s, c):
    m, k, n, r, g = (c[v] for v in "mknrg")
    mine = _rows_of(s, g)[:, :, None]
    dy, x, scale = s["dy"].float(), s["x"].float(), s["scales"][None, :, None]
    u = torch.where(mine, (dy @ s["b"].float().reshape(g * r, n).t()).view(m, g, r) * scale, 0.0).view(m, g * r)
    hs = torch.where(mine, s["h"][:, None, :] * scale, 0.0).view(m, g * r)
    dx = dy @ s["w"].float().t() + u @ s["a"].float().reshape(g * r, k)
    return {"dx": dx.to(TYPES[c["dtype"]]), "da": (u.t() @ x).view(g, r, k), "db": (hs.t() @ dy).view(g, r, n)}


def _plain_route(s, c):
    t, e, k = c["t"], c["e"], c["k"]
    valid = s["valid"] != 0
    x = s["logits"].float()
    top = x.max(1, keepdim=True).values
    ex = torch.exp(x - top)
    z = ex.sum(1, keepdim=True)
    p = torch.where(valid[:, None], ex / z, 0.0)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, order)
    if c["normalize"]:
        chosen = torch.exp(torch.gather(x, 1, order) - top)
        w = torch.where(valid[:, None], chosen / chosen.sum(1, keepdim=True), 0.0)
    ids = torch.where(valid[:, None], order, e)
    counts = (ids.reshape(-1)[:, None] == torch.arange(e, device="cuda")).sum(0)
    rows = valid.sum()
    mean = p.sum(0) / rows.clamp(min=1)
    loss = e * (counts.float() / (k * rows.clamp(min=1)) * mean).sum()
    out = {"ids": ids.to(torch.int32), "weights": w, "counts": counts.to(torch.int32), "mean": mean, "loss": loss.reshape(1)}
    return out, p, w, order, counts, rows, valid


def _plain_route_train(s, c):
    t, e, k = c["t"], c["e"], c["k"]
    out, p, w, order, counts, rows, valid = _plain_route(s, c)
    q = s["dloss"] * e * counts.float() / (k * rows.clamp(min=1).float() ** 2)
    dw = torch.where(valid[:, None], s["dweights"], 0.0)
    if c["normalize"]:
        d = p * (q - (p * q).sum(1, keepdim=True))
        d = d.scatter_add(1, order, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        dp = q.expand(t, e).scatter_add(1, order, dw)
        d = p * (dp - (p * dp).sum(1, keepdim=True))
    out["dlogits"] = torch.where(valid[:, None], d, 0.0).to(TYPES[c["dtype"]])
    return out


def _plain_clip(s, c):
    norm = torch.stack([v.float().square().sum() for v in s["grads"]]).sum().sqrt()
    scale = torch.where(norm > c["limit"], c["limit"] / norm, 1.0)
    return {"norm": norm.reshape(1), "out": [(v.float() * scale).to(v.dtype) for v in s["grads"]]}


def run(s):
    c = s["case"]
    op, dtype = c["op"], c["dtype"]
    if not own:
        if op == "adapter_forward":
            return _plain_adapter_forward(s, c)
        if op == "adapter_backward":
            return _plain_adapter_backward(s, c)
        if op == "route":
            return _plain_route(s, c)[0]
        return _plain_route_train(s, c) if op == "route_train" else _plain_clip(s, c)
    eng = s["eng"]
    if op == "adapter_forward":
        eng.adapter_forward(s["y"], s["h"], s["x"], s["w"], s["bias"], s["a"], s["b"], s["scales"], s["ids"],
                            c["m"], c["k"], c["n"], c["r"], c["g"], dtype)
        return {"y": s["y"], "h": s["h"]}
    if op == "adapter_backward":
        eng.adapter_backward(s["dx"], s["da"], s["db"], s["x"], s["h"], s["w"], s["dy"], s["a"], s["b"], s["scales"],
                             s["ids"], c["m"], c["k"], c["n"], c["r"], c["g"], dtype)
        return {"dx": s["dx"], "da": s["da"], "db": s["db"]}
    if op.startswith("route"):
        eng.router_forward(s["ids"], s["weights"], s["counts"], s["rows"], s["mean"], s["loss"], s["lse"], s["logits"],
                           s["valid"], c["t"], c["e"], c["k"], c["normalize"], dtype)
        out = {v: s[v] for v in ("ids", "weights", "counts", "mean", "loss")}
        if op == "route_train":
            eng.router_backward(s["dlogits"], s["logits"], s["lse"], s["ids"], s["weights"], s["counts"], s["rows"],
                                s["dweights"], s["dloss"], c["t"], c["e"], c["k"], c["normalize"], dtype)
            out["dlogits"] = s["dlogits"]
        return out
    eng.clip_gradients(s["out_set"], s["grad_set"], s["norm"], c["limit"])
    return {"norm": s["norm"], "out": s["out"]}


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op.startswith("adapter"):
        m, k, n, r, g = (case[v] for v in "mknrg")
        used = min(g, case["runs"], m)  # at most this many adapters are in use
        ab = used * r * (k + n)
        if op == "adapter_forward":
            return {"bytes": b * (m * k + k * n + n + m * n + ab) + 4 * (m * r + m + used),
                    "flops": 2 * m * k * n + 2 * m * r * (k + n)}
        return {"bytes": b * (2 * m * k + k * n + m * n + ab) + 4 * (g * r * (k + n) + m * r + m + used),
                "flops": 2 * m * k * n + 4 * m * r * (k + n)}
    if op.startswith("route"):
        t, e, k = case["t"], case["e"], case["k"]
        bytes_, flops = b * t * e + t + 8 * t * k + 8 * e + 4, 4 * t * e
        if op == "route_train":
            bytes_, flops = bytes_ + b * t * e + 4 * t * k, flops + 6 * t * e
        return {"bytes": bytes_, "flops": flops}
    return {"bytes": 2 * b * case["elements"], "flops": 3 * case["elements"]}


# ---- 64-bit values ---------------------------------------------------------

def _f64(v):
    return v.detach().double().cpu().numpy()


def exact(case, seed):
    op = case["op"]
    if op.startswith("adapter"):
        if case["m"] * case["k"] * case["n"] > 2e11:
            return None  # minutes of 64-bit products
        s = prepare(case, seed)
        x, w, a, b, sc = (_f64(s[v]) for v in ("x", "w", "a", "b", "scales"))
        ids, g = s["ids"].cpu().numpy(), case["g"]
        groups = [(j, np.flatnonzero(ids == j)) for j in range(g)]
        h = np.zeros((case["m"], case["r"]))
        if op == "adapter_forward":
            y = x @ w + _f64(s["bias"])
            for j, rows in groups:
                h[rows] = x[rows] @ a[j].T
                y[rows] += sc[j] * (h[rows] @ b[j])
            return {"y": y, "h": h}
        h, dy = _f64(s["h"]), _f64(s["dy"])
        dx = dy @ w.T
        da, db = np.zeros(a.shape), np.zeros(b.shape)
        for j, rows in groups:
            u = sc[j] * (dy[rows] @ b[j].T)
            dx[rows] += u @ a[j]
            da[j] = u.T @ x[rows]
            db[j] = (sc[j] * h[rows]).T @ dy[rows]
        return {"dx": dx, "da": da, "db": db}
    s = prepare(case, seed)
    if op.startswith("route"):
        t, e, k = case["t"], case["e"], case["k"]
        x, ok = _f64(s["logits"]), s["valid"].cpu().numpy() != 0
        z = np.exp(x - x.max(1, keepdims=True))
        p = z / z.sum(1, keepdims=True)
        p[~ok] = 0.0
        pick = np.argsort(-x, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(p, pick, 1)
        if case["normalize"]:
            total = w.sum(1, keepdims=True)
            w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
        ids = np.where(ok[:, None], pick, e)
        counts = np.bincount(ids.ravel(), minlength=e + 1)[:e]
        v = max(1, int(ok.sum()))
        mean = p.sum(0) / v
        f = counts / (k * v)
        out = {"ids": ids, "weights": w, "counts": counts, "mean": mean, "loss": np.array([e * float(f @ mean)])}
        if op == "route_train":
            q = float(s["dloss"].item()) * e * f / v
            dw = _f64(s["dweights"]) * ok[:, None]
            rows = np.arange(t)[:, None]
            if case["normalize"]:
                d = p * (q - (p @ q)[:, None])
                d[rows, pick] += w * (dw - (w * dw).sum(1, keepdims=True))
            else:
                dp = np.tile(q, (t, 1))
                dp[rows, pick] += dw
                d = p * (dp - (p * dp).sum(1, keepdims=True))
            d[~ok] = 0.0
            out["dlogits"] = d
        return out
    if case["elements"] > 200000000:
        return None  # tens of seconds of host work
    grads = [_f64(v) for v in s["grads"]]
    norm = math.sqrt(sum(float(np.dot(v, v)) for v in grads))
    scale = case["limit"] / norm if norm > case["limit"] else 1.0
    return {"norm": np.array([norm]), "out": [v * scale for v in grads]}
