"""A fine-tuning step over the framework's operators, repeated for a few steps.

Rows of several requests, each with its own low-rank adapter, go through a shared
projection (frozen) with their adapters, a router sends each row to k of E experts
(a grouped matmul, trained), and the step's gradients (adapters, router, experts)
are clipped to a global norm before a plain SGD update.  Every pass runs in the
library's deterministic kernels: two runs print the same losses and end with the
same bits.

    python examples/adapter_moe_step.py [--steps 5] [--rows 4096] [--dtype bf16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from deterministic_invariant_gemm_fixed_gb300.nn import adapter_linear, clip_grad_norm_, engine_for, route  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Experts(torch.autograd.Function):
    """y[m] = x[m] @ w[ids[m]].T with w [E, out, in]; ids >= E give zero rows."""

    @staticmethod
    def forward(ctx, x, w, ids):
        (m, k), (e, n, _) = x.shape, w.shape
        y = torch.empty(m, n, dtype=x.dtype, device=x.device)
        engine_for(x.device).grouped_forward(y, x, w, ids, m, k, n, e, x.dtype)
        ctx.save_for_backward(x, w, ids)
        return y

    @staticmethod
    def backward(ctx, gy):
        x, w, ids = ctx.saved_tensors
        (m, k), (e, n, _) = x.shape, w.shape
        dx, dw = torch.empty_like(x), torch.empty(e, n, k, dtype=torch.float32, device=x.device)
        engine_for(x.device).grouped_backward(dx, dw, x, w, gy.contiguous(), ids, m, k, n, e, x.dtype)
        return dx, dw.to(w.dtype), None


def run(steps=5, rows=4096, features=768, hidden=2048, experts=8, top=2, adapters=6, rank=16, dtype="bf16", lr=0.5,
        max_norm=1.0, seed=0, device="cuda"):
    """Trains for `steps` steps; returns (losses, norms, parameters)."""
    dt = TYPES[dtype]
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std, grad=True):
        return (torch.randn(*shape, generator=gen, device=device) * std).to(dt).requires_grad_(grad)

    x = normal(rows, features, std=1.0, grad=False)
    target = normal(rows, features, std=1.0, grad=False)
    ids = (torch.arange(rows, device=device) * (adapters + 1) // rows).int()  # the last request has no adapter
    valid = torch.ones(rows, dtype=torch.bool, device=device)
    valid[::17] = False  # padding rows
    w = normal(features, hidden, std=features ** -0.5, grad=False)
    a, b = normal(adapters, rank, features, std=features ** -0.5), normal(adapters, rank, hidden, std=0.05)
    scales = torch.full((adapters,), 2.0, device=device)
    gate = normal(hidden, experts, std=hidden ** -0.5)
    up = normal(experts, features, hidden, std=hidden ** -0.5)
    params = [a, b, gate, up]
    losses, norms = [], []
    for _ in range(steps):
        hid = torch.relu(adapter_linear(x, w, None, a, b, scales, ids))
        choice, weight, balance, _ = route(hid @ gate, top, valid=valid)
        out = Experts.apply(hid.repeat_interleave(top, 0), up, choice.reshape(-1))
        out = (out.float().view(rows, top, features) * weight[..., None]).sum(1)
        loss = torch.where(valid[:, None], out - target.float(), 0.0).square().mean() + 0.01 * balance
        loss.backward()
        norm = clip_grad_norm_(params, max_norm)
        with torch.no_grad():
            for p in params:
                p -= lr * p.grad
                p.grad = None
        losses.append(loss.detach())
        norms.append(norm)
    engine_for(x.device).check()
    return torch.stack(losses).tolist(), torch.cat(norms).tolist(), params


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    args = ap.parse_args()
    losses, norms, _ = run(steps=args.steps, rows=args.rows, dtype=args.dtype)
    for i, (l, n) in enumerate(zip(losses, norms)):
        print(f"step {i}: loss {l:.6f}, gradient norm {n:.4f}")
