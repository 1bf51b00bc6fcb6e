"""The autograd form of the MXFP4 products, and the expert layer behind its router.

The linear layer's results are products of quantized operands: they are compared with the
64-bit products of the same operands (tests/test_gpu_fp4.py has the bound: depth d,
(d/64 + 4) 2^-23 of the magnitudes' sum, and half a step of the type), the bias gradient
with the sum of the output gradient's rows (256 f32 additions a chunk: 2^-15 of the
magnitudes' sum).  Gradients of the function itself are checked by differences on integers
whose blocks are exact in MXFP4, where the rounding does nothing.
"""
import numpy as np
import pytest
import torch

import fp4_ref
from deterministic_invariant_gemm_fixed_gb300 import nn

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, a, b, dt, add=0.0):
    want, S = a @ b.T + add, np.abs(a) @ np.abs(b).T + np.abs(add)
    tol = (a.shape[1] / 64 + 4) * 2.0 ** -23 * S
    assert (np.abs(f64(got) - want) <= tol + HALF[dt] * (np.abs(want) + tol) + 2.0 ** -25).all()


@pytest.mark.parametrize("dt", HALF)
def test_linear_forward_and_gradients(dt):
    gen = torch.Generator(device="cuda").manual_seed(3)
    def t(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=gen) * std).to(dt).requires_grad_()
    x, w, b = t(3, 50, 72), t(72, 136, std=0.1), t(136)
    gy = torch.randn(3, 50, 136, device="cuda", generator=gen).to(dt)
    y = nn.deterministic_linear(x, w, b, fp4=True)
    y.backward(gy)
    X, W, G = f64(x).reshape(150, 72), f64(w), f64(gy).reshape(150, 136)
    r = fp4_ref.rounded
    near(y.reshape(150, 136), r(X), r(W.T), dt, f64(b))
    near(x.grad.reshape(150, 72), r(G), r(W), dt)
    near(w.grad, r(X.T), r(G.T), dt)
    assert (np.abs(f64(b.grad) - G.sum(0)) <= 2.0 ** -15 * np.abs(G).sum(0) + HALF[dt] * np.abs(G.sum(0)) * 1.01).all()
    # the same bits again, and with only some gradients asked for
    x2, w2 = x.detach().clone().requires_grad_(), w.detach().clone()
    y2 = nn.deterministic_linear(x2, w2, b.detach(), fp4=True)
    y2.backward(gy)
    assert torch.equal(y, y2) and torch.equal(x.grad, x2.grad)


def test_gradient_by_differences():
    """On values that MXFP4 holds exactly the function is the plain product: central differences of a linear function."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    table = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, -1.0, -2.0, -3.0, 6.0], device="cuda")
    def t(*s):
        return table[torch.randint(0, 9, s, device="cuda", generator=gen)]
    x, w, g = t(32, 64), t(64, 32), t(32, 32)
    for v in (x, w, g):
        v[::8, ::8] = 6.0  # every block of 32, either way, has its largest: scale 1
    def loss(a, b):
        return (nn.deterministic_linear(a, b, fp4=True).double() * g.double()).sum()
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss(a, b).backward()
    for leaf, base, other, first in ((a, x, w, True), (b, w, x, False)):
        for i, j in ((1, 1), (17, 30), (31, 9)):
            up, dn = base.clone(), base.clone()
            up[i, j], dn[i, j] = 2.0, -2.0
            hi, lo = (loss(up, other), loss(dn, other)) if first else (loss(other, up), loss(other, dn))
            assert float(leaf.grad[i, j]) == float((hi - lo) / 4.0)


def test_refusals():
    x, w = torch.randn(4, 32, device="cuda", requires_grad=True), torch.randn(32, 8, device="cuda")
    with pytest.raises(ValueError):
        nn.deterministic_linear(x, w, fp4=True, fp8=nn.Fp8Scales(1.0, 1.0, 1.0))
    y = nn.deterministic_linear(x, w, fp4=True)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    up, down, logits = torch.randn(4, 16, 32, device="cuda"), torch.randn(4, 8, 16, device="cuda"), torch.randn(4, 4, device="cuda")
    with pytest.raises(ValueError):
        nn.moe(x, logits, None, up, down, 2)  # x requires a gradient
    x = x.detach()
    with pytest.raises(ValueError):
        nn.moe(x, logits, None, nn.Fp4Weight.quantize(up), down, 2)
    with pytest.raises(ValueError):
        nn.moe(x, logits, up, up, torch.randn(4, 8, 15, device="cuda"), 2)
    with pytest.raises(ValueError):
        nn.moe(x, logits[:3], None, up, down, 2)
    with pytest.raises(ValueError):
        nn.moe(x, logits, None, up, down, 2, activation="tanh")
    with pytest.raises(ValueError):
        nn.moe(x.half(), logits, None, up, down, 2)


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dt", HALF)
def test_moe_behind_its_router(dt, fp4):
    """Router, experts, padding rows and a batch of several calls; each row as it is alone."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    def t(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=gen) * std).to(dt)
    e, k, f, n, tokens = 6, 64, 48, 40, 1100
    x, logits = t(tokens, k), t(tokens, e, std=2.0)
    gate, up, down = t(e, f, k, std=k ** -0.5), t(e, f, k, std=k ** -0.5), t(e, n, f, std=f ** -0.5)
    valid = torch.ones(tokens, dtype=torch.bool, device="cuda")
    valid[::13] = False
    w = [gate, up, down]
    if fp4:
        w = [nn.Fp4Weight.quantize(v) for v in w]
        gate, up, down = (v.dequantize() for v in w)
    with torch.no_grad():
        y = nn.moe(x, logits, *w, 2, valid=valid)
        ids, p, _, _ = nn.route(logits, 2, valid=valid)
    pick = ids.clamp(max=e - 1).long()
    g, u = (torch.einsum("tk,tcfk->tcf", x.double(), v.double()[pick]) for v in (gate, up))
    want = torch.einsum("tcf,tcnf,tc->tn", torch.nn.functional.silu(g) * u, down.double()[pick], p.double())
    # sums of 64 and 48 terms in f32 and h in 16-bit parts: below 2^-14 of the row's largest, and the type's half step
    tol = 2.0 ** -14 * want.abs().amax(1, keepdim=True) * 4 + HALF[dt] * want.abs()
    assert ((y.double() - want).abs() <= tol).all()
    assert not y[~valid].any()
    with torch.no_grad():
        for i in (1, 500, 1099):
            assert torch.equal(nn.moe(x[i:i + 1], logits[i:i + 1], *w, 2, valid=valid[i:i + 1]), y[i:i + 1])


def test_step_with_fp4_layers_and_captured_backward():
    """Layer, router and 4-bit experts in turn; a forward and backward captured beside an eager one of the same leaves."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    def t(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=gen) * std).bfloat16()
    x, w = t(64, 96).requires_grad_(), t(96, 64, std=0.1).requires_grad_()
    router = t(64, 8, std=0.2)
    experts = [nn.Fp4Weight.quantize(v) for v in (t(8, 32, 64, std=0.1), t(8, 32, 64, std=0.1), t(8, 64, 32, std=0.2))]

    def step():
        x.grad = w.grad = None
        h = nn.deterministic_linear(x, w, fp4=True)
        with torch.no_grad():
            out = nn.moe(h, h @ router, *experts, 2)
        h.backward(out)
        return out

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = step()
        grads = x.grad.clone(), w.grad.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(x.grad, grads[0]) and torch.equal(w.grad, grads[1])


def test_empty_batches():
    x, w, b = torch.empty(0, 64, device="cuda", requires_grad=True), torch.randn(64, 32, device="cuda", requires_grad=True), torch.randn(32, device="cuda", requires_grad=True)
    y = nn.deterministic_linear(x, w, b, fp4=True)
    assert y.shape == (0, 32)
    y.sum().backward()
    assert x.grad.shape == (0, 64) and not w.grad.any() and not b.grad.any()
    up, down = torch.randn(4, 16, 64, device="cuda"), torch.randn(4, 8, 16, device="cuda")
    with torch.no_grad():
        assert nn.moe(x, torch.empty(0, 4, device="cuda"), None, up, down, 2).shape == (0, 8)
