"""The autograd forms of the adapters, the router and the clipping, and the example that runs them together.

Gradients are compared with torch's own autograd of the same formulas in 64 bits.
f32 with the scalar tier: f32 additions over chains of at most 200 (in, out, rows,
rank), products of up to three such sums; each is within 256 * 2^-24 of the sum
of its magnitudes, which for these standard normal inputs is below 64 times the
root mean square of the result: 3 * 256 * 2^-24 * 64 = 3e-3 of the largest value.
"""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from deterministic_invariant_gemm_fixed_gb300 import nn

pytestmark = pytest.mark.gpu
TOL = 3 * 256 * 2.0 ** -24 * 64


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def near(got, want):
    assert got.shape == want.shape
    assert (got.double() - want).abs().max() <= TOL * want.abs().max()


def test_adapter_linear_gradients():
    gen = torch.Generator(device="cuda").manual_seed(1)
    def t(*s):
        return torch.randn(*s, device="cuda", generator=gen).requires_grad_()
    x, w, bias, a, b = t(5, 8, 48), t(48, 72), t(72), t(3, 4, 48), t(3, 4, 72)
    scales = torch.tensor([0.5, 2.0, 1.0], device="cuda")
    ids = torch.randint(0, 4, (5, 8), device="cuda", generator=gen, dtype=torch.int32)
    gy = torch.randn(5, 8, 72, device="cuda", generator=gen)
    y = nn.adapter_linear(x, w, bias, a, b, scales, ids, tensor_cores=False)
    y.backward(gy)
    leaves = [v.detach().double().requires_grad_() for v in (x, w, bias, a, b)]
    X, W, BI, A, B = leaves
    own = torch.nn.functional.one_hot(ids.long(), 4)[..., :3].double()
    h = torch.einsum("...k,grk->...gr", X, A) * (own * scales.double())[..., None]
    want = X @ W + BI + torch.einsum("...gr,grn->...n", h, B)
    want.backward(gy.double())
    near(y, want.detach())
    for got, leaf in zip((x, w, bias, a, b), leaves):
        near(got.grad, leaf.grad)


def test_adapter_linear_partial_gradients_and_refusals():
    x = torch.randn(6, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(64, 64, device="cuda", dtype=torch.bfloat16)
    a = torch.randn(2, 4, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    b = torch.randn(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(6, dtype=torch.int32, device="cuda")
    nn.adapter_linear(x, w, None, a, b, None, ids).float().sum().backward()
    assert a.grad is not None and a.grad.dtype == torch.bfloat16
    for bad in (dict(a=a[0]), dict(b=b[:, :, :32]), dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.cpu()),
                dict(scales=torch.ones(3, device="cuda")), dict(scales=torch.ones(2, device="cuda", dtype=torch.float64))):
        args = dict(dict(a=a, b=b, scales=None, ids=ids), **bad)
        with pytest.raises(ValueError):
            nn.adapter_linear(x, w, None, args["a"], args["b"], args["scales"], args["ids"])
    with pytest.raises(TypeError):
        nn.adapter_linear(x, w, None, a.float(), b, None, ids)


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradients(normalize):
    gen = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(7, 9, 16, device="cuda", generator=gen, requires_grad=True)
    valid = torch.rand(7, 9, device="cuda", generator=gen) > 0.2
    gw = torch.randn(7, 9, 3, device="cuda", generator=gen)
    ids, weights, loss, counts = nn.route(logits, 3, normalize, valid)
    ((weights * gw).sum() + 0.7 * loss).backward()
    x = logits.detach().double().requires_grad_()
    p = torch.softmax(x, -1)
    pick = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :3]
    w = torch.gather(p, -1, pick)
    if normalize:
        w = w / w.sum(-1, keepdim=True)
    w = torch.where(valid[..., None], w, 0.0)
    v = int(valid.sum())
    cnt = torch.bincount(pick[valid].reshape(-1), minlength=16)
    mean = torch.where(valid[..., None], p, 0.0).sum((0, 1)) / v
    l64 = 16 * (cnt.double() / (3 * v) * mean).sum()
    ((w * gw.double()).sum() + 0.7 * l64).backward()
    assert torch.equal(ids, torch.where(valid[..., None], pick, 16).int()) and torch.equal(counts, cnt.int())
    near(weights, w.detach())
    near(loss, l64.detach())
    near(logits.grad, x.grad)
    # only the loss, only the weights
    for f in (lambda w_, l_: l_, lambda w_, l_: w_.square().sum()):
        logits.grad = None
        _, w2, l2, _ = nn.route(logits, 3, normalize, valid)
        f(w2, l2).backward()
        assert torch.isfinite(logits.grad).all()


def test_clip_grad_norm():
    ps = [torch.nn.Parameter(torch.randn(n, device="cuda")) for n in (100, 7, 4097)] + [torch.nn.Parameter(torch.ones(3, device="cuda"))]
    for p in ps[:3]:
        p.grad = torch.randn_like(p)
    want = torch.cat([p.grad for p in ps[:3]]).double().norm()
    norm = nn.clip_grad_norm_(ps, 1.0)
    assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
    assert abs(float(torch.cat([p.grad for p in ps[:3]]).double().norm()) - 1.0) <= 1e-6
    assert float(nn.clip_grad_norm_([ps[3]], 1.0)) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_example_step_is_reproducible_and_learns(dtype):
    spec = importlib.util.spec_from_file_location("adapter_moe_step", os.path.join(ROOT, "examples", "adapter_moe_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    args = dict(steps=4, rows=320, features=96, hidden=160, experts=4, adapters=3, rank=8, dtype=dtype)
    l1, n1, p1 = ex.run(**args)
    l2, n2, p2 = ex.run(**args)
    # the gate's product and the weighted sum are torch's; everything else is the library's
    assert l1 == l2 and n1 == n2
    for u, v in zip(p1, p2):
        assert torch.equal(u, v)
    assert l1[-1] < l1[0] and all(n > 0 for n in n1)


def test_clip_grad_norm_of_the_same_parameter_twice():
    """Its gradient would be scaled by two warps at once: refused, and left as it is."""
    p = torch.nn.Parameter(torch.ones(3, device="cuda"))
    p.grad = torch.full_like(p, 2.0)
    with pytest.raises(ValueError):
        nn.clip_grad_norm_([p, p], 1.0)
    assert (p.grad == 2).all()


def test_clip_grad_norm_without_gradients_stays_on_the_device():
    p = torch.nn.Parameter(torch.ones(3, device="cuda"))
    norm = nn.clip_grad_norm_([p], 1.0)
    assert norm.device == p.device and norm.shape == (1,) and norm.dtype == torch.float32 and float(norm) == 0.0


def test_adapter_linear_does_not_drop_the_gradient_of_scales():
    """There is no gradient for the scales: one that asks for it is refused, not left without."""
    x, w = torch.randn(6, 64, device="cuda"), torch.randn(64, 64, device="cuda")
    a, b = torch.randn(2, 4, 64, device="cuda", requires_grad=True), torch.randn(2, 4, 64, device="cuda")
    ids = torch.zeros(6, dtype=torch.int32, device="cuda")
    scales = torch.ones(2, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        nn.adapter_linear(x, w, None, a, b, scales, ids)
    nn.adapter_linear(x, w, None, a, b, scales.detach(), ids).sum().backward()
    assert a.grad is not None
    with torch.no_grad():  # no gradient is asked for here
        nn.adapter_linear(x, w, None, a, b, scales, ids)


def test_second_derivatives_are_refused():
    """The backward passes are kernels without a backward of their own: a second derivative says so."""
    x, w = torch.randn(6, 64, device="cuda", requires_grad=True), torch.randn(64, 64, device="cuda")
    a, b = torch.randn(2, 4, 64, device="cuda"), torch.randn(2, 4, 64, device="cuda")
    ids = torch.zeros(6, dtype=torch.int32, device="cuda")
    y = nn.adapter_linear(x, w, None, a, b, None, ids)
    gx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (gx.square().sum() + x.sum()).backward()
    logits = torch.randn(6, 8, device="cuda", requires_grad=True)
    _, weights, loss, _ = nn.route(logits, 2)
    gl, = torch.autograd.grad(weights.square().sum() + loss, logits, create_graph=True)
    with pytest.raises(RuntimeError):
        (gl.square().sum() + logits.sum()).backward()
