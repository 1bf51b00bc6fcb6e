"""The MXFP4 expert layer over many experts and choices, whose lists leave the ring in
shared memory fewer stages than the kernel has warps for the weights' scales, with
contractions of several stages and blocks that go round the ring many times.

Some rows against 64 bits (tests/test_gpu_moe.py has the tolerance) and, bit for bit,
against calls of that row alone, whose ring is deep.  Weights are random codes, made on the
GPU; sizes are multiples of a piece of scales, so an expert's part can be dequantized alone.
"""
import math

import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
from deterministic_invariant_gemm_fixed_gb300 import nn
from test_gpu_moe import TYPES, check, f64, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    torch.cuda.synchronize()
    e.close()


def weight(gen, e, rows, length):
    """Random codes with scales that make an inner product about 1."""
    assert rows % 128 == 0 and length % 256 == 0
    q = torch.randint(0, 256, (e * rows * length // 2,), dtype=torch.uint8, device="cuda", generator=gen)
    byte = 127 - round(math.log2(3 * math.sqrt(length)))
    s = torch.randint(byte - 1, byte + 2, (e * rows * length // 32,), dtype=torch.uint8, device="cuda", generator=gen)
    return q, s


def of_experts(eng, pair, e, experts, rows, length):
    """Their weights in 64 bits."""
    out = []
    for j in experts:
        v = torch.empty(rows, length, device="cuda")
        q, s = (b[j * (b.numel() // e):(j + 1) * (b.numel() // e)] for b in pair)
        eng.fp4_dequantize(v, q, s, rows, length, "f32")
        out.append(f64(v))
    return np.stack(out)


# t, c, e, k, f, n
SHAPES = [(64, 8, 512, 512, 256, 512), (32, 2, 1024, 2048, 512, 1024), (512, 4, 1024, 512, 256, 512), (53, 8, 256, 1024, 512, 2048),
          (256, 8, 256, 1024, 512, 512), (200, 8, 128, 2048, 512, 1024), (256, 8, 64, 2048, 1024, 2048), (17, 10, 512, 512, 512, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,c,e,k,f,n", SHAPES)
def test_many_experts(eng, t, c, e, k, f, n, dtype):
    gen = torch.Generator(device="cuda").manual_seed(t + e)
    gate, up, down = weight(gen, e, f, k), weight(gen, e, f, k), weight(gen, e, n, f)
    x = torch.randn(t, k, device="cuda", generator=gen).to(TYPES[dtype])
    ids = torch.rand(t, e, device="cuda", generator=gen).argsort(1)[:, :c].to(torch.int32).contiguous()
    p = torch.rand(t, c, device="cuda", generator=gen)
    y = torch.full((t, n), 9.0, device="cuda").to(TYPES[dtype])
    eng.moe_forward_fp4(y, x, ids, p, *gate, *up, *down, t, c, k, f, n, e, "silu", dtype)
    eng.check()
    again = torch.empty_like(y)
    eng.moe_forward_fp4(again, x, ids, p, *gate, *up, *down, t, c, k, f, n, e, "silu", dtype)
    assert torch.equal(again, y)
    for r in {0, 1, t // 3, t // 2, t - 2, t - 1}:
        one = torch.empty(1, n, device="cuda", dtype=y.dtype)
        eng.moe_forward_fp4(one, x[r:r + 1], ids[r:r + 1], p[r:r + 1], *gate, *up, *down, 1, c, k, f, n, e, "silu", dtype)
        assert torch.equal(one[0], y[r]), r
    rows = [0, t // 2, t - 1]
    chosen = sorted(set(ids[rows].flatten().tolist()))
    near = np.vectorize(chosen.index)(ids[rows].cpu().numpy())
    w = [of_experts(eng, v, e, chosen, r, length) for v, r, length in ((gate, f, k), (up, f, k), (down, n, f))]
    check(y[rows], reference(f64(x[rows]), near, f64(p[rows]), *w, "silu"), dtype)
    eng.check()


def test_layer_behind_its_router_in_several_calls():
    """nn.moe cuts 600 tokens of 8 choices each, over 64 experts, into calls of at most 2048 choices."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    e, k, f, n, t, c = 64, 512, 384, 256, 600, 8
    def w(*s):
        return (torch.randn(*s, device="cuda", generator=gen) * s[2] ** -0.5).bfloat16()
    experts = [nn.Fp4Weight.quantize(v) for v in (w(e, f, k), w(e, f, k), w(e, n, f))]
    x, logits = torch.randn(t, k, device="cuda", generator=gen).bfloat16(), torch.randn(t, e, device="cuda", generator=gen)
    with torch.no_grad():
        y = nn.moe(x, logits, *experts, c)
        for r in (0, 255, 256, 599):
            assert torch.equal(nn.moe(x[r:r + 1], logits[r:r + 1], *experts, c), y[r:r + 1])
        ids, p, _, _ = nn.route(logits, c)
    rows = [0, 130, 255, 256, 511, 512, 599]
    check(y[rows], reference(f64(x[rows]), ids[rows].cpu().numpy(), f64(p[rows]), *[f64(v.dequantize()) for v in experts], "silu"), "bf16")
    nn.engine_for(x.device).check()
