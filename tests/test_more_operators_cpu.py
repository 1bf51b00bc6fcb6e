"""MXFP4 and the expert layer on a machine without a GPU: calls refuse bad arguments on
the host, buffers have the documented sizes, the reference of the 4-bit tests and the timed
cases are well formed."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

import fp4_ref
from conftest import ROOT


@pytest.fixture(scope="module")
def bi():
    from deterministic_invariant_gemm_fixed_gb300 import build as _b
    try:
        _b.build()
    except FileNotFoundError as e:
        pytest.skip(f"cannot build the library here: {e}")
    import deterministic_invariant_gemm_fixed_gb300 as m
    m.library()
    return m


def test_null_engine_is_rejected_on_the_host(bi):
    p = 16
    calls = [lambda: bi.bi_fp4_quantize(None, p, p, None, None, p, 4, 32, "bf16", 0),
             lambda: bi.bi_fp4_dequantize(None, p, p, p, 4, 32, "bf16", 0),
             lambda: bi.bi_fp4_forward(None, p, p, p, p, p, None, 4, 32, 8, "bf16", 0),
             lambda: bi.bi_fp4_backward_dx(None, p, p, p, p, p, 4, 32, 8, "bf16", 0),
             lambda: bi.bi_fp4_backward_dw(None, p, p, p, p, p, 4, 32, 8, "f32", 0),
             lambda: bi.bi_moe_forward(None, p, p, p, p, p, p, p, 4, 2, 32, 16, 8, 4, "silu", "bf16", 0),
             lambda: bi.bi_moe_forward_fp4(None, *[p] * 10, 4, 2, 32, 16, 8, 4, "relu", "bf16", 0)]
    for call in calls:
        assert call() == bi.BI_ERR_INVALID_ARG
        assert "NULL" in bi.bi_last_error(None)


def test_buffer_sizes(bi):
    for rows, cols in ((0, 1), (1, 1), (128, 256), (129, 257), (1000, 8192)):
        q, s = fp4_ref.pack(np.zeros((rows, cols), np.uint8), np.zeros((rows, -(-cols // 32)), np.uint8))
        assert (bi.bi_fp4_code_bytes(rows, cols), bi.bi_fp4_scale_bytes(rows, cols)) == (q.size, s.size)
    assert bi.bi_fp4_code_bytes(-1, 8) == bi.bi_fp4_scale_bytes(8, 2 ** 31) == -1
    with pytest.raises(ValueError):
        bi.fp4_buffers(2 ** 31, 8, device="cpu")


def test_wrong_tensors_are_refused(bi):
    q, s = bi.fp4_buffers(4, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        bi.bi_fp4_dequantize(None, 16, q, s, 4, 64, "f32", 0)
    with pytest.raises(ValueError, match="bytes"):  # too small for the sizes
        bi.bi_fp4_dequantize(None, 16, q, s, 5, 64, "f32", 0)
    with pytest.raises(ValueError, match="bytes"):
        bi.bi_fp4_quantize(None, None, None, q, s, 16, 4, 64, "f32", 0)
    with pytest.raises(ValueError, match="activation"):
        bi.bi_moe_forward(None, *[16] * 7, 4, 2, 32, 16, 8, 4, "tanh", "bf16", 0)
    from deterministic_invariant_gemm_fixed_gb300 import nn
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        nn.deterministic_linear(x, torch.zeros(8, 4), fp4=True)
    with pytest.raises(ValueError):
        nn.Fp4Weight.quantize(torch.zeros(2, 4, 8))
    with pytest.raises(ValueError):
        nn.moe(x, torch.zeros(2, 4), None, torch.zeros(4, 8, 8), torch.zeros(4, 8, 8), 2)


def test_reference_is_the_definition():
    """A value at a time, from the words of the format."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((6, 70)) * np.exp(3 * rng.standard_normal((6, 70)))).astype(np.float32).astype(np.float64)
    x[2, 32:64] = 0
    got = fp4_ref.rounded(x)
    grid = sorted({s * v for v in fp4_ref.VALUES for s in (1, -1)})
    for i in range(6):
        for b in range(0, 70, 32):
            blk = x[i, b:b + 32]
            top = np.abs(blk).max()
            scale = 0.0
            if top:
                scale = 2.0 ** -127
                while 8 * scale <= top:
                    scale *= 2
            for j, v in enumerate(blk):
                want = min((abs(v / scale - g), g) for g in grid)[0] if scale else 0.0
                assert abs(got[i, b + j] - v) == pytest.approx(want * scale, abs=0)
    codes, scales = fp4_ref.quantize(x)
    q, s = fp4_ref.pack(codes, scales)
    c2, s2, clean = fp4_ref.unpack(q, s, 6, 70)
    assert clean and np.array_equal(c2, codes) and np.array_equal(s2, scales)


def test_timed_cases_are_well_formed():
    spec = importlib.util.spec_from_file_location("more_operators_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    assert len({c["name"] for c in cases}) == len(cases)
    rng = random.Random(3)
    for c in cases + [m.draw(rng) for _ in range(50)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
        if c["op"].startswith("moe"):
            assert c["t"] * c["c"] <= 2048 and c["c"] <= c["e"]
    x = np.random.default_rng(0).standard_normal((9, 77)).astype(np.float32).astype(np.float64)
    assert np.array_equal(m._np_fp4(x), fp4_ref.rounded(x))
