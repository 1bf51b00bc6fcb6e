"""Adapters, router and clipping on a machine without a GPU: every call refuses bad
arguments on the host, and the timed cases are well formed."""
import importlib.util
import os
import random

import pytest
import torch

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
    assert bi.bi_adapter_forward(None, *[16] * 9, 1, 8, 8, 1, 1, "bf16", 0) == bi.BI_ERR_INVALID_ARG
    assert "NULL" in bi.bi_last_error(None)
    assert bi.bi_adapter_backward(None, *[16] * 11, 1, 8, 8, 1, 1, "bf16", 0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_router_forward(None, *[16] * 9, 1, 8, 2, 1, "f32", 0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_router_backward(None, *[16] * 9, 1, 8, 2, 1, "f32", 0) == bi.BI_ERR_INVALID_ARG
    empty = bi.TensorSet([])
    assert bi.bi_grad_norm(None, 16, empty, 0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_clip(None, empty, empty, 16, 1.0, 0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_norm_clip(None, empty, empty, 16, 1.0, 0) == bi.BI_ERR_INVALID_ARG


def test_host_tensors_are_refused(bi):
    with pytest.raises(ValueError):
        bi.TensorSet([torch.zeros(4)])
    with pytest.raises(ValueError):
        bi.bi_adapter_forward(None, torch.zeros(2, 8), *[16] * 8, 2, 8, 8, 1, 1, "f32", 0)
    from deterministic_invariant_gemm_fixed_gb300 import nn
    x, w, a, b = torch.zeros(2, 8), torch.zeros(8, 8), torch.zeros(1, 2, 8), torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        nn.adapter_linear(x, w, None, a, b, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        nn.route(torch.zeros(2, 8), 2)
    assert float(nn.clip_grad_norm_([torch.nn.Parameter(torch.zeros(3))], 1.0)) == 0.0


def test_timed_cases_are_well_formed():
    spec = importlib.util.spec_from_file_location("operators_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    assert len({c["name"] for c in cases}) == len(cases)
    rng = random.Random(3)
    for c in cases + [m.draw(rng) for _ in range(50)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
        if c["op"].startswith("adapter"):
            assert 1 <= c["runs"] <= c["m"] and c["g"] * c["r"] <= 1024 and c["r"] <= 256
        elif c["op"].startswith("route"):
            assert 1 <= c["k"] <= c["e"]
