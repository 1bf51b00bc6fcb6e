"""MXFP4 and the expert layer: allocation failure, refused sizes, calls side by side on streams."""
import random

import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi

pytestmark = pytest.mark.gpu


@pytest.fixture()
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    torch.cuda.synchronize()
    e.close()


def experts(dtype, t, c, k, f, n, e, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return (torch.randn(*s, device="cuda", generator=gen) * s[-1] ** -0.5).to(dtype)
    ids = torch.randint(0, e, (t, c), device="cuda", generator=gen, dtype=torch.int32)
    return r(t, k), ids, torch.rand(t, c, device="cuda", generator=gen), r(e, f, k), r(e, f, k), r(e, n, f)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_allocation_failure_leaves_the_output(eng, dtype):
    x, ids, p, g, u, d = experts(dtype, 4, 2, 64, 48, 40, 3)
    y = torch.full((4, 40), 7.0, device="cuda", dtype=dtype)
    before = eng.launches()
    bi.bi_engine_fail_allocations(eng.handle, 1)
    with pytest.raises(bi.BiError) as err:
        eng.moe_forward(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 3, "silu", dtype)
    assert err.value.status == bi.BI_ERR_OOM and eng.launches() == before
    torch.cuda.synchronize()
    assert (y == 7).all()
    eng.moe_forward(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 3, "silu", dtype)
    eng.check()
    assert not (y == 7).any()


def test_bad_arguments(eng):
    x, ids, p, g, u, d = experts(torch.bfloat16, 4, 2, 64, 48, 40, 3)
    y = torch.empty(4, 40, device="cuda", dtype=torch.bfloat16)
    q, s = bi.fp4_buffers(64, 64)
    def status(call):
        with pytest.raises(bi.BiError) as err:
            call()
        return err.value.status
    moe = eng.moe_forward
    INV, UNS, MIS = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED, bi.BI_ERR_MISALIGNED
    assert status(lambda: moe(y, x, ids, p, g, u, d, -1, 2, 64, 48, 40, 3, "silu", "bf16")) == INV
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 0, 64, 48, 40, 3, "silu", "bf16")) == INV
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 0, "silu", "bf16")) == INV
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 3, 7, "bf16")) == INV
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 3, "silu", 9)) == INV
    assert status(lambda: moe(y, x, None, p, g, u, d, 4, 2, 64, 48, 40, 3, "silu", "bf16")) == INV
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 1025, "silu", "bf16")) == UNS
    assert status(lambda: moe(y, x, ids, p, g, u, d, 1025, 2, 64, 48, 40, 3, "silu", "bf16")) == UNS
    assert status(lambda: moe(y, x, ids, p, g, u, d, 4, 2, 64, 2 ** 23, 40, 1024, "silu", "bf16")) == UNS
    assert status(lambda: moe(y.data_ptr() + 1, x, ids, p, g, u, d, 4, 2, 64, 48, 40, 3, "silu", "bf16")) == MIS
    a = (q.data_ptr(), s.data_ptr())
    assert status(lambda: eng.moe_forward_fp4(y, x, ids, p, *a, None, None, *a, 4, 2, 64, 8, 8, 1, "silu", "bf16")) == INV
    assert status(lambda: eng.moe_forward_fp4(y, x, ids, p, a[0], None, *a, *a, 4, 2, 64, 8, 8, 1, "silu", "bf16")) == INV
    assert status(lambda: eng.moe_forward_fp4(y, x, ids, p, a[0] + 4, a[1], *a, *a, 4, 2, 64, 8, 8, 1, "silu", "bf16")) == MIS
    assert status(lambda: eng.fp4_quantize(*a, None, None, x, -1, 64, "bf16")) == INV
    assert status(lambda: eng.fp4_quantize(*a, None, None, x, 4, 0, "bf16")) == INV
    assert status(lambda: eng.fp4_quantize(a[0], None, None, None, x, 4, 64, "bf16")) == INV
    assert status(lambda: eng.fp4_quantize(None, None, None, None, x, 4, 64, "bf16")) == INV
    assert status(lambda: eng.fp4_quantize(a[0] + 8, a[1], None, None, x, 4, 64, "bf16")) == MIS
    assert status(lambda: eng.fp4_quantize(*a, None, None, x, 2 ** 31, 64, "bf16")) == UNS
    assert status(lambda: eng.fp4_dequantize(None, *a, 4, 64, "bf16")) == INV
    assert status(lambda: eng.fp4_forward(y, *a, *a, None, 4, 0, 40, "bf16")) == INV
    assert status(lambda: eng.fp4_forward(y, *a, *a, None, 4, 64, 2 ** 24, "bf16")) == UNS
    assert status(lambda: eng.fp4_forward(y, a[0], None, *a, None, 4, 64, 40, "bf16")) == INV
    assert status(lambda: eng.fp4_forward(y, *a, a[0], a[1] + 4, None, 4, 64, 40, "bf16")) == MIS
    assert status(lambda: eng.fp4_forward(y.data_ptr() + 1, *a, *a, None, 4, 64, 40, "bf16")) == MIS


def test_streams_side_by_side(eng):
    """Calls of three streams in random order give the results they give alone."""
    def calls(seed):
        x, ids, p, g, u, d = experts(torch.bfloat16, 5, 2, 256, 128, 96, 8, seed)
        y, z, w = torch.empty(5, 96, device="cuda", dtype=torch.bfloat16), torch.empty(5, 96, device="cuda"), torch.empty(5, 128, device="cuda")
        qs = []
        for v in (g, u, d):
            q = bi.fp4_buffers(v.shape[0] * v.shape[1], v.shape[2])
            eng.fp4_quantize(*q, None, None, v, v.shape[0] * v.shape[1], v.shape[2], "bf16")
            qs += q
        xf, xq, wq = x.float(), bi.fp4_buffers(5, 256), bi.fp4_buffers(128, 256)
        eng.fp4_quantize(*wq, None, None, u[0], 128, 256, "bf16")
        def product():
            eng.fp4_quantize(*xq, None, None, xf, 5, 256, "f32")
            eng.fp4_forward(w, *xq, *wq, None, 5, 256, 128, "f32")
        return [lambda: eng.moe_forward(y, x, ids, p, g, u, d, 5, 2, 256, 128, 96, 8, "silu", "bf16"),
                lambda: eng.moe_forward_fp4(z, xf, ids, p, *qs, 5, 2, 256, 128, 96, 8, "gelu", "f32"), product], (y, z, w)

    sets = [calls(s) for s in range(3)]
    for fs, _ in sets:
        for f in fs:
            f()
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    rng = random.Random(1)
    for _ in range(40):
        for s, (fs, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                for f in rng.sample(fs, len(fs)):
                    f()
    torch.cuda.synchronize()
    for (_, outs), ref in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_tensors_of_another_stream_and_two_graphs(eng):
    """Two captured calls with scratch of their own, replayed one after the other and in turn."""
    a, b = experts(torch.float16, 6, 2, 128, 64, 64, 4, 1), experts(torch.float16, 3, 3, 128, 64, 64, 4, 2)
    outs = [torch.empty(len(v[0]), 64, device="cuda", dtype=torch.float16) for v in (a, b)]
    def run(v, y):
        x, ids, p, g, u, d = v
        eng.moe_forward(y, x, ids, p, g, u, d, len(x), ids.shape[1], 128, 64, 64, 4, "relu", "f16")
    for v, y in zip((a, b), outs):
        run(v, y)
    torch.cuda.synchronize()
    want = [y.clone() for y in outs]
    graphs = []
    for v, y in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(v, y)
        graphs.append(g)
    for y in outs:
        y.zero_()
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(outs, want))


def test_offsets_beyond_32_bits(eng):
    """A matrix of more than 2^31 elements, and expert weights of more than 2^32 bytes: the last rows and the last expert."""
    import numpy as np
    import fp4_ref
    rows, cols = 270016, 8192
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    x[-3:] = torch.randn(3, cols, device="cuda")
    q, s = bi.fp4_buffers(rows, cols)
    eng.fp4_quantize(q, s, None, None, x, rows, cols, "bf16")
    back = torch.empty_like(x)
    eng.fp4_dequantize(back, q, s, rows, cols, "bf16")
    assert np.array_equal(back[-3:].double().cpu().numpy(), fp4_ref.rounded(x[-3:].double().cpu().numpy()))
    assert not back[:-3].any()
    del x, back, q, s
    e, f, k, n = 600, 1024, 4096, 64
    up, down = torch.zeros(e, f, k, device="cuda", dtype=torch.bfloat16), torch.zeros(e, n, f, device="cuda", dtype=torch.bfloat16)
    up[-1] = torch.randn(f, k, device="cuda") / 64
    down[-1] = torch.randn(n, f, device="cuda") / 32
    xt = torch.randn(2, k, device="cuda").bfloat16()
    ids = torch.tensor([[e - 1], [0]], device="cuda", dtype=torch.int32)
    y = torch.empty(2, n, device="cuda", dtype=torch.bfloat16)
    eng.moe_forward(y, xt, ids, torch.ones(2, 1, device="cuda"), None, up, down, 2, 1, k, f, n, e, "relu", "bf16")
    want = torch.relu(xt[0].double() @ up[-1].double().T) @ down[-1].double().T
    # sums of 4096 and 1024 products in f32 (2^-15 of their magnitudes at most, which are below 64 times the result's rms)
    assert (y[0].double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 2.0 ** -9 * want.square().mean().sqrt()
    assert not y[1].any()


@pytest.mark.parametrize("dtype,off", [("bf16", 1), ("f16", 1), ("f32", 1), ("f32", 2)])
def test_matrix_off_its_types_alignment(eng, dtype, off):
    """The unquantized matrix is read and written an element at a time at least: addresses
    between elements are refused on the host."""
    x = torch.zeros(5, 64, device="cuda")
    buf = bi.fp4_buffers(4, 64)
    for call in (lambda: eng.fp4_quantize(*buf, None, None, x.data_ptr() + off, 4, 64, dtype),
                 lambda: eng.fp4_dequantize(x.data_ptr() + off, *buf, 4, 64, dtype)):
        with pytest.raises(bi.BiError) as err:
            call()
        assert err.value.status == bi.BI_ERR_MISALIGNED
    assert not x.any()
