"""Gradient norm and clipping against 64 bits.

The norm: a chunk of 32768 elements is summed with 512 threads of at most 8
squares per running sum and f32 trees, at most (8 + 3 + 5) roundings of 2^-24 on
positive terms behind any of them for f32 inputs and 16-bit inputs alike (64
elements a thread, 8 running sums); then f64; the square root halves the
relative error and rounds once: 10 * 2^-24.  A scaled element: the norm's error,
the division and the product, one rounding each: 14 * 2^-24, plus the output's
rounding.
"""
import math

import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
from helpers import ulp_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    e.close()


def make(sizes, dtypes, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, device="cuda", generator=gen) * std).to(t) for n, t in zip(sizes, dtypes)]


def norm64(ts):
    return math.sqrt(sum(float(np.dot(v, v)) for v in (t.double().cpu().numpy() for t in ts)))


F, B, H = torch.float32, torch.bfloat16, torch.float16
SETS = [([1], [F]), ([7, 1, 0, 33], [B, F, H, H]), ([32768, 32769, 32767], [F, B, H]), ([100003, 5, 4096 * 64], [B, B, F]),
        ([1000] * 300, [F, B, H] * 100), ([0, 0, 12, 0], [F] * 4), ([3000001], [H])]


@pytest.mark.parametrize("limit", [0.5, 1e9])
@pytest.mark.parametrize("sizes,dtypes", SETS)
def test_norm_and_clip(eng, sizes, dtypes, limit):
    src = make(sizes, dtypes, seed=len(sizes))
    keep = [t.clone() for t in src]
    dst = [torch.full_like(t, float("nan")) for t in src]
    norm = torch.empty(1, device="cuda")
    eng.clip_gradients(dst, src, norm, limit)
    want = norm64(src)
    assert abs(float(norm) - want) <= 10 * U * want
    c = limit / want if want > limit else 1.0
    for s, k, d in zip(src, keep, dst):
        assert torch.equal(s, k)
        if c == 1.0:
            assert torch.equal(d, s)
            continue
        w, g = k.double().cpu().numpy() * c, d.double().cpu().numpy()
        dt = {F: "f32", B: "bf16", H: "f16"}[s.dtype]
        tol = 14 * U * abs(w) + 0.5 * ulp_of(np.maximum(abs(w), abs(g)), dt)
        assert (abs(g - w) <= tol).all()
    again = torch.empty(1, device="cuda")
    eng.grad_norm(again, src)
    assert torch.equal(norm, again)
    eng.clip_gradients(src, src, norm, limit)  # in place
    for s, d in zip(src, dst):
        assert torch.equal(s, d)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e25, 3e37])
def test_norm_where_squares_leave_f32(eng, scale):
    """Squares under- or overflow f32: the sum is taken again in f64, whose own error is below 2^-40."""
    src = make([40000, 100], [F, B], std=1.0)
    src = [(t.double() * scale).to(t.dtype) for t in src]
    norm = torch.empty(1, device="cuda")
    eng.grad_norm(norm, src)
    want = norm64(src)
    if want < 3.4e38:
        assert abs(float(norm) - want) <= 2 * U * want
    else:
        assert math.isinf(float(norm))


def test_mixed_magnitudes_and_zeros(eng):
    z = torch.zeros(70000, device="cuda")
    big = torch.full((10,), 2e19, device="cuda")
    small = torch.full((40000,), 1e-25, device="cuda")
    norm = torch.empty(1, device="cuda")
    for ts in ([z], [z, small], [z, big, small], [small]):
        eng.grad_norm(norm, ts)
        assert abs(float(norm) - norm64(ts)) <= 10 * U * norm64(ts)


def test_not_finite(eng):
    a, b = torch.ones(100, device="cuda"), torch.ones(33000, device="cuda", dtype=torch.bfloat16)
    norm = torch.empty(1, device="cuda")
    b[40] = float("inf")
    eng.clip_gradients([a, b], [a, b], norm, 1.0)
    assert math.isinf(float(norm)) and not a.any() and math.isnan(float(b[40])) and not b[:40].any()
    a = torch.ones(100, device="cuda")
    a[3] = float("nan")
    eng.clip_gradients([a], [a], norm, 1e9)
    assert math.isnan(float(norm)) and torch.isnan(a).all()


def test_unaligned_views_and_neighbours(eng):
    """Views off 16-byte alignment, with the elements around them left alone."""
    for dt in (F, B, H):
        buf = make([1000], [dt], seed=3)[0]
        ref = buf.clone()
        v = [buf[1:400], buf[403:999]]
        norm = torch.empty(1, device="cuda")
        want = norm64(v)
        eng.clip_gradients(v, v, norm, 1.0)
        assert abs(float(norm) - want) <= 10 * U * want
        for i in (0, 400, 401, 402, 999):
            assert torch.equal(buf[i], ref[i])
        assert abs(norm64(v) - 1.0) <= (2 ** -7 if dt is B else 2 ** -10)


def test_limit_zero_empty_and_refusals(eng):
    t = make([50], [F])
    norm = torch.empty(1, device="cuda")
    eng.clip_gradients(t, t, norm, 0.0)
    assert not t[0].any()
    eng.grad_norm(norm, [])
    assert float(norm) == 0.0
    eng.grad_clip([], [], norm, 1.0)
    t = make([50], [F])
    s = bi.TensorSet(t)
    assert len(s) == 1
    assert bi.bi_grad_norm(eng.handle, None, s) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_clip(eng.handle, s, s, norm, -1.0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_clip(eng.handle, s, s, norm, float("nan")) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_clip(eng.handle, s, s, None, 1.0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_norm(None, norm, s) == bi.BI_ERR_INVALID_ARG
    s.dtypes[0] = 9
    assert bi.bi_grad_norm(eng.handle, norm, s) == bi.BI_ERR_INVALID_ARG
    s = bi.TensorSet(t)
    s.counts[0] = -1
    assert bi.bi_grad_norm(eng.handle, norm, s) == bi.BI_ERR_INVALID_ARG
    s = bi.TensorSet(t)
    s.ptrs[0] = s.ptrs[0] + 2
    assert bi.bi_grad_norm(eng.handle, norm, s) == bi.BI_ERR_MISALIGNED
    with pytest.raises(ValueError):
        eng.grad_clip(make([49], [F]), t, norm, 1.0)
    with pytest.raises(ValueError):
        bi.TensorSet([torch.zeros(4)])
    with pytest.raises(ValueError):
        bi.TensorSet([torch.zeros(4, 4, device="cuda").t()])
    bi.bi_engine_fail_allocations(eng.handle, 1)
    assert bi.bi_grad_norm(eng.handle, norm, bi.TensorSet(t)) == bi.BI_ERR_OOM
    bi.bi_engine_fail_allocations(eng.handle, 0)


def test_offsets_beyond_32_bits(eng):
    """One tensor of more than 2^31 elements: its last elements count and are scaled."""
    n = (1 << 31) + 4096 + 3
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-2:] = 3.0
    t[0] = 4.0
    norm = torch.empty(1, device="cuda")
    eng.clip_gradients([t], [t], norm, math.sqrt(34.0) / 2)
    assert abs(float(norm) - math.sqrt(34.0)) <= 10 * U * 6
    assert t[[0, n - 2, n - 1]].tolist() == [2.0, 1.5, 1.5] and not t[1:1000].any()


@pytest.mark.parametrize("sizes,dtypes", SETS + [([4000] * 700, [F] * 700)])
def test_one_call_equals_two(eng, sizes, dtypes):
    src = make(sizes, dtypes, seed=9)
    a, b = [torch.empty_like(t) for t in src], [torch.empty_like(t) for t in src]
    n1, n2 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    eng.grad_norm(n1, src)
    eng.grad_clip(a, src, n1, 0.75)
    eng.clip_gradients(b, src, n2, 0.75)
    assert torch.equal(n1, n2) and all(torch.equal(p, q) for p, q in zip(a, b))
    s = bi.TensorSet(src)
    assert bi.bi_grad_norm_clip(eng.handle, s, s, n1, -1.0) == bi.BI_ERR_INVALID_ARG
    assert bi.bi_grad_norm_clip(eng.handle, s, s, None, 1.0) == bi.BI_ERR_INVALID_ARG


def test_a_set_follows_its_tensors(eng):
    """A tensor whose storage was replaced or resized: the set's next call goes to the new one."""
    a, b = torch.full((9,), 2.0, device="cuda"), torch.full((5,), 1.0, device="cuda", dtype=torch.bfloat16)
    s, norm = bi.TensorSet([a, b]), torch.empty(1, device="cuda")
    eng.grad_norm(norm, s)
    assert abs(float(norm) - math.sqrt(41.0)) <= 10 * U * 7
    old = a.data  # (kept, so that its memory is not given away while this test runs)
    a.data = torch.full((4, 4), 3.0, device="cuda")
    eng.clip_gradients(s, s, norm, math.sqrt(149.0) / 2)
    assert abs(float(norm) - math.sqrt(149.0)) <= 10 * U * 13
    assert torch.allclose(a, torch.full_like(a, 1.5)) and torch.equal(old, torch.full_like(old, 2.0))
    with torch.no_grad():
        b.set_(torch.full((70,), 4.0, device="cuda", dtype=torch.bfloat16).untyped_storage(), 8, (3,), (1,))
        a.resize_(2)
    eng.grad_norm(norm, s)
    assert abs(float(norm) - math.sqrt(2 * 1.5 ** 2 + 3 * 16.0)) <= 10 * U * 8
    d = bi.TensorSet([torch.empty_like(a), torch.empty_like(b)])
    eng.grad_clip(d, s, norm, 1.0e9)
    b.data = torch.ones(6, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        eng.grad_clip(d, s, norm, 1.0e9)  # the two sets no longer match
    a.data = torch.ones(4, 4, device="cuda").t()[:2]
    with pytest.raises(ValueError):
        eng.grad_norm(norm, s)


def test_a_tensor_twice_in_a_set(eng):
    """Its squares count twice; scaling it in place would be a race, and is refused."""
    t = torch.full((8,), 2.0, device="cuda")
    norm = torch.empty(1, device="cuda")
    eng.grad_norm(norm, [t, t])
    assert float(norm) == 8.0
    for call in (lambda: eng.clip_gradients([t, t], [t, t], norm, 1.0), lambda: eng.grad_clip([t, t], [t.clone(), t], norm, 1.0)):
        with pytest.raises(ValueError):
            call()
    assert (t == 2).all()


@pytest.mark.parametrize("dtype", [F, B, H])
@pytest.mark.parametrize("n", [5, 64, 1000, 2048 * 3 + 9, 700001])
def test_results_do_not_depend_on_alignment(eng, n, dtype):
    """The same values at any offset of a buffer: the same norm and the same scaled values, bit for bit.
    (Few values each of many times: a long sum's rounding to f32 hides the order of its additions.)"""
    for seed in range(40 if n < 5000 else 3):
        val = make([n], [dtype], seed=seed)[0]
        want, norm = torch.empty_like(val), torch.empty(1, device="cuda")
        eng.clip_gradients([want], [val], norm, 0.5)
        for off in (1, 2, 3, 5, 7):
            buf = torch.zeros(n + 16, dtype=dtype, device="cuda")
            v = buf[off:off + n]
            v.copy_(val)
            got = torch.empty(1, device="cuda")
            eng.grad_norm(got, [v])
            assert torch.equal(got, norm), (seed, off, float(got), float(norm))
            eng.clip_gradients([v], [v], got, 0.5)
            assert torch.equal(got, norm) and torch.equal(v, want)
            assert not buf[:off].any() and not buf[off + n:].any()


@pytest.mark.parametrize("sizes,dtypes", SETS)
def test_norm_within_its_own_bound(eng, sizes, dtypes):
    """16 or 32 squares in 8 running sums: at most 2 roundings of an f32 square and its addition, or 3
    additions of 16-bit squares (exact in f32), then 3 additions of the sums, 6 * 2^-24 on positive
    terms; f64 from there (its own error below 2^-40); the root halves it and rounds once: 4 * 2^-24."""
    for seed in range(5):
        src = make(sizes, dtypes, seed=seed)
        norm = torch.empty(1, device="cuda")
        eng.grad_norm(norm, src)
        want = norm64(src)
        assert abs(float(norm) - want) <= (4 * U + 2.0 ** -40) * want
