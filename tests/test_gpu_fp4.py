"""MXFP4 quantization and the products of it, against 64 bits.

Quantization is exact: codes, scale bytes and padding are compared as they are.

Tolerance of a product of depth K, element by element, with S = sum |a b| (+ |bias|):
the accumulator takes ceil(K / 64) blocks, each addition and each block's own sum off
by at most one step of f32 at a partial sum's magnitude (2^-23, truncation allowed),
f32 pieces and the bias as many more additions: (ceil(K/64) + K/8192 + 4) 2^-23 S,
and half a step of the output's type.  Problems on small integers are exact.
"""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
import fp4_ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half a subnormal step


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    torch.cuda.synchronize()
    e.close()


def f64(t):
    return t.detach().double().cpu().numpy()


def buffers(rows, cols):
    q, s = bi.fp4_buffers(rows, cols)
    q.fill_(0xAB)
    s.fill_(0xCD)
    return q, s


def quantized(eng, x, both=True):
    r, c = x.shape
    a, b = buffers(r, c), buffers(c, r)
    eng.fp4_quantize(*a, *(b if both else (None, None)), x, r, c, x.dtype)
    return a, b


def operand(eng, v):
    """v [R, C] f32 on the GPU as an operand, and its values in 64 bits."""
    a, _ = quantized(eng, v.contiguous(), both=False)
    return a, fp4_ref.rounded(f64(v))


def check_operand(bufs, want64, rows, cols):
    torch.cuda.synchronize()
    codes, scales, clean = fp4_ref.unpack(*(b.cpu().numpy() for b in bufs), rows, cols)
    wc, ws = fp4_ref.quantize(want64)
    assert np.array_equal(scales, ws)
    assert np.array_equal(codes, wc)
    assert clean


SIZES = [(1, 1), (1, 32), (3, 33), (31, 257), (128, 128), (130, 255), (333, 1000), (64, 4096), (2049, 40)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_exact(eng, rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, device="cuda", generator=gen) * torch.exp(2 * torch.randn(rows, cols, device="cuda", generator=gen))
    x = x.to(TYPES[dtype])
    a, b = quantized(eng, x)
    check_operand(a, f64(x), rows, cols)
    check_operand(b, f64(x).T, cols, rows)
    # one direction alone writes the same
    one, other = buffers(rows, cols), buffers(cols, rows)
    eng.fp4_quantize(*one, None, None, x, rows, cols, dtype)
    eng.fp4_quantize(None, None, *other, x, rows, cols, dtype)
    for got, want in zip(one + other, a + b):
        assert torch.equal(got, want)
    back = torch.empty_like(x)
    eng.fp4_dequantize(back, *a, rows, cols, dtype)
    assert np.array_equal(f64(back), fp4_ref.rounded(f64(x)))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_off_alignment(eng, dtype):
    """A source that starts one element off 16 bytes, and rows that do."""
    x = torch.randn(41 * 136 + 1, device="cuda").to(TYPES[dtype])[1:].view(41, 136)
    a, b = quantized(eng, x)
    check_operand(a, f64(x), 41, 136)
    check_operand(b, f64(x).T, 136, 41)


def test_quantize_borders_and_specials(eng):
    """Every border between two codes at several scales, signs, subnormals, the largest numbers, zeros, infinities, NaN."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = np.concatenate([np.nextafter(mids.astype(np.float32), np.float32(9)), mids, np.nextafter(mids.astype(np.float32), np.float32(0))])
    row = np.zeros(32)
    row[:21], row[21:25], row[25:29] = near, [4.0, 6.0, 7.999, 0.0], [-0.0, -2.5, -5.0, -0.25]
    rows = [row * 2.0 ** e for e in (-60, -3, 0, 7, 100)]
    tiny = np.float32(2.0 ** -149)
    rows += [np.arange(32) * float(tiny), np.arange(32) * float(tiny) * 2 ** 20, np.zeros(32), -np.zeros(32)]
    top = float(np.finfo(np.float32).max)
    rows.append(np.where(np.arange(32) % 2, top, -top / np.arange(1, 33)))
    for v in (np.inf, -np.inf, np.nan):
        r = np.ones(32)
        r[5] = v
        rows.append(r)
    x = torch.tensor(np.stack(rows).astype(np.float32), device="cuda")
    a, b = quantized(eng, x)
    check_operand(a, f64(x), *x.shape)
    check_operand(b, f64(x).T, *x.T.shape)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(eng, dtype):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    q, s = (torch.from_numpy(v).cuda() for v in fp4_ref.pack(codes, scales))
    out = torch.empty(256, 32, device="cuda", dtype=TYPES[dtype])
    eng.fp4_dequantize(out, q, s, 256, 32, dtype)
    want = torch.from_numpy(fp4_ref.values(codes, scales)).to(TYPES[dtype])
    assert torch.equal(torch.nan_to_num(out.cpu().double(), nan=7.25), torch.nan_to_num(want.double(), nan=7.25))


def check_product(out, a64, b64, bias64, dtype):
    k = a64.shape[1]
    want, S = a64 @ b64.T, np.abs(a64) @ np.abs(b64).T
    if bias64 is not None:
        want, S = want + bias64, S + np.abs(bias64)
    err = np.abs(f64(out) - want)
    tol = (-(-k // 64) + k / 8192 + 4) * 2.0 ** -23 * S
    tol = tol + HALF[dtype] * (np.abs(want) + tol) + TINY[dtype]
    assert (err <= tol).all(), (err / tol).max()


# m, n, k: single elements, tile edges, ragged rows and columns, more tiles than CTA pairs, pieces of 8192
SHAPES = [(1, 1, 1), (1, 8, 32), (3, 5, 7), (1, 520, 300), (128, 256, 256), (129, 257, 513), (300, 520, 1000), (256, 256, 4096),
          (513, 768, 768), (1, 11008, 256), (2600, 2600, 320), (70, 40, 8192 + 300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(eng, m, n, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m + 3 * n + 7 * k)
    a, a64 = operand(eng, torch.randn(m, k, device="cuda", generator=gen))
    b, b64 = operand(eng, torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5)
    bias = torch.randn(n, device="cuda", generator=gen).to(TYPES[dtype])
    y = torch.full((m, n), 77.0, device="cuda").to(TYPES[dtype])
    eng.fp4_forward(y, *a, *b, bias, m, k, n, dtype)
    eng.check()
    check_product(y, a64, b64, f64(bias), dtype)
    again = torch.empty_like(y)
    eng.fp4_forward(again, *a, *b, bias, m, k, n, dtype)
    assert torch.equal(y, again)
    # the other passes are the same product with the sizes in other places
    dx, dw = torch.empty(m, n, device="cuda", dtype=TYPES[dtype]), torch.empty(m, n, device="cuda", dtype=TYPES[dtype])
    eng.fp4_backward_dx(dx, *a, *b, m, n, k, dtype)
    eng.fp4_backward_dw(dw, *a, *b, k, m, n, dtype)
    check_product(dx, a64, b64, None, dtype)
    assert torch.equal(dx, dw)


def test_integers_are_exact(eng):
    """Values 0, .5, 1, .. 6 with a scale of 1: every partial sum is a multiple of 1/4 below 2^22."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    table = torch.tensor(list(fp4_ref.VALUES) + [-v for v in fp4_ref.VALUES], device="cuda", dtype=torch.float32)
    a, b = (table[torch.randint(0, 16, s, device="cuda", generator=gen)] for s in ((300, 4000), (270, 4000)))
    a[:, ::32] = b[:, ::32] = 6.0  # the block's largest: scale 1
    (qa, a64), (qb, b64) = operand(eng, a), operand(eng, b)
    assert np.array_equal(a64, f64(a)) and np.array_equal(b64, f64(b))
    y = torch.empty(300, 270, device="cuda")
    eng.fp4_forward(y, *qa, *qb, None, 300, 4000, 270, "f32")
    assert np.array_equal(f64(y), a64 @ b64.T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_do_not_depend_on_the_batch(eng, dtype):
    k, n = 1100, 648
    x = torch.randn(700, k, device="cuda")
    w, _ = operand(eng, torch.randn(n, k, device="cuda"))
    whole = torch.empty(700, n, device="cuda", dtype=TYPES[dtype])
    eng.fp4_forward(whole, *operand(eng, x)[0], *w, None, 700, k, n, dtype)
    for rows in (slice(0, 1), slice(130, 133), slice(255, 700)):
        part = x[rows].contiguous()
        y = torch.empty(len(part), n, device="cuda", dtype=TYPES[dtype])
        eng.fp4_forward(y, *operand(eng, part)[0], *w, None, len(part), k, n, dtype)
        assert torch.equal(y, whole[rows])


def test_nan_and_extreme_scales_stay_in_their_rows(eng):
    m, n, k = 200, 300, 600
    a, b = torch.randn(m, k, device="cuda"), torch.randn(n, k, device="cuda")
    clean = torch.empty(m, n, device="cuda")
    eng.fp4_forward(clean, *operand(eng, a)[0], *operand(eng, b)[0], None, m, k, n, "f32")
    a[7, 40], a[150, 599], b[280, 3] = float("nan"), float("inf"), float("-inf")
    a[11] *= 2.0 ** -100
    y = torch.empty(m, n, device="cuda")
    eng.fp4_forward(y, *operand(eng, a)[0], *operand(eng, b)[0], None, m, k, n, "f32")
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[7, 150]] = True
    bad[:, 280] = True
    assert torch.equal(torch.isnan(y), bad)
    clean[11] *= 2.0 ** -100  # exact: the values and every partial sum scale by a power of two
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("n", [264, 263])
def test_outputs_stay_in_bounds(eng, n):
    m, k = 131, 300
    a, b = operand(eng, torch.randn(m, k, device="cuda"))[0], operand(eng, torch.randn(n, k, device="cuda"))[0]
    for dtype in TYPES:
        for off in (64, 65):  # aligned to 16 bytes, and not
            buf = torch.full((m * n + 130,), 3.0, device="cuda", dtype=TYPES[dtype])
            y = buf[off:off + m * n].view(m, n)
            eng.fp4_forward(y, *a, *b, None, m, k, n, dtype)
            assert (buf[:off] == 3).all() and (buf[off + m * n:] == 3).all()
            z = torch.empty(m, n, device="cuda", dtype=TYPES[dtype])
            eng.fp4_forward(z, *a, *b, None, m, k, n, dtype)
            assert torch.equal(y, z)


def test_no_rows(eng):
    e = torch.empty(0, device="cuda")
    q, s = bi.fp4_buffers(0, 64)
    eng.fp4_quantize(q, s, None, None, e, 0, 64, "f32")
    w, _ = operand(eng, torch.randn(8, 64, device="cuda"))
    eng.fp4_forward(e, q, s, *w, None, 0, 64, 8, "f32")
    dw = torch.full((64, 8), 5.0, device="cuda")
    eng.fp4_backward_dw(dw, *bi.fp4_buffers(64, 0), *bi.fp4_buffers(8, 0), 0, 64, 8, "f32")
    assert not dw.any()


def test_captured_and_replayed(eng):
    m, k, n = 150, 500, 400
    x = torch.randn(m, k, device="cuda")
    w, _ = operand(eng, torch.randn(n, k, device="cuda"))
    xq, y = buffers(m, k), torch.empty(m, n, device="cuda")

    def step():
        eng.fp4_quantize(*xq, None, None, x, m, k, "f32")
        eng.fp4_forward(y, *xq, *w, None, m, k, n, "f32")
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(torch.randn(m, k, device="cuda"))
    g.replay()
    got = y.clone()
    step()
    assert torch.equal(got, y)


@pytest.mark.parametrize("m,k,n", [(8500, 96, 530), (4400, 8500, 530)])
def test_many_row_tiles(eng, m, k, n):
    """More row tiles than share a sweep over the columns, the last group a short one: the
    rows are those of calls with few."""
    a, _ = quantized(eng, torch.randn(m, k, device="cuda", dtype=torch.bfloat16), both=False)
    b, _ = quantized(eng, torch.randn(n, k, device="cuda", dtype=torch.bfloat16), both=False)
    y = torch.full((m, n), 7.0, device="cuda", dtype=torch.bfloat16)
    eng.fp4_forward(y, *a, *b, None, m, k, n, "bf16")
    cp = -(-k // 256) * 256
    z = torch.empty_like(y)
    for r in range(0, m, 1024):  # whole pieces of scales
        c = min(1024, m - r)
        eng.fp4_forward(z[r:r + c], a[0][r * cp // 2:], a[1][r // 128 * cp * 4:], *b, None, c, k, n, "bf16")
    assert torch.equal(y, z)
