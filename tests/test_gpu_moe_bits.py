"""What the expert layer keeps of a hidden value, and of values at the end of f32's range."""
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = bi.Engine(0)
    yield e
    torch.cuda.synchronize()
    e.close()


@pytest.mark.parametrize("off", [0, 1], ids=["aligned", "off alignment"])
def test_hidden_values_keep_24_bits_in_bf16(eng, off):
    """h = a + 2^-8 b + 2^-16 c beside hidden values a and 2^-8 b, which are taken from it again:
    2^-16 c is left, which two bf16 parts of h do not hold.  Each of the sums has three terms below 2,
    so at most six truncations of 2^-23, and the result's half step is 2^-23: within 2^-20."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    e, k, f, n = 64, 64, 64, 16
    def part(lo, hi):  # bf16 values in [1, 2): eight bits
        return 1 + torch.randint(lo, hi, (e,), device="cuda", generator=gen) / 128
    a, b, c = part(0, 128), part(0, 128), part(32, 96)
    up = torch.zeros(e, f, k, device="cuda")
    up[:, 0, 0], up[:, 0, 1], up[:, 0, 2] = a, b * 2.0 ** -8, c * 2.0 ** -16
    up[:, 1, 0], up[:, 2, 1] = a, b * 2.0 ** -8
    down = torch.zeros(e, n, f, device="cuda")
    down[:, :, 0], down[:, :, 1], down[:, :, 2] = 1, -1, -1
    def placed(t):
        out = torch.empty(t.numel() + off, device="cuda", dtype=torch.bfloat16)[off:].view(t.shape)
        return out.copy_(t)
    assert torch.equal(placed(up).float(), up)
    ids = torch.arange(e, device="cuda", dtype=torch.int32).view(e, 1)
    y = torch.empty(e, n, device="cuda", dtype=torch.bfloat16)
    eng.moe_forward(y, placed(torch.ones(e, k, device="cuda")), ids, torch.ones(e, 1, device="cuda"), None, placed(up), placed(down), e, 1, k, f, n,
                    e, "relu", "bf16")
    assert ((y.double() - (c.double() * 2.0 ** -16)[:, None]).abs() <= 2.0 ** -20).all()


def codes(eng, dtype, rows, length, values):
    """A weight [rows, length] in MXFP4, zeros but for {(row, column): value}."""
    w = torch.zeros(rows, length, device="cuda").to(TYPES[dtype])
    for at, v in values.items():
        w[at] = v
    q = bi.fp4_buffers(rows, length)
    eng.fp4_quantize(*q, None, None, w, rows, length, dtype)
    return q


# Values near 2^128, of which the nearest code is 4 * 2^126.  The weights are powers of two, so every sum has one
# term in eight parts, which stand for x and h to 2^-23 of their block's largest: with the parts' sums and the
# products 20 roundings of 2^-23, and the result's half step.
@pytest.mark.parametrize("top", [2.9e38, 3.3e38, 3.38e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_x_at_the_end_of_f32s_range(eng, dtype, top):
    k, f, n = 96, 64, 40
    x = torch.zeros(2, k, device="cuda", dtype=TYPES[dtype])
    x[0, 5], x[1, 70] = top, -top
    up = codes(eng, dtype, f, k, {(3, 5): 2.0 ** -20, (4, 70): -2.0 ** -20, (9, 5): 0.5})
    down = codes(eng, dtype, n, f, {(7, 3): 2.0 ** -10, (8, 4): 2.0 ** -10, (9, 9): 2.0 ** -20})
    y = torch.empty(2, n, device="cuda", dtype=x.dtype)
    eng.moe_forward_fp4(y, x, torch.zeros(2, 1, device="cuda", dtype=torch.int32), torch.ones(2, 1, device="cuda"), None, None, *up, *down,
                        2, 1, k, f, n, 1, "relu", dtype)
    want = torch.zeros(2, n, device="cuda", dtype=torch.float64)
    v = x[0, 5].double()
    want[0, 7], want[1, 8], want[0, 9] = v * 2.0 ** -30, v * 2.0 ** -30, v * 2.0 ** -21
    tol = (HALF[dtype] + 20 * 2.0 ** -23) * want
    # row 0's h at 3 is v 2^-20 in one block with v 2^-1 at 9: it keeps 2^-23 of that, and enters with 2^-10
    tol[0, 7] += v * 2.0 ** (-1 - 23 - 10)
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_h_at_the_end_of_f32s_range(eng, dtype):
    """The same of h: a gate of 1.96875 * 2^63 times an up of it."""
    k, f, n = 64, 64, 40
    x = torch.zeros(1, k, device="cuda", dtype=TYPES[dtype])
    x[0, 5] = 1.96875 * 2.0 ** 63
    gate, up = codes(eng, dtype, f, k, {(3, 5): 1.0}), codes(eng, dtype, f, k, {(3, 5): 1.0})
    down = codes(eng, dtype, n, f, {(7, 3): 2.0 ** -10})
    y = torch.empty(1, n, device="cuda", dtype=x.dtype)
    eng.moe_forward_fp4(y, x, torch.zeros(1, 1, device="cuda", dtype=torch.int32), torch.ones(1, 1, device="cuda"), *gate, *up, *down,
                        1, 1, k, f, n, 1, "relu", dtype)
    want = torch.zeros(1, n, device="cuda", dtype=torch.float64)
    want[0, 7] = (1.96875 * 2.0 ** 63) ** 2 * 2.0 ** -10
    assert ((y.double() - want).abs() <= (HALF[dtype] + 20 * 2.0 ** -23) * want).all()
