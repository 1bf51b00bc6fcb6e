"""What the expert layer keeps of a hidden value, and of values at the end of f32's range."""
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi

pytestmark = pytest.mark.gpu


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
