"""The few-token expert layer, against 64 bits.

Tolerance, element by element.  An inner product of length L: at most L/32 + 64
roundings or truncations of at most 2^-23 of a partial sum, eps(L) = (L/32 + 64) 2^-23
times the sum of its terms' magnitudes.  Those of the gate and of up go through the
activation (slope at most 1.13, its own value to 16 roundings) and the product; h
may enter the second product as two 16-bit parts (2^-16 of it).  y adds the second
product's own eps(F), C + 2 roundings for the weighted sum, and half a step of its type.
"""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_fixed_gb300 as bi
import fp4_ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
U = 2.0 ** -23


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


ACT = {"silu": lambda v: v / (1 + np.exp(-v)),
       "gelu": lambda v: 0.5 * v * (1 + np.tanh(0.79788456 * (v + 0.044715 * v ** 3))),
       "relu": lambda v: np.maximum(v, 0)}


def reference(x, ids, p, gate, up, down, act):
    """y and its tolerance before the last rounding, in 64 bits."""
    t, k = x.shape
    f, n = up.shape[1], down.shape[1]
    y, tol = np.zeros((t, n)), np.zeros((t, n))
    def eps(length):
        return (length / 32 + 64) * U
    for j in range(up.shape[0]):
        for row, c in zip(*np.nonzero(ids == j)):
            u, su = up[j] @ x[row], np.abs(up[j]) @ np.abs(x[row])
            if gate is None:
                a, da = ACT[act](u), 1.13 * eps(k) * su
                h, dh = a, da + 16 * U * np.abs(a)
            else:
                g, sg = gate[j] @ x[row], np.abs(gate[j]) @ np.abs(x[row])
                a = ACT[act](g)
                da = 1.13 * eps(k) * sg + 16 * U * np.abs(a)
                h, dh = a * u, da * (np.abs(u) + eps(k) * su) + np.abs(a) * eps(k) * su
            dh = dh + (2.0 ** -16 + 4 * U) * np.abs(h)
            o, so = down[j] @ h, np.abs(down[j]) @ (np.abs(h) + dh)
            y[row] += p[row, c] * o
            tol[row] += abs(p[row, c]) * (np.abs(down[j]) @ dh + (eps(f) + (ids.shape[1] + 2) * U) * so)
    return y, tol


def check(y, ref, dtype):
    want, tol = ref
    tol = tol + HALF[dtype] * (np.abs(want) + tol) + TINY[dtype]
    err = np.abs(f64(y) - want)
    assert (err <= tol).all(), (err / tol).max()


class Layer:
    def __init__(self, eng, dtype, e, k, f, n, fp4=False, gated=True, seed=0, scale=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = TYPES[dtype]
        self.eng, self.dtype, self.sizes, self.fp4, self.gen = eng, dtype, (k, f, n, e), fp4, gen

        def w(*s):
            return (torch.randn(*s, device="cuda", generator=gen) * s[2] ** -0.5 * scale).to(dt)
        gate, up, down = w(e, f, k) if gated else None, w(e, f, k), w(e, n, f)
        self.w64 = [None if v is None else f64(v) for v in (gate, up, down)]
        self.w = [gate, up, down]
        if fp4:
            self.w64 = [None if v is None else fp4_ref.rounded(v.reshape(-1, v.shape[2])).reshape(v.shape) for v in self.w64]
            pairs = []
            for v in self.w:
                if v is None:
                    pairs += [None, None]
                    continue
                r, c = v.shape[0] * v.shape[1], v.shape[2]
                q = bi.fp4_buffers(r, c)
                eng.fp4_quantize(*q, None, None, v, r, c, dtype)
                pairs += q
            self.w = pairs

    def tokens(self, t, c, pad=0.0):
        k, _, _, e = self.sizes
        x = torch.randn(t, k, device="cuda", generator=self.gen).to(TYPES[self.dtype])
        ids = torch.rand(t, e, device="cuda", generator=self.gen).argsort(1)[:, :c].to(torch.int32).contiguous()
        if pad:
            ids[torch.rand(t, c, device="cuda", generator=self.gen) < pad] = e
        return x, ids, torch.rand(t, c, device="cuda", generator=self.gen)

    def run(self, x, ids, p, act="silu", y=None):
        k, f, n, e = self.sizes
        t, c = ids.shape
        if y is None:
            y = torch.full((t, n), 9.0, device="cuda").to(TYPES[self.dtype])
        call = self.eng.moe_forward_fp4 if self.fp4 else self.eng.moe_forward
        call(y, x, ids, p, *self.w, t, c, k, f, n, e, act, self.dtype)
        return y

    def ref(self, x, ids, p, act="silu"):
        return reference(f64(x), ids.cpu().numpy(), f64(p), *self.w64, act)


# t, c, e, k, f, n
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 2, 4, 64, 40, 72), (2, 1, 3, 17, 33, 5), (5, 3, 8, 300, 130, 257), (9, 2, 5, 512, 520, 128),
          (40, 4, 6, 520, 264, 96), (64, 6, 64, 128, 64, 80), (130, 2, 3, 96, 100, 48), (3, 2, 1024, 40, 24, 32), (7, 2, 8, 1000, 1000, 1000)]


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,c,e,k,f,n", SHAPES)
def test_layer(eng, t, c, e, k, f, n, dtype, fp4):
    layer = Layer(eng, dtype, e, k, f, n, fp4, seed=t + k)
    data = layer.tokens(t, c, pad=0.1 if t > 2 else 0.0)
    y = layer.run(*data)
    check(y, layer.ref(*data), dtype)
    assert torch.equal(y, layer.run(*data))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations(eng, act, gated, dtype):
    for fp4 in (False, True):
        layer = Layer(eng, dtype, 4, 136, 72, 64, fp4, gated=gated, scale=3.0)
        data = layer.tokens(6, 2)
        check(layer.run(*data, act=act), layer.ref(*data, act=act), dtype)


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_do_not_depend_on_the_batch(eng, dtype, fp4):
    for k, f, n in ((1304, 1048, 72), (40, 36, 24), (75, 33, 21)):
        layer = Layer(eng, dtype, 3, k, f, n, fp4)
        x, ids, p = layer.tokens(100, 2)
        whole = layer.run(x, ids, p)
        for rows in (slice(0, 1), slice(17, 19), slice(40, 73)):
            part = [v[rows].contiguous() for v in (x, ids, p)]
            assert torch.equal(layer.run(*part), whole[rows])
        perm = torch.randperm(100, device="cuda")
        assert torch.equal(layer.run(x[perm].contiguous(), ids[perm].contiguous(), p[perm].contiguous()), whole[perm])


@pytest.mark.parametrize("dtype", TYPES)
def test_padding_repeats_and_one_expert_for_all(eng, dtype):
    layer = Layer(eng, dtype, 5, 96, 64, 40)
    x, ids, p = layer.tokens(50, 3)
    ids[7], ids[9, 1], ids[10] = 5, -1, 2 ** 31 - 1  # no choice at all; ids outside either way
    ids[11] = 3                                      # the same expert three times
    ids[20:] = 1                                     # most tokens at one expert
    p[7], p[9, 1] = float("nan"), float("inf")       # weights of choices that are none
    y = layer.run(x, ids, p)
    ref_ids = ids.clone()
    ref_ids[9, 1] = 5
    check(y, layer.ref(x, ref_ids, torch.nan_to_num(p, nan=0, posinf=0)), dtype)
    assert not y[7].any() and not y[10].any()


def test_values_stay_with_their_tokens(eng):
    """An infinity or NaN of one token reaches its own row only; experts that nobody chose may hold anything."""
    for dtype in TYPES:
        layer = Layer(eng, dtype, 4, 64, 48, 32)
        x, ids, p = layer.tokens(12, 2)
        ids[ids == 3] = 4
        clean = layer.run(x, ids, p)
        for w in layer.w:
            w[3] = float("nan")
        x[5, 3], x[6, 1] = float("nan"), float("inf")
        y = layer.run(x, ids, p)
        keep = torch.ones(12, dtype=torch.bool, device="cuda")
        keep[5] = keep[6] = False
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[5]).all() or (ids[5] == 4).all()


def test_large_hidden_values_in_f16(eng):
    """h beyond 65504 is no infinity: f16 is the type of the operands, not of h."""
    layer = Layer(eng, "f16", 2, 64, 64, 64, scale=1.0)
    layer.w[2].mul_(2.0 ** -10)
    layer.w64[2] = f64(layer.w[2])
    x, ids, p = layer.tokens(4, 2)
    x = (x * 400).half()
    y = layer.run(x, ids, p)
    ref = layer.ref(x, ids, p)
    assert np.isfinite(ref[0]).all() and np.abs(ref[0]).max() < 65504
    check(y, ref, "f16")


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_off_alignment(eng, dtype):
    """Operands and outputs that start one element off 16 bytes."""
    layer = Layer(eng, dtype, 3, 64, 40, 48)
    x, ids, p = layer.tokens(10, 2)
    want = layer.ref(x, ids, p)
    def off(t):
        b = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:].view(t.shape)
        return b.copy_(t)
    layer.w = [off(w) for w in layer.w]
    buf = torch.full((10 * 48 + 128,), 5.0, device="cuda").to(TYPES[dtype])
    layer.run(off(x), ids, p, y=buf[63:63 + 480].view(10, 48))
    check(buf[63:63 + 480].view(10, 48), want, dtype)
    assert (buf[:63] == 5).all() and (buf[63 + 480:] == 5).all()


def test_largest_batch(eng):
    layer = Layer(eng, "bf16", 4, 64, 32, 24)
    data = layer.tokens(1024, 2)
    check(layer.run(*data), layer.ref(*data), "bf16")
    with pytest.raises(bi.BiError) as err:
        layer.run(*layer.tokens(1025, 2))
    assert err.value.status == bi.BI_ERR_UNSUPPORTED


def test_no_tokens(eng):
    layer = Layer(eng, "bf16", 4, 64, 32, 24)
    layer.run(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, 2, device="cuda", dtype=torch.int32),
              torch.empty(0, 2, device="cuda"))


def test_captured_and_replayed(eng):
    layer = Layer(eng, "bf16", 8, 128, 96, 64)
    x, ids, p = layer.tokens(6, 2)
    y = torch.empty(6, 64, device="cuda", dtype=torch.bfloat16)
    layer.run(x, ids, p, y=y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run(x, ids, p, y=y)
    for v, w in zip((x, ids, p), layer.tokens(6, 2)):
        v.copy_(w)
    g.replay()
    got = y.clone()
    assert torch.equal(got, layer.run(x, ids, p))


def test_two_streams(eng):
    layer = Layer(eng, "f16", 8, 256, 128, 64)
    data = [layer.tokens(5, 2) for _ in range(2)]
    want = [layer.run(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = []
        for s, d in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(layer.run(*d))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_most_choices_and_experts(eng, dtype, fp4):
    """2048 choices over 1024 experts: the largest lists."""
    layer = Layer(eng, dtype, 1024, 40, 24, 16, fp4)
    data = layer.tokens(512, 4)
    check(layer.run(*data), layer.ref(*data), dtype)


def test_nan_scale_of_a_weight_block(eng):
    """A weight block without a scale makes the rows NaN that chose its expert, and no other."""
    layer = Layer(eng, "bf16", 4, 96, 64, 48, fp4=True)
    x, ids, p = layer.tokens(20, 1)
    clean = layer.run(x, ids, p)
    scales = layer.w[5]  # of down: rows e * 48 + n, blocks along 64; row 2 * 48 is expert 2's first
    r = 2 * 48
    scales[(r // 128) * 2 * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + 1] = 255
    y = layer.run(x, ids, p)
    hit = (ids[:, 0] == 2)
    assert torch.isnan(y[hit, 0]).all() and torch.equal(y[~hit], clean[~hit]) and torch.equal(y[:, 1:], clean[:, 1:])


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dtype", TYPES)
def test_x_and_y_off_alignment_keep_the_bits(eng, dtype, fp4):
    """x and y one element off 16 bytes beside weights that are on it."""
    layer = Layer(eng, dtype, 5, 136, 72, 56, fp4)
    x, ids, p = layer.tokens(21, 2)
    want = layer.run(x, ids, p)
    off = torch.empty(x.numel() + 1, device="cuda", dtype=x.dtype)[1:].view(x.shape).copy_(x)
    buf = torch.full((21 * 56 + 2,), 5.0, device="cuda").to(x.dtype)
    layer.run(off, ids, p, y=buf[1:-1].view(21, 56))
    assert torch.equal(buf[1:-1].view(21, 56), want) and buf[0] == 5 and buf[-1] == 5


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
@pytest.mark.parametrize("dtype", TYPES)
def test_no_choice_at_all(eng, dtype, fp4):
    layer = Layer(eng, dtype, 3, 64, 48, 40, fp4)
    for t in (2, 40):
        x, ids, p = layer.tokens(t, 2)
        ids.fill_(3)
        y = layer.run(x, ids, p)
        assert not y.any() and not torch.signbit(y).any()
    eng.check()


@pytest.mark.parametrize("fp4", [False, True], ids=["plain", "fp4"])
def test_popular_expert_and_long_batch(eng, fp4):
    """Experts with several passes beside ones with a single token, and more tokens than one pass of the batch."""
    layer = Layer(eng, "bf16", 6, 320, 80, 136, fp4)
    x, ids, p = layer.tokens(600, 1)
    ids[:] = 2
    ids[::50] = 4
    ids[7], ids[599] = 0, 5
    y = layer.run(x, ids, p)
    rows = torch.tensor([0, 1, 7, 50, 255, 256, 300, 511, 512, 599], device="cuda")
    check(y[rows], layer.ref(x[rows], ids[rows], p[rows]), "bf16")
    for r in (7, 300, 599):
        assert torch.equal(layer.run(x[r:r + 1].contiguous(), ids[r:r + 1].contiguous(), p[r:r + 1].contiguous()), y[r:r + 1])
