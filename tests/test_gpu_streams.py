"""Calls on several streams of one engine: they do not wait for one another, end, and give the results they give alone."""
import random
import time

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


def adapter_calls(eng, seed, m, k, n, r, g, dtype=torch.bfloat16):
    """A forward and a backward, and their results' buffers."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def t(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=gen) * std).to(dtype)
    x, w, a, b, dy = t(m, k), t(k, n, std=k ** -0.5), t(g, r, k, std=k ** -0.5), t(g, r, n, std=0.3), t(m, n)
    ids = (torch.arange(m, device="cuda") * g // m).int()
    y, h, dx = torch.empty_like(dy), torch.zeros(m, r, device="cuda"), torch.empty_like(x)
    da, db = torch.empty(g, r, k, device="cuda"), torch.empty(g, r, n, device="cuda")
    sizes = (m, k, n, r, g, dtype)
    return (lambda: eng.adapter_forward(y, h, x, w, None, a, b, None, ids, *sizes),
            lambda: eng.adapter_backward(dx, da, db, x, h, w, dy, a, b, None, ids, *sizes)), (y, h, dx, da, db)


def test_scratch_makes_no_stream_wait_for_another(eng):
    """One stream's call takes scratch beside another stream's that pauses between two calls: it is done long before."""
    a, b = ([torch.randn(300001, device="cuda") for _ in range(5)] for _ in range(2))
    n, m, want = (torch.empty(1, device="cuda") for _ in range(3))
    eng.grad_norm(want, b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        eng.grad_norm(n, a)
        torch.cuda._sleep(1_000_000_000)  # about half a second
        eng.grad_norm(n, a)
        end = torch.cuda.Event()
        end.record()
    with torch.cuda.stream(t):
        eng.grad_norm(m, b)
        done = torch.cuda.Event()
        done.record()
    began = time.time()
    while not done.query() and time.time() - began < 20:
        time.sleep(0.001)
    assert not end.query(), "the call waited for the other stream"
    torch.cuda.synchronize()
    assert torch.equal(m, want)


def test_adapter_calls_take_turns(eng):
    """Adapter calls of one engine run one behind the other, whatever their streams: the second starts when the first has ended."""
    (one, _), _ = adapter_calls(eng, 1, 4096, 1024, 512, 64, 4)
    (other, _), (y, *_) = adapter_calls(eng, 2, 64, 1024, 512, 16, 4)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for stream, call in ((s, one), (t, other)):
        with torch.cuda.stream(stream):
            call()
    torch.cuda.synchronize()
    want = y.clone()
    y.zero_()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
        one()
        end = torch.cuda.Event()
        end.record()
    with torch.cuda.stream(t):
        other()
        done = torch.cuda.Event()
        done.record()
    while not done.query():
        time.sleep(0.001)
    assert end.query()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_two_streams_side_by_side(eng):
    """Forward, backward, routing and clipping in random order on two streams: all ends, with the bits that each gives alone."""
    calls, outs = [], []
    for q in (0, 1):
        own = []
        for i, (m, k, n, r, g) in enumerate(((8192, 4096, 4096, 32, 3), (1333, 768, 2048, 20, 17), (64, 1024, 1024, 16, 8))):
            fb, res = adapter_calls(eng, 10 * q + i, m, k, n, r, g, torch.float16 if i == 1 else torch.bfloat16)
            own += list(fb)
            outs.append(res)
        logits = torch.randn(20000, 64, device="cuda")
        route = [torch.empty(20000, 6, dtype=torch.int32, device="cuda"), torch.empty(20000, 6, device="cuda"),
                 torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"),
                 torch.empty(64, device="cuda"), torch.empty(1, device="cuda"), torch.empty(20000, device="cuda")]
        own.append(lambda logits=logits, route=route: eng.router_forward(*route, logits, None, 20000, 64, 6, 1, "f32"))
        outs.append(route)
        src = [torch.randn(100003, device="cuda") for _ in range(9)]
        dst, norm = [torch.empty_like(v) for v in src], torch.empty(1, device="cuda")
        pair = bi.TensorSet(dst), bi.TensorSet(src)
        own.append(lambda pair=pair, norm=norm: eng.clip_gradients(*pair, norm, 1.0))
        outs.append([*dst, norm])
        calls.append(own)
    for own in calls:
        for f in own:
            f()
    torch.cuda.synchronize()
    want = [[v.clone() for v in res] for res in outs]
    streams, rng = [torch.cuda.Stream(), torch.cuda.Stream()], random.Random(1)
    for _ in range(100):
        for _ in range(5):
            order = [rng.sample(range(len(own)), len(own)) for own in calls]
            for i in range(len(calls[0])):
                for q in (0, 1):
                    with torch.cuda.stream(streams[q]):
                        calls[q][order[q][i]]()
        torch.cuda.synchronize()
    eng.check()
    for res, w in zip(outs, want):
        assert all(torch.equal(p, v) for p, v in zip(res, w))
