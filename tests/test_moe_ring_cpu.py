"""The expert layer's shared-memory ring on a machine without a GPU: its sizes for every
call that the entry points take (moe_ring.h compiled for the host), and its barriers
replayed in random orders of the warps that work on it."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "deterministic_invariant_gemm_fixed_gb300", "csrc")

SHIM = r"""
#include "moe_ring.h"
using namespace bi;
extern "C" int scale_warps(int depth) { return moe_scale_warps(depth); }
extern "C" int ring(int fp4, int out, int T, int C, int E, int64_t* o) {
    const MoeRing r = moe_ring(fp4 != 0, out != 0, T, int64_t(T) * C, E);
    o[0] = r.cap; o[1] = r.passes; o[2] = r.stage; o[3] = r.depth; o[4] = r.fixed;
    return 0;
}
// seen[depth] += 1 for every call's ring; returns calls whose ring does not fit its memory,
// or 1 << 40 and more where a list has more entries than its room
extern "C" int64_t sweep(int fp4, int out, int64_t* seen) {
    int64_t bad = 0;
    for (int T = 1; T <= MOE_MAX_PAIRS; ++T)
        for (int C = 1; int64_t(T) * C <= MOE_MAX_PAIRS; ++C)
            for (int E = 1; E <= MOE_MAX_E; ++E) {
                const int64_t P = int64_t(T) * C, active = E < P ? E : P;
                const MoeRing r = moe_ring(fp4 != 0, out != 0, T, P, E);
                if (r.depth < 1 || r.depth > MAX_STAGES || r.fixed + int64_t(r.depth) * r.stage > T_LIMIT) ++bad;
                // the most passes: every expert has one choice, and what is left makes whole passes more
                const int64_t all = fp4 || out ? active + (P - active) / r.cap : active * ((T + r.cap - 1) / r.cap);
                if ((fp4 || out ? P : T) > r.cap && all > r.passes) bad += int64_t(1) << 40;
                if (r.depth >= 0 && r.depth <= MAX_STAGES) ++seen[r.depth];
            }
    return bad;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SHIM)
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "ring.cpp"), "-o", str(d / "ring.so")], check=True)
    lib = ctypes.CDLL(str(d / "ring.so"))
    lib.sweep.restype = ctypes.c_int64
    return lib


def replay(rng, depth, turn, uses):
    """The ring's barriers in a random order of steps: the producer (arrives on full), `turn`
    warps that each fill every turn-th use (arrive on full too; full counts two), the MMA warp.  A wait by
    parity passes when the barrier's current phase has the other one.  Returns whether every
    use was consumed with what was filled for it."""
    class Bar:
        def __init__(self, count):
            self.count, self.left, self.phase = count, count, 0

        def arrive(self):
            self.left -= 1
            if self.left == 0:
                self.left, self.phase = self.count, self.phase + 1

        def done(self, parity):  # the phase of this parity has completed
            return self.phase % 2 != parity

    full, empty = [Bar(2) for _ in range(depth)], [Bar(1) for _ in range(depth)]
    weights, scales = [None] * depth, [None] * depth
    at = {"producer": 0, "mma": 0, **{i: i for i in range(turn)}}
    while at["mma"] < uses:
        ready = []
        for who, n in at.items():
            s, parity = n % depth, n // depth % 2
            if n < uses and (full[s].done(parity) if who == "mma" else empty[s].done(parity ^ 1)):
                ready.append(who)
        if not ready:
            return False  # a wait that never ends
        who = rng.choice(ready)
        n = at[who]
        s = n % depth
        if who == "mma":
            if weights[s] != n or scales[s] != n:
                return False
            empty[s].arrive()
        elif who == "producer":
            weights[s] = n
            full[s].arrive()
        else:
            scales[s] = n
            full[s].arrive()
        at[who] = n + (turn if isinstance(who, int) else 1)
    return True


def test_every_ring_fits_and_no_more_warps_than_stages(host):
    for fp4 in (0, 1):
        for out in (0, 1):
            seen = (ctypes.c_int64 * 13)()
            assert host.sweep(fp4, out, seen) == 0
            depths = [d for d in range(13) if seen[d]]
            assert min(depths) >= 2
            if fp4:
                for d in depths:
                    assert 1 <= host.scale_warps(d) <= d


def test_pass_lists_take_the_room_they_need(host):
    """Room for every expert's choices in passes of `cap`, however they fall, and hardly more: a place per
    choice cost calls of a few dozen experts a stage of the ring."""
    o = (ctypes.c_int64 * 5)()
    rng = random.Random(5)
    for fp4, out in ((1, 0), (1, 1), (0, 1)):
        for _ in range(400):
            c = rng.randint(1, 16)
            t, e = rng.randint(1, 2048 // c), rng.randint(1, 1024)
            host.ring(fp4, out, t, c, e, o)
            cap, room, choices = o[0], o[1], t * c
            worst = min(e, choices) + (choices - min(e, choices)) // cap
            assert worst <= room <= worst + 1 + min(e, choices) // cap
            counts = [0] * e  # and some choice of them
            some = rng.randint(1, e)
            for _ in range(choices):
                counts[rng.randrange(some)] += 1
            assert sum(-(-n // cap) for n in counts) <= room
    for out in (0, 1):
        host.ring(1, out, 256, 8, 64, o)
        assert o[3] == 4


@pytest.mark.parametrize("depth", range(1, 13))
def test_scale_warps_keep_to_the_phases(host, depth):
    rng = random.Random(depth)
    for _ in range(60):
        assert replay(rng, depth, host.scale_warps(depth), rng.choice([1, 6, 7, 8, 40]))


def test_the_replay_finds_more_warps_than_stages():
    """Four warps on three stages go wrong from the seventh use on; on four they do not."""
    rng = random.Random(0)
    assert not all(replay(rng, 3, 4, 40) for _ in range(50))
    assert all(replay(rng, 3, 4, 6) for _ in range(50))
    assert all(replay(rng, 4, 4, 40) for _ in range(50))


def test_layers_of_many_experts_have_the_short_ring(host):
    """Calls that the GPU tests take for the ring of three stages do have it."""
    o = (ctypes.c_int64 * 5)()
    for t, c, e in ((32, 2, 1024), (64, 8, 512), (512, 4, 1024)):
        for out in (0, 1):
            host.ring(1, out, t, c, e, o)
            assert o[3] == 3
