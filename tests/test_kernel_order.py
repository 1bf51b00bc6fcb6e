"""What the kernels' source has to keep to whatever they compute: checked on the text."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "deterministic_invariant_gemm_fixed_gb300", "csrc")


def kernels(path):
    """(name, body) of each __global__ function of a file, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__", text):
        name = re.search(r"(\w+)\s*\(const|(\w+)\s*\(\s*\w", text[m.end():].split("__launch_bounds__")[-1])
        start = text.index("{", m.end())
        depth, i = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            if depth == 0:
                break
            i += 1
        yield name.group(0) if name else "?", text[start:i]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_dependents_start_after_the_wait(path):
    """A kernel lets the next one of its stream start only once it has waited for the one before itself."""
    for name, body in kernels(path):
        launch = body.find("grid_dep_launch()")
        if launch >= 0:
            wait = body.find("grid_dep_wait()")
            assert 0 <= wait < launch, name


def test_waits_are_bounded():
    """Every loop on a barrier's try_wait stands in one of the helpers that watch the clock."""
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for line in text.split("\n"):
            assert not ("mbar_try_wait(" in line and re.search(r"\b(for|while)\b", line)), (os.path.basename(path), line)
