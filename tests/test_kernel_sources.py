"""What the kernels' sources and the built library show without a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_mixed_precision_router_b200", "csrc")


def _kernels():
    """(file, name, parameters, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^()]*)\)\s*\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), m.group(1), m.group(2), text[m.end():end]


def test_every_kernel_is_found():
    names = [name for _, name, _, _ in _kernels()]
    count = sum(len(re.findall(r"__global__", re.sub(r"//[^\n]*", "", open(p).read()))) for p in glob.glob(os.path.join(CSRC, "*.cu*")))
    assert len(names) == count and {"k_norm_weight_sum", "k_spread", "k_linear_umma", "k_ffn_gemv"} <= set(names)


def test_kernels_launched_ahead_promise_nothing_of_what_they_wait_for():
    """A kernel that starts before an earlier one has ended (griddepcontrol.wait) reads data that is written while it
    runs: `const __restrict__` would promise the compiler that nobody does, and allow the read-only path or a load ahead of
    the wait."""
    waiting = [(f, n, p, b) for f, n, p, b in _kernels() if "griddepcontrol.wait" in b]
    assert waiting
    for f, name, params, body in waiting:
        for p in params.split(","):
            assert not ("const" in p and "__restrict__" in p), (f, name, p.strip())
        assert "__ldg" not in body and "ld.global.nc" not in body, (f, name)
