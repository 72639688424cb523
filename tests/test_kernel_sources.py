"""What the kernels' sources and the built library show without a GPU."""
import glob
import os
import re
import subprocess

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


def _norm_forms(V, routed):
    """(V, vectors per thread, threads at most, CTAs asked for, routed) of every forward block norm that a call reaches."""
    forms = set()
    for nv in range(1, 16384 // V + 1):
        for T in (1, 295, 296, 1 << 20):
            if nv <= 1024 and (T < 296 or nv <= 64):
                forms.add((V, 1, 1024, 1, routed))
            elif nv <= 1024:
                forms.add((V, 2, 512, 3 if nv > 768 and not routed else 2, routed))
            elif nv <= 4096:
                forms.add((V, 4, 512 if V == 8 else 1024, 1, routed))
            else:
                forms.add((V, 8 if nv <= 8192 else 16, 1024, 1, routed))
    return forms


def test_no_block_norm_is_built_that_no_call_reaches():
    from bit_mixed_precision_router_b200 import build
    names = subprocess.run(["nm", "-C", build.build()], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"k_block_norm<(\w+), (\d+), (\d+), (\d+), (\d+), (\w+)>\(", names))
    built = {(t, int(v), int(w), int(n), int(c), r == "true") for t, v, w, n, c, r in built}
    reached = {(t,) + f for t, V in (("__nv_bfloat16", 8), ("__half", 8), ("float", 4)) for v in (V, 1) for r in (False, True)
               for f in _norm_forms(v, r)}
    assert built == reached, (sorted(built - reached), sorted(reached - built))
