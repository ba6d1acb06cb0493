"""Rules that the CUDA sources keep and no run can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_diffusion_model_b200", "csrc")


def kernels():
    """(file, name, parameters, body) of every __global__ function."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            at = text.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield name, m.group(1), text[m.end():at], text[at:end]


def test_kernels_that_start_early_read_through_plain_pointers():
    """A kernel that waits for the grid before it starts while that grid still writes what it reads: a `const __restrict__`
    pointer would let the compiler take the read-only path, or move a load ahead of the wait. (Kernels that bring their
    inputs by bulk copies load nothing through such pointers.)"""
    found, seen = [], 0
    for file, name, params, body in kernels():
        if "grid_dependency_wait()" not in body or "bulk_load(" in body:
            continue
        seen += 1
        if re.search(r"\bconst\b[^,]*__restrict__", params):
            found.append(f"{file}: {name}")
    assert seen >= 12 and not found, found
