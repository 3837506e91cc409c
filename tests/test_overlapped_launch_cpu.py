"""Kernels that are launched while the kernel before them still runs: what that
kernel writes is read by coherent loads behind the wait.  The read-only path
(`__ldg`, or a `const __restrict__` pointer, which lets the compiler choose it)
is for data that nothing writes during the reading kernel's whole life, and such
loads may be moved ahead of the wait.  Checked in the sources: no run shows it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_x128_b200", "csrc")
FILES = ("norm.cu", "moe_grad.cu", "moe_masked.cu")

# kernel: parameters that the kernel before it writes
PRODUCED = {"norm_param_grad_kernel": ["part"], "moe_permute_kernel": ["pos", "m_indices"],
            "moe_dispatch_masked_kernel": ["pos"]}


def kernels():
    """name -> (parameter list, body) of every __global__ function, comments taken out."""
    found = {}
    for fn in FILES:
        with open(os.path.join(CSRC, fn)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            params, j = text[m.end():i - 1], text.index("{", i)
            depth, k = 1, j + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[k], 0)
                k += 1
            found[m.group(1)] = (params, text[j:k])
    return found


def test_every_kernel_that_waits_is_listed():
    waiting = {n for n, (_, body) in kernels().items() if "grid_dependency_wait" in body}
    assert waiting == set(PRODUCED)


@pytest.mark.parametrize("kernel,name", [(k, n) for k, names in PRODUCED.items() for n in names])
def test_produced_arrays_are_read_coherently(kernel, name):
    params, body = kernels()[kernel]
    mine = [p for p in params.split(",") if re.search(rf"\b{name}\s*$", p)]
    assert len(mine) == 1 and "__restrict__" not in mine[0], mine
    assert not re.search(rf"__ldg\(\s*&?\s*\(?\s*{name}\b", body)
    # nor handed as a whole to a function that might read it so
    assert not re.search(rf"\w\((?:[^()]*,)?\s*{name}\s*[,)]", body)
