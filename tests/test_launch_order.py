"""Kernels that let the next one start hold their tensor memory first.  A kernel may be given
SMs as soon as every CTA of the one before has let it start.  If it then took the tensor
memory of an SM where such a CTA has yet to allocate its own, that CTA would wait for it, and
it for that CTA's grid: neither wait has a bound.  Read from the sources, no GPU."""
import glob
import os
import re

import pytest

import sparse_rank_linear_b200

CSRC = os.path.join(os.path.dirname(sparse_rank_linear_b200.__file__), "csrc")


def kernels():
    """(name, body) of every kernel, comments removed."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for piece in text.split("__global__")[1:]:
            start = piece.index("{")
            depth, end = 0, start
            for end in range(start, len(piece)):
                depth += {"{": 1, "}": -1}.get(piece[end], 0)
                if depth == 0:
                    break
            yield re.findall(r"\w+_kernel", piece[:start])[0], piece[start:end]


FOUND = {name: body for name, body in kernels()
         if "tmem_alloc" in body and "griddep_launch_dependents()" in body}


def test_the_kernels_are_found():
    assert {"grad_skinny_kernel", "grad_dx_kernel", "salr_t_kernel", "salr_stream_kernel"} <= set(FOUND)


@pytest.mark.parametrize("name", sorted(FOUND))
def test_tensor_memory_is_held_before_the_next_kernel_may_start(name):
    body = FOUND[name]
    held = body.index("__syncthreads()", body.rindex("tmem_alloc"))
    assert body.index("griddep_launch_dependents()") > held
