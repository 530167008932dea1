"""Orders in the kernels' sources that no run shows (no GPU needed)."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "splat_rendering_gb300", "csrc")


def _kernels():
    """(name, body without comments) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for part in re.split(r"\b__global__\b", text)[1:]:
            name = re.search(r"\b(k_\w+)\s*\(", part)
            yield name.group(1), part[:part.index("\n}\n")]


ALLOCATING = [(name, body) for name, body in _kernels() if "tmem_alloc" in body]


def test_the_kernels_are_found():
    assert {"k_linear_product", "k_linear_stream", "k_linear_narrow"} <= {n for n, _ in ALLOCATING}


@pytest.mark.parametrize("name,body", ALLOCATING, ids=[n for n, _ in ALLOCATING])
def test_tensor_memory_before_the_next_launch(name, body):
    """A block lets the next launch's blocks in only when it has its tensor memory: one that came to
    lie beside it could take the columns, and wait, holding them, for this block's end."""
    if "pdl_next" not in body:
        return
    allocated = body.index("tmem_alloc")
    barrier = body.index("__syncthreads", allocated)
    assert body.index("pdl_next") > barrier
