"""Kernels launched as programmatic dependents are resident while the kernel ahead still writes what
they read after the dependency wait: none of their inputs is read-only for their life, so none may
be loaded on the read-only path (__ldg, ld.global.nc, const __restrict__ parameters)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_27_b200", "csrc")
FILES = ["kv4.cu", "merge.cu", "paged.cuh", "paged_attn.cu", "rope.cu"]


def code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    for pattern in (r"\b__ldg\w*\s*\(", r"\bld\.global(\.\w+)*\.nc\b", r"\b__restrict__\b", r"\b__restrict\b"):
        assert not re.search(pattern, code(name)), (name, pattern)
