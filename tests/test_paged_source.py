"""What the sources of libfa_paged.so have to keep to, read as text."""

import glob
import os
import re

import pytest

from exact_io_aware_69_b200 import build


def kernels():
    """(file, name, parameters) of every kernel."""
    out = []
    for path in sorted(glob.glob(os.path.join(build.CSRC_PAGED, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^{;]*?\)\s*)?(\w+)\s*\(",
                             text):
            depth, at = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            out.append((os.path.basename(path), m.group(1), text[m.end():at - 1]))
    return out


KERNELS = kernels()


def test_the_kernels_are_found():
    assert {name for _, name, _ in KERNELS} == {
        "fa_rope_kernel", "fa_paged_step_kernel", "fa_paged_chunk_kernel", "fa_paged_merge_kernel"}


@pytest.mark.parametrize("file,name,params", KERNELS, ids=[k[1] for k in KERNELS])
def test_no_kernel_declares_its_inputs_constant(file, name, params):
    """Every launch overlaps the end of the kernel before it, which may still write what this
    one reads: a pointer to const with __restrict__ says that nobody writes there while
    the kernel lives, and allows loads through a cache that does not see those writes."""
    declared = [p.strip() for p in params.split(",")
                if "const" in p.split("*")[0].split() and "__restrict__" in p and "*" in p]
    assert not declared, declared
