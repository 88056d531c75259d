"""Rules of the kernel sources that no run can show to be broken."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_13_gb300", "csrc")


def code(name):
    """A source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def files_launched_early():
    """Sources of kernels that may start while the kernel before them still writes."""
    return [f for f in sorted(os.listdir(CSRC)) if "pdl_wait()" in code(f) and f != "ptx.cuh"]


def test_there_are_such_files():
    assert {"cache.cu", "tree_api.cu", "tree_kernel.cuh"} <= set(files_launched_early())


@pytest.mark.parametrize("name", files_launched_early())
def test_no_read_only_loads_of_what_an_earlier_kernel_may_write(name):
    """The read-only path is defined only for data that does not change while the kernel
    lives, and such a kernel lives before its predecessor has written its results."""
    text = code(name)
    for form in ("__ldg", "ld.global.nc", "__restrict__", "tex1D"):
        assert form not in text, form


def test_every_exit_of_the_tree_kernel_leaves_the_merge_kernel_its_answer():
    """The merge kernel follows whatever p.cut says.  No exit may leave what the workspace
    held before: the one before the work starts (shared memory not where it has to be,
    which no launch here shows) writes "no unit", after the kernel before has let go of
    the workspace."""
    text = code("tree_kernel.cuh")
    body = text[text.index("attn_tree_kernel(const"):text.index("attn_tree_merge_kernel(const")]
    exits = [m.start() for m in re.finditer(r"(?m)^ +return;", body)]  # (others leave a lambda)
    assert len(exits) == 1
    early = body[body.index("& 1023u"):exits[0]]
    assert "p.cut[blockIdx.x] = make_int4(-1, 0, 0, 0)" in early
    assert "pdl_wait()" in early and early.index("pdl_wait()") < early.index("p.cut[")
