"""Kernels that start while the kernel before them ends may not read what that
one writes by non-coherent loads, which the wait for it does not order."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layer_streamed_qlora_b200", "csrc")


def code(path):
    src = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", src)


EARLY = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "grid_dep_wait()" in code(p))


def test_the_kernels_that_start_early_are_known():
    assert EARLY == ["mx4.cu", "mx4_few.cu", "mx4_mid.cu", "optim_group.cu"]
    launching = [os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "dependent_launch(" in code(p)]
    assert sorted(launching) == EARLY


@pytest.mark.parametrize("name", EARLY + ["mx4.cuh"])
def test_no_non_coherent_loads(name):
    src = code(os.path.join(CSRC, name))
    for word in (r"__ldg\b", r"global\.nc\b", r"const\s[^,;()]*\*\s*__restrict__"):
        assert not re.findall(word, src), word


def test_the_shared_global_accesses_are_coherent():
    body = code(os.path.join(CSRC, "ptx.cuh"))
    assert "ld.global.v8.b32" in body and "global.nc" not in body
