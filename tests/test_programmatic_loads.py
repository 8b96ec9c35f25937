"""Kernels launched programmatically run while the kernel before them still writes what
they are going to read: they may not read it as data that stays constant (__ldg, or
const __restrict__, which lets the compiler choose that load and move it across the
wait for the kernel before). Looked up in the sources (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routed_expert_ffn_05_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["fp8_gemm.cu", "norm.cu", "combine.cu"])
def test_no_load_that_promises_constant_data(name):
    src = code(name)
    assert "programmaticStreamSerializationAllowed" in src and "grid_dep_wait();" in src
    assert not re.findall(r"__ldg\(|ld\.global\.nc|__restrict__", src)
