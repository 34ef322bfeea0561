"""CPU: what the kernels' sources may not do, because every launch may start
before the one in front of it has ended (programmatic stream serialization).
The effect of a breach depends on timing and on what a cache happens to hold,
so the sources are read."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "dense_gemm_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["ops_linear.cuh", "ops_norm.cuh"])
def test_nothing_is_promised_to_stay_the_same(name):
    """A restricted pointer to const and __ldg say that the data does not change
    while the kernel runs; what the launch in front of it writes does."""
    assert not re.findall(r"__restrict__|__ldg\s*\(|ld\.global\.nc", code(name))
