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


@pytest.mark.parametrize("name", ["ops_linear.cuh", "ops_norm.cuh", "gemm_kernel.cuh", "gemm_pair.cuh"])
def test_nothing_is_promised_to_stay_the_same(name):
    """A restricted pointer to const and __ldg say that the data does not change
    while the kernel runs; what the launch in front of it writes does."""
    assert not re.findall(r"__restrict__|__ldg\s*\(|ld\.global\.nc", code(name))


def test_reads_before_the_own_wait_pass_l1():
    """The first loads of kernels that start without waiting (`late`): D's pass and
    the last step of the column sums."""
    linear, norm = code("ops_linear.cuh"), code("ops_norm.cuh")
    fetch = linear[linear.index("struct GradLoad"):linear.index("struct GradLoad") + linear[linear.index("struct GradLoad"):].index("values(")]
    assert fetch.count("load_raw_l2<T>(") == 3 and "load_raw<" not in fetch
    rows = linear[linear.index("void grad_rows("):linear.index("void grad_rows(") + linear[linear.index("void grad_rows("):].index("__global__")]
    assert ".fetch(" in rows and "load_raw" not in rows
    body = norm[norm.index("sum_partials_kernel("):]
    assert body.count("partial + r * width + col") == 1 and "__ldcg(partial + r * width + col)" in body
    raw = norm[norm.index("load_raw_l2(const T *p)"):]
    assert "__ldcg(" in raw[:raw.index("return r;")]
