"""CPU: test_launch_rules.py's reading of the sources, for layer norm, rows in 8 bits and what
stands in front of 16-bit products."""
import re

import pytest

from test_launch_rules import code


@pytest.mark.parametrize("name", ["elements.cuh", "ops_rows.cu", "ops_eight.cuh"])
def test_nothing_is_promised_to_stay_the_same(name):
    assert not re.findall(r"__restrict__|__ldg\s*\(|ld\.global\.nc", code(name))


def test_reads_before_the_own_wait_pass_l1():
    """D's pass from 8-bit values, which may start without waiting (`late`)."""
    eight = code("ops_eight.cuh")
    rows = eight[eight.index("void saved_grad_rows("):eight.index("saved_grad_kernel(")]
    assert ".fetch(" in rows and "load_eight<" in rows and "__ldcg(s.scale + row)" in rows and "load_raw" not in rows
    load = eight[eight.index("uint2 load_eight("):]
    load = load[:load.index("\n}")]
    assert load.count("__ldcg(") == 3


def test_every_kernel_along_rows_waits_for_the_one_before():
    rows = code("ops_rows.cu")
    kernels = re.findall(r"__global__ void[^{]*\{", rows)
    assert len(kernels) == rows.count("griddep_wait();") == rows.count("griddep_launch_dependents();") == 8


def test_integer_products_read_nothing_but_weights_before_their_wait():
    """With the tokens copied by the kernel before it, linear_int8 starts on the weights (by TMA, from
    L2) at once; tokens, factors and the residual come after a wait of the warp that reads them."""
    eight = code("ops_eight.cuh")
    body = eight[eight.index("linear_int8(const __grid_constant__"):]
    wait = body.index("if constexpr (kWide) {\n                griddep_wait();")
    assert body.index("load_x(mode, st, uint32_t(st - st0))") > wait
    assert body.index("griddep_launch_dependents();") > wait
    assert body.index("split_columns<true, true>") > body.index("if constexpr (kWide) griddep_wait();") > wait
