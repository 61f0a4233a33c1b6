"""What the MoE step's kernel sources have to keep to, read as text: rules whose
breach gives right results on most days."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_fp8_weight_gb300", "csrc")


def _code(path):
    """The file without comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def _dependents():
    """Sources of kernels launched as programmatic dependents, and what they include."""
    files = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_step(" in _code(p)]
    extra = {os.path.join(CSRC, h) for p in files
             for h in re.findall(r'#include "([^"]+)"', open(p).read())}
    return sorted(files) + sorted(p for p in extra if os.path.exists(p))


def test_there_are_such_kernels():
    names = {os.path.basename(p) for p in _dependents()}
    assert {"moe_exchange.cu", "quant_rows.cu", "linear_fp8.cu", "linear_pair.cu", "adamw.cu",
            "linear_table.cuh"} <= names


@pytest.mark.parametrize("path", _dependents(), ids=os.path.basename)
def test_inputs_are_read_with_ordinary_loads(path):
    """A programmatic dependent may be running while the kernel before it writes
    what it is going to read.  The read-only path is for data that nothing
    writes while the kernel runs, and waiting does not order it."""
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", _code(path))


@pytest.mark.parametrize("path", [p for p in _dependents() if p.endswith(".cu")], ids=os.path.basename)
def test_every_kernel_waits_for_the_one_before(path):
    code = _code(path)
    assert len(re.findall(r"\bkernel_begin\(\)", code)) == len(re.findall(r"__global__", code))
