"""Kernel attributes and occupancy belong to a device: launchers keep them for
each device (csrc/per_device.h), not once per process."""
import glob
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "grouped_fp8_weight_gb300", "csrc")


def test_once_for_each_index():
    nvcc = next((c for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
                 if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "per_device_check")
        r = subprocess.run([nvcc, "-std=c++17", "-O2", "-I", CSRC, "-Xcompiler", "-pthread",
                            os.path.join(ROOT, "tests", "native", "per_device_check.cu"), "-o", exe],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_launcher_keeps_one_device_s_answer_for_all(path):
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.search(r"\bstatic\s+const\b[^;]*\bcuda(FuncSetAttribute|Occupancy|DeviceGet)", code)
