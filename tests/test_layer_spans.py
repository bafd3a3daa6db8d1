"""The span arithmetic of the layer operators (kda_spans.h, built here for the
host) at sizes that no test runs on a device."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kda_gated_delta_chunked_amd", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("spans") / "libspans_host.so")
    subprocess.check_call([hipcc, "-O1", "-std=c++17", "-fPIC", "-shared", "--offload-arch=gfx950",
                           "-I", CSRC, os.path.join(os.path.dirname(__file__), "spans_host.cpp"), "-o", out])
    return ctypes.CDLL(out)


@pytest.mark.parametrize("most", [32, 64])
@pytest.mark.parametrize("row_bytes,width", [(4, 4), (48, 4), (512, 4), (1 << 18, 8), ((1 << 24) - 16, 256)])
def test_a_window_covers_the_rows_that_are_read(lib, most, row_bytes, width):
    for left in (-96, 0, 1, 2, most - 1, most, most + 1, 1 << 13, 1 << 20, 1 << 23, (1 << 23) + 1, 1 << 30, (1 << 31) - 1):
        rows = max(0, min(left, most))
        want = (rows - 1) * row_bytes + width if rows else 0
        assert lib.kda_test_window_bytes(left, most, row_bytes, width) == want < 1 << 31


def test_every_window_has_a_bound():
    # the scan takes its windows through kda::window_bytes, with a bound on the rows
    text = open(os.path.join(CSRC, "kda_ssm.hip")).read()
    assert len(re.findall(r"make_buffer_rsrc", text)) == 1 and "window_bytes(left, MOST, row_bytes, width)" in text
    assert set(re.findall(r"\.window<(\w+)>\(", text)) == {"L", "BLOCK"} and ".window(" not in text


def test_no_row_of_a_long_sequence_is_left_out(lib):
    lib.kda_test_rows_left.argtypes = [ctypes.c_int64, ctypes.c_int64]
    for start in (0, 1, 1 << 30):
        for rows in (0, 1, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 1 - start):
            if rows <= (1 << 31) - 1 - start:
                assert lib.kda_test_rows_left(start, start + rows) == rows
    # the scan counts with it, from all rows down
    text = open(os.path.join(CSRC, "kda_ssm.hip")).read()
    assert re.findall(r"int rem = (.*?);", text) == ["rows_left(from, to)"]
