"""The windows through which the attention kernels copy rows, built here for the host: no
row ahead of a sequence or behind it is ever inside one."""
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
    out = str(tmp_path_factory.mktemp("attn") / "libattn_host.so")
    subprocess.check_call([hipcc, "-O1", "-std=c++17", "-fPIC", "-shared", "--offload-arch=gfx950", "-I", CSRC,
                           os.path.join(os.path.dirname(__file__), "attn_host.cpp"), "-o", out])
    return ctypes.CDLL(out)


@pytest.mark.parametrize("row_bytes,width", [(128, 128), (3328, 256), ((1 << 24) - 16, 256)])
def test_a_window_holds_rows_of_the_sequence_alone(lib, row_bytes, width):
    most = 32
    for length in (1, 31, 32, 33, 300, (1 << 31) - 1):
        for first in (0, 1, 32, length - 1, length, min(length + 96, (1 << 31) - 1)):
            rows = max(0, min(most, length - first))
            assert lib.kda_test_rows_bytes(first, length, most, row_bytes) == rows * row_bytes < 1 << 31
            # which holds these rows' columns, and nothing of others
            assert all(r * row_bytes + width <= rows * row_bytes for r in range(rows))
            assert all(r * row_bytes >= rows * row_bytes for r in range(rows, most))


def test_every_copy_goes_through_a_window():
    text = open(os.path.join(CSRC, "kda_attn.hip")).read()
    # one kind of copy, of a window whose rows are counted, from the sequence's first row on
    assert len(re.findall(r"copy_to_lds\(", text)) == 1 and "rows_bytes(first, length, KEYS, bytes)" in text
    assert "(key ? copied : max(copied - 2, 0)) * (KEYS * SPLIT)" in text
    # and all are waited for before the workgroup ends
    assert "memory_left<0>();  // no copy outlives the workgroup" in open(os.path.join(CSRC, "kda_attn_tiles.h")).read()
