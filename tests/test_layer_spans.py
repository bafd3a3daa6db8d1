"""The span arithmetic of the layer operators (kda_spans.h, built here for the
host) at sizes that no test runs on a device."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
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


def spans(lib, cu, T, length, N=None):
    """[slots, 4] of (sequence, span, begin, end); cu None: N equal sequences."""
    packed = cu is not None
    N = len(cu) - 1 if packed else N
    cu = np.ascontiguousarray(cu if packed else [0], np.int64)
    out = np.full((T // length + N * (1 if packed else T // N // length + 2) + 1, 4), -7, np.int64)
    lib.kda_test_spans.restype = ctypes.c_int64
    n = lib.kda_test_spans(ctypes.c_void_p(cu.ctypes.data), int(packed), N, ctypes.c_int64(T), ctypes.c_uint32(length),
                           ctypes.c_void_p(out.ctypes.data), ctypes.c_int64(len(out)))
    assert n >= 0
    joins = np.zeros((N, 2), np.int64)
    for seq in range(N):
        lib.kda_test_join_slots(ctypes.c_void_p(cu.ctypes.data), int(packed), N, ctypes.c_int64(T),
                                ctypes.c_uint32(length), seq, ctypes.c_void_p(joins[seq:].ctypes.data))
    return out[:n], joins


def check_inside(got, joins, N, T, length):
    """What a workgroup of each slot touches: tokens of its span, the initial and
    final state of its sequence, its slot and (where pieces follow) the next."""
    for slot, (seq, k, begin, end) in enumerate(got.tolist()):
        assert 0 <= seq < N
        if k < 0:
            continue
        first = begin + k * length
        assert 0 <= begin <= end <= T and (first < end or (k == 0 and begin == end))
        if end - first > length:
            assert slot + 1 < len(got)
    for first, pieces in joins.tolist():
        assert 0 <= first and first + max(pieces, 1) <= len(got)


LENGTHS = [8, 16, 64, 192, 1 << 31]


@pytest.mark.parametrize("length", LENGTHS)
def test_every_token_has_one_span(lib, length):
    rng = np.random.default_rng(1)
    for case in range(150):
        N = int(rng.integers(1, 200)) if case % 3 else int(rng.integers(1, 4))
        lens = rng.integers(0, rng.choice([2, 9, 70, 500]), N)
        if case % 3 == 0:
            lens[:] = lens[0]
        cu = np.concatenate([[0], np.cumsum(lens)])
        T = int(cu[-1]) + int(rng.integers(0, 40))
        equal = case % 3 == 0 and T == cu[-1]
        for got, joins in [spans(lib, cu, T, length)] + ([spans(lib, None, T, length, N)] if equal else []):
            check_inside(got, joins, N, T, length)
            want = [(n, k, int(cu[n]), int(cu[n + 1])) for n in range(N) for k in range(max(1, -(-int(lens[n]) // length)))]
            assert [tuple(r) for r in got.tolist() if r[1] >= 0] == want
            for n in range(N):  # a sequence's pieces follow one another where the join looks for them
                at = [i for i, r in enumerate(got.tolist()) if r[1] >= 0 and r[0] == n]
                assert at == list(range(joins[n, 0], joins[n, 0] + len(at)))


@pytest.mark.parametrize("length", LENGTHS)
def test_bad_offsets_stay_inside(lib, length):
    rng = np.random.default_rng(2)
    for case in range(300):
        N, T = int(rng.integers(1, 300 if case % 4 == 0 else 12)), int(rng.integers(0, 600))
        kind = case % 3
        if kind == 0:    # any order
            cu = rng.integers(0, T + 1, N + 1)
        elif kind == 1:  # outside the batch
            cu = rng.integers(-2 * T - 3, 3 * T + 3, N + 1)
        else:            # far outside
            cu = rng.choice([-(1 << 40), -1, 0, T, T + 1, 1 << 31, 1 << 33], N + 1)
        got, joins = spans(lib, cu, T, length)
        check_inside(got, joins, N, T, length)
