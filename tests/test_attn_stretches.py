"""How a decode step's contexts are cut into stretches, and which bytes of a page a tile's copies read,
built here for the host: every unit of a context is taken once, what is joined is what was written,
and no copy leaves its page."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kda_gated_delta_chunked_amd", "csrc")
UNIT = 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("stretches") / "libstretches_host.so")
    subprocess.check_call([hipcc, "-O1", "-std=c++17", "-fPIC", "-shared", "--offload-arch=gfx950", "-I", CSRC,
                           os.path.join(os.path.dirname(__file__), "stretches_host.cpp"), "-o", out])
    lib = ctypes.CDLL(out)
    lib.kda_test_in_cache.argtypes = [ctypes.c_int] * 3 + [ctypes.c_int64] * 2
    lib.kda_test_in_cache.restype = ctypes.c_int64
    return lib


def rows_of(f, lengths, parts, cols):
    cap = 2 * parts + len(lengths) + 8
    out = (ctypes.c_int64 * (cols * cap))()
    n = f((ctypes.c_int * len(lengths))(*lengths), len(lengths), parts, out, cap)
    assert 0 <= n <= cap
    return [tuple(out[cols * i:cols * (i + 1)]) for i in range(n)]


def check(lib, lengths, parts):
    taken = rows_of(lib.kda_test_stretches, lengths, parts, 5)
    units = [max(1, -(-x // UNIT)) for x in lengths]
    # every unit of every context once, in order, and stretches of one length but for the last
    assert [(n, u) for _, n, unit, take, _ in taken for u in range(unit, unit + take)] == \
        [(n, u) for n, of in enumerate(units) for u in range(of)]
    length = -(-sum(units) // parts)
    sizes = [sum(t[3] for t in taken if t[0] == w) for w in sorted({t[0] for t in taken})]
    assert all(s == length for s in sizes[:-1]) and 0 < sizes[-1] <= length and len(sizes) <= parts
    # whole requests alone are written out; each piece has a slot of its own
    written = [(n, slot) for _, n, _, take, slot in taken if take != units[n]]
    assert all((slot == -1) == (take == units[n]) for _, n, _, take, slot in taken)
    slots = [s for _, s in written]
    assert len(set(slots)) == len(slots) and all(0 <= s < 2 * parts for s in slots)
    # what is joined: the same requests' same slots, in the pieces' order
    joined = rows_of(lib.kda_test_cuts, lengths, parts, 3)
    assert [(n, slot) for n, _, slot in joined] == written
    of = {}
    for n, p, _ in joined:
        assert p == of.get(n, 0)
        of[n] = p + 1
    assert all(x >= 2 for x in of.values()) and len(of) <= min(parts - 1, len(lengths))


LISTS = [[5000], [0], [1, 128, 129, 0, 256, 257], [3000, 5, 0, 7000], [131072], [1] * 1000, [128] * 512, [129] * 512,
         [0] * 300 + [100000] + [0] * 300, [10 ** 9]]


@pytest.mark.parametrize("parts", [2, 3, 7, 32, 64, 256, 512])
@pytest.mark.parametrize("lengths", LISTS, ids=lambda x: f"{len(x)}x{max(x)}")
def test_stretches(lib, lengths, parts):
    if max(lengths) == 10 ** 9:  # (by its slots alone: it has 2^23 units)
        joined = rows_of(lib.kda_test_cuts, lengths, parts, 3)
        assert [t[4] for t in rows_of(lib.kda_test_stretches, lengths, parts, 5)] == [s for _, _, s in joined]
        return
    check(lib, lengths, parts)


def test_stretches_of_random_contexts(lib):
    rng = random.Random(5)
    for _ in range(300):
        n = int(2 ** rng.uniform(0, 10.5))
        most = int(2 ** rng.uniform(0, 14))
        lengths = [rng.choice((0, 1, UNIT, rng.randint(0, most), rng.randint(0, most))) for _ in range(n)]
        check(lib, lengths, rng.choice((2, 3, 5, 16, 31, 64, 128, 256, 512)))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("KV,gap", [(1, 0), (8, 0), (8, 1), (3, 16)])
def test_copies_of_a_tile(lib, KV, gap, D, e4m3):
    size = 1 if e4m3 else 2
    row = D * size
    token = KV * row * (1 + gap)
    per_row = row // 16
    out, places = (ctypes.c_int64 * (3 * 64 * 32))(), (ctypes.c_int * (32 * 16))()
    n = lib.kda_test_copies(D, int(e4m3), token, out, places)
    assert n == 32 * per_row
    at = {out[3 * i + 2]: (out[3 * i], out[3 * i + 1]) for i in range(n)}
    assert sorted(at) == list(range(0, 32 * row, 16))  # all of the tile, once
    for r in range(32):
        for c in range(per_row):  # a chunk is read from where its copy has put it
            assert at[places[r * per_row + c]] == (r // 16, r % 16 * token + c * 16)


def test_copies_of_the_longest_rows(lib):
    out, places = (ctypes.c_int64 * (3 * 64 * 32))(), (ctypes.c_int * (32 * 16))()
    token = ((1 << 23) - 16) * 2
    n = lib.kda_test_copies(128, 0, token, out, places)
    assert all(0 <= out[3 * i + 1] <= 15 * token + 256 - 16 for i in range(n))
    assert max(out[3 * i + 1] for i in range(n)) == 15 * token + 256 - 16


@pytest.mark.parametrize("shift", [4, 6, 10])
def test_halves_of_tiles_lie_in_one_page(lib, shift):
    rng = random.Random(shift)
    for _ in range(500):
        token = rng.choice((128, 1024, (1 << 23) - 16))
        page_stride = (token << shift) + rng.choice((0, 16, 1 << 20))
        page, pos = rng.choice((0, 1, (1 << 31) - 2, rng.randrange(1 << 31))), 16 * rng.randrange(1 << 26)
        page = min(page, (1 << 56) // page_stride)  # (no address space holds more)
        first, last = (lib.kda_test_in_cache(page, p, shift, page_stride, token) for p in (pos, pos + 15))
        assert first == page * page_stride + pos % (1 << shift) * token
        assert last == first + 15 * token and last + token <= page * page_stride + (token << shift)
