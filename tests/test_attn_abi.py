"""Host-side checks of include/kda_attn.h: every declared function is exported,
the binding's structures are the header's, and bad arguments are refused
before anything reaches a device (fake addresses, never dereferenced)."""
import ctypes
import inspect
import os
import re
import shutil
import subprocess

import pytest

import kda_gated_delta_chunked_amd as K
from kda_gated_delta_chunked_amd import attn as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_attn.h")
OK, INVALID, UNSUPPORTED, ALIGN, OVERLAP, WS, TOO_LARGE = 0, -1, -2, -3, -4, -5, -6


def at(i):
    return (1 << 44) + (i << 38)


def test_library_exports_every_declared_function():
    names = set(re.findall(r"^kda_status (kda_[a-z_]+)\(", open(HEADER).read(), re.M))
    assert names == set(A._SIGNATURES)
    lib = K.load_library()
    for name in names:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("struct,mirror", [
    ("kda_attn_problem", A.PrefillProblem), ("kda_kv_cache", A.KvCache), ("kda_attn_decode_problem", A.DecodeProblem),
    ("kda_kv_store_problem", A.StoreProblem), ("kda_kv_assign_problem", A.AssignProblem)])
def test_header_is_c_and_structures_match(struct, mirror, tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    fields = [f[0] for f in mirror._fields_]
    lines = "".join(f'printf("%zu %zu\\n", offsetof({struct}, {f}), sizeof((({struct}*)0)->{f}));\n' for f in fields)
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kda_attn.h"\n'
                   f'int main(void) {{ printf("%zu 0\\n", sizeof({struct}));\n{lines}return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [tuple(map(int, x.split())) for x in subprocess.check_output([str(exe)], text=True).splitlines()]
    assert got[0][0] == ctypes.sizeof(mirror)
    for (off, size), f in zip(got[1:], fields):
        assert (off, size) == (getattr(mirror, f).offset, getattr(mirror, f).size), f


# ---------------------------------------------------------------------------

def prompt(N=2, T=100, H=4, KV=2, D=64, scale=0.125, cu64=0, qs=0, ks=0, vs=0, os_=0, **over):
    names = ["q", "k", "v", "cu", "out", "lse"]
    a = {n: at(i) for i, n in enumerate(names)} | over
    return A.call_raw("kda_attn_validate", A.PrefillProblem(N, T, H, KV, D, scale, cu64, qs, ks, vs, os_),
                      *[a[n] for n in names])


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(lse=0)), (OK, dict(cu=0)), (OK, dict(T=0, q=0, k=0, v=0, out=0, lse=0)),
    (OK, dict(k=at(0), v=at(0))),                                   # inputs may share
    (OK, dict(qs=512, ks=512, vs=512, k=at(0) + 512, v=at(0) + 768)),  # columns of one row
    (OK, dict(D=128, H=6, KV=1)),
    (INVALID, dict(N=0)), (INVALID, dict(T=-1)), (INVALID, dict(H=0)), (INVALID, dict(KV=0)), (INVALID, dict(KV=3)),
    (UNSUPPORTED, dict(D=96)), (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=float("nan"))), (INVALID, dict(cu64=2)),
    (INVALID, dict(qs=248)), (INVALID, dict(qs=260)), (INVALID, dict(ks=120)), (INVALID, dict(vs=1 << 23)),
    (INVALID, dict(os_=-8)), (INVALID, dict(cu=0, T=101)), (INVALID, dict(q=0)), (INVALID, dict(v=0)),
    (INVALID, dict(out=0)), (ALIGN, dict(k=at(1) + 8)), (ALIGN, dict(lse=at(5) + 4)), (OVERLAP, dict(out=at(0))),
    (OVERLAP, dict(out=at(1) + 64)), (OVERLAP, dict(lse=at(4))), (OVERLAP, dict(lse=at(3))),
    (OVERLAP, dict(out=at(0) + 256 * 2, qs=512)),                   # inside the strided span of q
    (TOO_LARGE, dict(T=1 << 31)), (TOO_LARGE, dict(H=1 << 17)), (TOO_LARGE, dict(N=1 << 24, lse=0)),
    (OK, dict(N=1 << 21, lse=0))])
def test_prompt_checks(want, kw):
    assert prompt(**kw) == want


def cache(KV=2, D=64, dt=0, size=16, pages=10, page=0, token=0):
    return A.KvCache(KV, D, dt, size, pages, page, token)


STEP = ["q", "kc", "vc", "table", "rows", "lens", "tree", "ks", "vs", "out", "lse", "ws"]


def step(n=3, T=2, H=4, scale=0.125, R=5, W=4, per_seq=1, qs=0, os_=0, ws_bytes=1 << 30, c=None, **over):
    a = {x: at(i) for i, x in enumerate(STEP)} | {"ks": 0, "vs": 0} | over
    p = A.DecodeProblem(n, T, H, scale, R, W, per_seq, qs, os_, c or cache())
    return A.call_raw("kda_attn_decode_validate", p, *[a[x] for x in STEP], ws_bytes)


E4M3 = dict(ks=at(7), vs=at(8))


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(tree=0, rows=0, lse=0)), (OK, dict(per_seq=0)), (OK, dict(out=at(0))),
    (OK, dict(n=0, **{x: 0 for x in STEP})), (OK, dict(R=0, table=0)), (OK, dict(T=64)),
    (OK, dict(c=cache(dt=1), **E4M3)), (OK, dict(qs=512, os_=512, out=at(0))),
    (OK, dict(vc=at(1))),                                           # only read: may share
    (INVALID, dict(n=-1)), (INVALID, dict(T=0)), (UNSUPPORTED, dict(T=65)), (INVALID, dict(H=3)), (INVALID, dict(H=0)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(R=-1)), (INVALID, dict(W=0)), (INVALID, dict(per_seq=2)),
    (TOO_LARGE, dict(W=(1 << 26) + 1)), (TOO_LARGE, dict(R=1 << 31)), (INVALID, dict(qs=100)),
    (INVALID, dict(q=0)), (INVALID, dict(kc=0)), (INVALID, dict(table=0)), (INVALID, dict(lens=0)),
    (INVALID, dict(out=0)), (INVALID, E4M3), (INVALID, dict(c=cache(dt=1))), (INVALID, dict(c=cache(dt=1), ks=at(7))),
    (UNSUPPORTED, dict(c=cache(dt=2))), (UNSUPPORTED, dict(c=cache(D=96))), (UNSUPPORTED, dict(c=cache(size=8))),
    (UNSUPPORTED, dict(c=cache(size=48))), (UNSUPPORTED, dict(c=cache(size=2048))), (INVALID, dict(c=cache(KV=0))),
    (INVALID, dict(c=cache(pages=0))), (TOO_LARGE, dict(c=cache(pages=1 << 31))), (INVALID, dict(c=cache(token=120))),
    (INVALID, dict(c=cache(token=136))), (INVALID, dict(c=cache(page=2032))), (INVALID, dict(c=cache(page=-2048))),
    (TOO_LARGE, dict(c=cache(page=1 << 41))),
    (ALIGN, dict(lens=at(5) + 4)), (ALIGN, dict(kc=at(1) + 8)), (OVERLAP, dict(out=at(0) + 16)),
    (OVERLAP, dict(out=at(0), qs=512)), (OVERLAP, dict(out=at(1))), (OVERLAP, dict(out=at(3))),
    (OVERLAP, dict(lse=at(0))), (OVERLAP, dict(lse=at(6))), (OVERLAP, dict(ws=at(9))), (OVERLAP, dict(ws=at(2))),
    (WS, dict(W=4096, ws_bytes=64)), (WS, dict(W=4096, ws=0)), (TOO_LARGE, dict(n=1 << 30, T=4)),
    (TOO_LARGE, dict(n=1 << 23, T=1, H=8, c=cache(KV=8)))])
def test_decode_checks(want, kw):
    assert step(**kw) == want


def test_decode_workspace():
    # contexts over long tables are cut into stretches, with two numbers and a row of
    # sums for each end of a stretch and row; many rows of many requests, or short tables, are not
    def size(n, T, H, W, **c):
        return A.decode_workspace_size(A.DecodeProblem(n, T, H, 0.1, n, W, 0, 0, 0, cache(**c)))
    assert size(1024, 64, 32, 1024, KV=8) == 0
    assert size(1, 1, 4, 1) == 0
    assert size(4096, 1, 32, 1024, KV=8) == size(512, 1, 32, 1024, KV=8)
    assert size(0, 1, 4, 1024) == 0
    got = size(1, 1, 8, 8192, KV=8, D=128)
    assert got > 0 and got % (8 * 130 * 4) == 0
    # never more than some share of what the contexts themselves hold
    for n in (1, 3, 17, 200):
        for T in (1, 4, 64):
            assert size(n, T, 32, 4096, KV=8, D=128) <= 1 << 30


def test_store_checks():
    names = ["k", "v", "slots", "ks", "vs", "kc", "vc"]

    def call(T=100, ks_=0, vs_=0, c=None, **over):
        a = {n: at(i) for i, n in enumerate(names)} | {"ks": 0, "vs": 0} | over
        return A.call_raw("kda_kv_store_validate", A.StoreProblem(T, ks_, vs_, c or cache()), *[a[n] for n in names])

    e4m3 = dict(ks=at(3), vs=at(4))
    assert call() == OK
    assert call(T=0, **{n: 0 for n in names}) == OK
    assert call(c=cache(dt=1), **e4m3) == OK
    assert call(v=at(0)) == OK
    assert call(ks_=256, vs_=256, v=at(0) + 256) == OK
    for kw in (dict(T=-1), dict(ks_=120), dict(ks_=132), dict(vs_=-128), dict(k=0), dict(slots=0), dict(vc=0), e4m3,
               dict(c=cache(dt=1))):
        assert call(**kw) == INVALID, kw
    assert call(T=1 << 31) == TOO_LARGE
    assert call(T=1 << 30, c=cache(KV=1)) == TOO_LARGE
    assert call(slots=at(2) + 8) == ALIGN
    for kw in (dict(kc=at(0)), dict(vc=at(2)), dict(vc=at(1) + 64), dict(vc=at(5)), dict(vc=at(5) + 256)):
        assert call(**kw) == OVERLAP, kw


def test_caches_may_be_halves_of_one_buffer():
    KV, D, size, pages = 2, 64, 16, 10
    row, page = KV * D, KV * D * size

    def call(gap, **c):
        return A.call_raw("kda_kv_store_validate", A.StoreProblem(4, 0, 0, cache(KV, D, 0, size, pages, **c)),
                          at(0), at(1), at(2), 0, 0, at(5), at(5) + gap * 2)

    both = lambda p, t: dict(page=p, token=t)
    assert call(page, **both(2 * page, 0)) == OK                  # [pages, 2, size, KV, D]
    assert call(row, **both(2 * page, 2 * row)) == OK             # [pages, size, 2, KV, D]
    assert call(page * pages) == OK                               # [2, pages, size, KV, D]
    assert call(page - 8, **both(2 * page, 0)) == OVERLAP
    assert call(page + 8, **both(2 * page, 0)) == OVERLAP
    assert call(row - 8, **both(2 * page, 2 * row)) == OVERLAP
    assert call(row + 8, **both(2 * page, 2 * row)) == OVERLAP
    assert call(page) == OVERLAP


def test_assign_checks():
    names = ["lens", "rows", "cu", "table", "free", "head", "slots", "lens_out", "head_out"]

    def call(N=3, T=9, size=16, W=4, R=5, F=20, cu64=0, **over):
        a = {n: at(i) for i, n in enumerate(names)} | over
        return A.call_raw("kda_kv_assign_validate", A.AssignProblem(N, T, size, W, R, F, cu64), *[a[n] for n in names])

    assert call() == OK
    assert call(rows=0, cu=0) == OK
    assert call(T=0, slots=0) == OK
    assert call(R=0, table=0, F=0, free=0) == OK
    for kw in (dict(N=0), dict(T=-1), dict(W=0), dict(R=-1), dict(F=-1), dict(cu64=2), dict(cu=0, T=10), dict(lens=0),
               dict(head=0), dict(slots=0), dict(lens_out=0), dict(head_out=0), dict(table=0), dict(free=0)):
        assert call(**kw) == INVALID, kw
    assert call(size=24) == UNSUPPORTED
    for kw in (dict(T=1 << 31), dict(W=(1 << 26) + 1), dict(R=1 << 31), dict(F=1 << 31)):
        assert call(**kw) == TOO_LARGE, kw
    assert call(head=at(5) + 4) == ALIGN
    for kw in (dict(lens_out=at(0)), dict(head_out=at(5)), dict(table=at(1)), dict(slots=at(2)), dict(table=at(4)),
               dict(slots=at(3)), dict(head_out=at(7))):
        assert call(**kw) == OVERLAP, kw


def test_a_null_problem_is_refused():
    for name, (_, rest) in A._SIGNATURES.items():
        assert A._fn(name)(None, *[0 if t is ctypes.c_size_t else None for t in rest]) == INVALID, name


def test_binding_refuses_before_the_library():
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    x, pool, table, lens = z(1, 4, 64), z(2, 16, 1, 64), z(1, 2, dtype=i32), z(1, dtype=i32)
    for call in (lambda: A.prefill(x, x, x), lambda: A.decode(x[None], pool, pool, table, lens),
                 lambda: A.store(x, x, pool, pool, z(1, dtype=torch.int64)),
                 lambda: A.assign_pages(lens, table, lens, lens, page_size=16)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_the_submodule_is_public():
    assert K.attn is A and "attn" in K.__all__
    assert set(A.__all__) <= set(dir(A))
    streams = {n for n in A.__all__ if inspect.isfunction(getattr(A, n)) and "stream" in inspect.signature(getattr(A, n)).parameters}
    assert streams == {"prefill", "decode", "store", "assign_pages"}
