"""Host-side checks of include/kda_ssm.h: every declared function is exported,
the binding's structures are the header's, and bad arguments are refused
before anything reaches a device (fake addresses, never dereferenced)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import kda_gated_delta_chunked_amd as K
from kda_gated_delta_chunked_amd import ssm_ops as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_ssm.h")
OK, INVALID, UNSUPPORTED, ALIGN, OVERLAP, WS, TOO_LARGE = 0, -1, -2, -3, -4, -5, -6
FAR = 1 << 36


def at(i):
    return (1 << 44) + i * FAR


def test_library_exports_every_declared_function():
    names = set(re.findall(r"^kda_status (kda_[a-z_]+)\(", open(HEADER).read(), re.M))
    assert names == set(S._SIGNATURES)
    lib = K.load_library()
    for name in names:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("struct,mirror", [
    ("kda_conv_problem", S.ConvProblem), ("kda_conv_decode_problem", S.ConvDecodeProblem),
    ("kda_ssm_problem", S.SsmProblem), ("kda_ssm_decode_problem", S.SsmDecodeProblem),
    ("kda_norm_problem", S.NormProblem)])
def test_header_is_c_and_structures_match(struct, mirror, tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    fields = [f[0] for f in mirror._fields_]
    lines = "".join(f'printf("%zu %zu\\n", offsetof({struct}, {f}), sizeof((({struct}*)0)->{f}));\n' for f in fields)
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "kda_ssm.h"\n'
                   f'int main(void) {{ printf("%zu 0\\n", sizeof({struct}));\n{lines}return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [tuple(map(int, x.split())) for x in subprocess.check_output([str(exe)], text=True).splitlines()]
    assert got[0][0] == ctypes.sizeof(mirror)
    for (off, size), f in zip(got[1:], fields):
        assert (off, size) == (getattr(mirror, f).offset, getattr(mirror, f).size), f


# ---------------------------------------------------------------------------

def conv(T=100, N=2, D=64, W=4, act=1, cu64=0, xs=0, os_=0, **over):
    a = dict(x=at(0), w=at(1), b=at(2), cu=at(3), s0=at(4), out=at(5), fin=at(6)) | over
    p = S.ConvProblem(N, T, D, W, act, cu64, xs, os_)
    return S.call_raw("kda_conv_validate", p, a["x"], a["w"], a["b"], a["cu"], a["s0"], a["out"], a["fin"])


def test_conv_accepts():
    assert conv() == OK
    assert conv(b=0, s0=0, fin=0) == OK
    assert conv(cu=0) == OK
    assert conv(T=0, x=0, out=0) == OK
    assert conv(fin=at(4)) == OK          # the state updated in place
    assert conv(xs=72, os_=128) == OK


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(N=0)), (INVALID, dict(T=-1)), (INVALID, dict(D=0)), (UNSUPPORTED, dict(D=12)),
    (UNSUPPORTED, dict(W=1)), (UNSUPPORTED, dict(W=5)), (UNSUPPORTED, dict(act=2)), (INVALID, dict(cu64=2)),
    (INVALID, dict(xs=56)), (INVALID, dict(xs=68)), (INVALID, dict(os_=-8)), (INVALID, dict(w=0)),
    (INVALID, dict(x=0)), (INVALID, dict(out=0)), (INVALID, dict(cu=0, T=101)), (ALIGN, dict(x=at(0) + 2)),
    (ALIGN, dict(fin=at(6) + 8)), (OVERLAP, dict(out=at(0))), (OVERLAP, dict(out=at(0) + 64)),
    (OVERLAP, dict(out=at(4))), (OVERLAP, dict(fin=at(4) + 128)), (OVERLAP, dict(fin=at(0))),
    (OVERLAP, dict(out=at(0) + 6400 * 2, xs=128)),  # inside the strided span of x
    (TOO_LARGE, dict(T=1 << 31)), (TOO_LARGE, dict(T=1 << 30, D=1 << 20, x=1 << 50, out=1 << 56))])
def test_conv_refuses(want, kw):
    assert conv(**kw) == want


def conv_step(n=3, T=2, D=64, W=4, act=1, pool=5, xs=0, os_=0, **over):
    a = dict(x=at(0), w=at(1), b=at(2), pool=at(3), idx=at(4), out=at(5)) | {k: v for k, v in over.items()}
    p = S.ConvDecodeProblem(n, T, D, W, act, pool, xs, os_)
    return S.call_raw("kda_conv_decode_validate", p, a["x"], a["w"], a["b"], over.get("sp", at(3)), a["idx"], a["out"])


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(n=0, x=0, w=0, sp=0, idx=0, out=0)), (OK, dict(out=at(0))), (OK, dict(b=0)),
    (OK, dict(xs=128, os_=128, out=at(0))), (OVERLAP, dict(xs=128, out=at(0))), (OVERLAP, dict(out=at(0) + 128)),
    (INVALID, dict(n=-1)), (INVALID, dict(T=0)), (INVALID, dict(pool=0)), (INVALID, dict(sp=0)),
    (INVALID, dict(idx=0)), (OVERLAP, dict(sp=at(0))), (OVERLAP, dict(out=at(3))), (ALIGN, dict(idx=at(4) + 4)),
    (UNSUPPORTED, dict(D=4)), (TOO_LARGE, dict(n=1 << 30, T=8))])
def test_conv_decode_checks(want, kw):
    assert conv_step(**kw) == want


def ssm_problem(N=2, T=128, H=4, G=2, P=64, S_=128, soft=1, sd=0, cu64=0, piece=0, packed=1, xs=0, bs=0, cs=0, zs=0,
                os_=0):
    return S.SsmProblem(N, T, H, G, P, S_, soft, sd, cu64, piece, packed, xs, bs, cs, zs, os_)


NAMES = ["x", "dt", "A", "B", "C", "D", "z", "bias", "cu", "s0", "out", "fin", "ws"]


def ssm(ws_bytes=0, p=None, **kw):
    over = {k: kw.pop(k) for k in list(kw) if k in NAMES}
    a = {k: at(i) for i, k in enumerate(NAMES)} | {"ws": 0} | over
    return S.call_raw("kda_ssm_validate", p or ssm_problem(**kw), *[a[k] for k in NAMES], ws_bytes)


def test_ssm_accepts():
    assert ssm() == OK
    assert ssm(D=0, z=0, bias=0, s0=0, fin=0) == OK
    assert ssm(cu=0, packed=0) == OK
    assert ssm(T=0, x=0, dt=0, B=0, C=0, out=0) == OK
    assert ssm(fin=at(NAMES.index("s0"))) == OK
    # x, B and C as columns of one row
    assert ssm(xs=512, bs=512, cs=512, B=at(0) + 512, C=at(0) + 768) == OK


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, dict(P=32)), (UNSUPPORTED, dict(S_=256)), (INVALID, dict(H=0)), (INVALID, dict(G=0)),
    (INVALID, dict(G=3)), (INVALID, dict(soft=2)), (UNSUPPORTED, dict(sd=2)), (INVALID, dict(N=0)),
    (INVALID, dict(T=-1)), (INVALID, dict(piece=-64)), (INVALID, dict(piece=32)), (INVALID, dict(piece=96)), (WS, dict(piece=64)), (INVALID, dict(xs=248)), (INVALID, dict(xs=1 << 23)),
    (INVALID, dict(bs=250)), (INVALID, dict(zs=260)), (INVALID, dict(A=0)), (INVALID, dict(x=0)),
    (INVALID, dict(dt=0)), (INVALID, dict(C=0)), (INVALID, dict(out=0)), (INVALID, dict(cu=0, packed=0, T=129)),
    (INVALID, dict(cu=0)), (INVALID, dict(packed=0)), (INVALID, dict(packed=2)), (ALIGN, dict(dt=at(1) + 4)), (ALIGN, dict(B=at(3) + 2)), (OVERLAP, dict(out=at(0))),
    (OVERLAP, dict(out=at(1))), (OVERLAP, dict(out=at(9))), (OVERLAP, dict(fin=at(9) + 16)),
    (OVERLAP, dict(fin=at(6))), (TOO_LARGE, dict(T=1 << 31)), (TOO_LARGE, dict(H=1 << 24)),
    (TOO_LARGE, dict(N=1 << 30, H=2, G=2))])
def test_ssm_refuses(want, kw):
    assert ssm(**kw) == want


def test_ssm_workspace_of_a_split():
    p = ssm_problem(N=3, T=1000, H=4, G=1, P=64, S_=128, piece=256)
    # floor(1000 / 256) + 3 pieces, a state and a decay per head
    want = (3 + 3) * 4 * (64 * 128 + 1) * 4
    assert K.ssm_workspace_size(p) == want and K.ssm_plan(p) == 256
    ws = dict(ws=at(12), p=p)
    assert ssm(want, **ws) == OK
    assert ssm(want - 1, **ws) == WS
    assert ssm(want, ws=0, p=p) == WS
    assert ssm(want, ws=at(10), p=p) == OVERLAP
    # no sequence is longer than the piece: nothing to split
    assert K.ssm_workspace_size(ssm_problem(N=1, T=256, piece=256)) == 0


@pytest.mark.parametrize("want,kw", [
    (1024, dict(N=8, T=65536, H=12, G=1, P=128, packed=0)), (0, dict(N=32, T=16384, H=12, G=1, P=128, packed=0)),
    (0, dict(N=1, T=37, H=4, P=64)), (0, dict(N=1, T=0)), (0, dict(N=256, T=4096, H=64))])
def test_ssm_automatic_pieces(want, kw):
    p = ssm_problem(**kw)
    assert K.ssm_plan(p) == want
    assert (K.ssm_workspace_size(p) > 0) == (want > 0)
    # without the workspace the scan runs unsplit
    assert ssm(0, p=p, **({} if kw.get("packed", 1) else dict(cu=0))) == OK


STEP = ["x", "dt", "A", "B", "C", "D", "z", "bias", "pool", "idx", "out"]


def ssm_step(n=3, T=1, H=4, G=2, P=64, S_=128, soft=0, sd=0, size=5, xs=0, os_=0, **over):
    a = {k: at(i) for i, k in enumerate(STEP)} | over
    p = S.SsmDecodeProblem(n, T, H, G, P, S_, soft, sd, size, xs, 0, 0, 0, os_)
    return S.call_raw("kda_ssm_decode_validate", p, *[a[k] for k in STEP])


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(out=at(0))), (OK, dict(n=0, **{k: 0 for k in STEP})), (OK, dict(D=0, z=0, bias=0)),
    (OVERLAP, dict(out=at(0), xs=512)), (OVERLAP, dict(out=at(0) + 16)), (OVERLAP, dict(out=at(8))),
    (OVERLAP, dict(pool=at(0))), (OVERLAP, dict(out=at(6))), (INVALID, dict(pool=0)), (INVALID, dict(size=0)),
    (INVALID, dict(T=0)), (INVALID, dict(H=3)), (UNSUPPORTED, dict(P=100)), (ALIGN, dict(pool=at(8) + 4)),
    (TOO_LARGE, dict(n=1 << 28, H=2)), (INVALID, dict(xs=100))])
def test_ssm_decode_checks(want, kw):
    assert ssm_step(**kw) == want


def norm(rows=4, D=256, eps=1e-6, dt=0, group=0, xs=0, **over):
    a = dict(x=at(0), res=at(1), w=at(2), out=at(3), sc=at(4) if dt else 0, ro=at(5)) | over
    p = S.NormProblem(rows, D, eps, dt, group, xs)
    return S.call_raw("kda_add_rmsnorm_validate", p, a["x"], a["res"], a["w"], a["out"], a["sc"], a["ro"])


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(dt=1)), (OK, dict(dt=1, group=128)), (OK, dict(res=0, ro=0)), (OK, dict(ro=0)),
    (OK, dict(ro=at(1))), (OK, dict(out=at(0))), (OK, dict(rows=0, x=0, w=0, out=0, res=0, ro=0)),
    (INVALID, dict(rows=-1)), (INVALID, dict(D=0)), (UNSUPPORTED, dict(D=12)), (UNSUPPORTED, dict(D=16392)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (UNSUPPORTED, dict(dt=2)),
    (UNSUPPORTED, dict(group=128)), (UNSUPPORTED, dict(dt=1, group=64)), (INVALID, dict(dt=1, sc=0)),
    (INVALID, dict(sc=at(4))), (INVALID, dict(res=0)), (INVALID, dict(x=0)), (INVALID, dict(xs=100)),
    (ALIGN, dict(w=at(2) + 2)), (OVERLAP, dict(out=at(0) + 16)), (OVERLAP, dict(out=at(0), dt=1)),
    (OVERLAP, dict(out=at(0), xs=512)), (OVERLAP, dict(ro=at(1) + 16)), (OVERLAP, dict(ro=at(0))),
    (OVERLAP, dict(out=at(1))), (OVERLAP, dict(dt=1, sc=at(3))), (TOO_LARGE, dict(rows=1 << 31))])
def test_norm_checks(want, kw):
    assert norm(**kw) == want


def test_a_null_problem_is_refused():
    for name, (_, rest) in S._SIGNATURES.items():
        assert S._fn(name)(None, *[0 if t is ctypes.c_size_t else None for t in rest]) == INVALID, name


def test_binding_refuses_before_the_library():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        K.conv_prefill(x, w)
    with pytest.raises(ValueError, match="GPU"):
        K.add_rmsnorm(x, w[:, 0])
    with pytest.raises(ValueError, match="x must be"):
        K.ssm_prefill(x, None, None, None, None)


@pytest.mark.parametrize("call", [
    # a launch has fewer than 2^32 threads: 64 per 8 or 16 tokens and 512
    # channels, 64 per request and 512 channels
    lambda far: conv(T=(1 << 30) + (1 << 29), N=1, D=8, x=at(0), out=at(0) + far),
    lambda far: conv(T=0, N=(1 << 26) + 1, D=8, x=0, out=0, cu=at(0), s0=0, fin=0),
    lambda far: conv_step(n=1 << 26, T=1, D=8, pool=4, x=at(0), out=at(0) + far),
    # two per sequence, head and column of an unsplit scan, or per piece of one
    lambda far: ssm(N=1 << 25, T=1 << 25, H=1, G=1, P=64, S_=64, s0=0, fin=0, x=at(0), out=at(0) + far),
    # one per four state elements of all sequences in a split's join
    lambda far: ssm(ws_bytes=1 << 47, N=100000, T=10000000, H=11, G=1, P=128, S_=128, piece=64, s0=0, fin=0, x=at(0),
                    out=at(0) + far, ws=at(0) + 2 * far),
    # 256 per request, head and 32 or 64 columns
    lambda far: ssm_step(n=1 << 22, T=1, H=1, G=1, P=128, x=at(0), out=at(0) + far),
    # 16 to 256 per row
    lambda far: norm(rows=1 << 28, D=8, x=at(0), out=at(0) + far, res=0, ro=0),
    lambda far: norm(rows=1 << 24, D=2056, x=at(0), out=at(0) + far, res=0, ro=0),
])
def test_more_threads_than_a_launch_takes_are_refused(call):
    assert call(1 << 50) == TOO_LARGE


@pytest.mark.parametrize("call", [
    # 2^26 - 7 waves of 64, in workgroups of four
    lambda far: conv(T=(1 << 30) - 128, N=1, D=8, x=at(0), out=at(0) + far),
    lambda far: ssm(N=1 << 24, T=1 << 24, H=1, G=1, P=64, S_=64, s0=0, fin=0, x=at(0), out=at(0) + far),
    lambda far: norm(rows=(1 << 28) - 16, D=8, x=at(0), out=at(0) + far, res=0, ro=0),
    # an automatic piece length whose join would be too large: unsplit
    lambda far: ssm(ws_bytes=0, N=100000, T=100000000, H=11, G=1, P=128, S_=128, s0=0, fin=0, x=at(0),
                    out=at(0) + far, ws=0),
])
def test_the_largest_launches_are_accepted(call):
    assert call(1 << 50) == OK


def test_short_sequences_are_not_split_unasked():
    # the binding relies on it: no workspace, and no call to ask for one
    text = open(HEADER).read()
    assert f"#define KDA_SSM_SPLIT_TOKENS {S.SPLIT_TOKENS}\n" in text
    for N in (1, 2, 7, 64, 300):
        for H, P, D in ((1, 64, 64), (4, 128, 128), (12, 128, 128), (64, 64, 128)):
            for packed in (0, 1):
                for T in (0, N, S.SPLIT_TOKENS * N):
                    assert S.ssm_plan(ssm_problem(N=N, T=T, H=H, G=1, P=P, S_=D, packed=packed)) == 0
    assert S.ssm_plan(ssm_problem(N=1, T=129, H=1, G=1, P=64, S_=64, piece=64)) == 64
