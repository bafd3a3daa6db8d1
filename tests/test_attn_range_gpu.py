"""Values near either end of bf16's range: outputs are weighted means of values, so what is summed on
the way to them may not leave fp32's range where they do not.

Bounds.  As tests/attn_reference.py, which counts the roundings relative to the values; at the
lower end what falls below fp32's normal numbers (2^-126) may be lost.  Sums are held 2^-31 as
large as weights of at most 1 make them, so that is an output's error of L 2^-95 at most over L
positions."""
import math

import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, E4M3, attn, cache_of, offsets, pages_for, rand, to_gpu

pytestmark = pytest.mark.gpu
i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
dims = pytest.mark.parametrize("D", [64, 128])


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(g, rise, T, L, D, H=2):
    """Queries [T, H, D], keys and values [L, 1, D] and a scale: scores of 8 at a key of every 64
    behind the first 64 and of 0 at others, all of 0, or of randoms."""
    q, k = torch.zeros(T, H, D), torch.zeros(L, 1, D)
    v = torch.where(torch.rand(L, 1, D, generator=g) < 0.3, -1.0, 1.0) * (1 + torch.rand(L, 1, D, generator=g)) / 2
    if rise == "random":
        return rand(g, T, H, D, scale=1.4), rand(g, L, 1, D, scale=1.4), v, D ** -0.5
    q[..., 0] = 16.0
    if rise == "rising":
        k[100::64, 0, 0] = 4.0
    return q.to(BF), k.to(BF), v, 0.125


def check(out, lse, ref, floor):
    want, lse_ref, mag, terms = ref
    out = out.cpu().double()
    assert torch.isfinite(out).all()
    off = (out - want).abs()
    assert (off <= R.STEP * (mag + want.abs()) * (1 + 2 ** -6) + floor).all()
    R.assert_lse(lse.cpu(), lse_ref, terms, 128)


def floor_of(L):
    return L * 2.0 ** -95


SIZES = [(2.0 ** 127, "rising"), (2.0 ** 127, "equal"), (2.0 ** 127, "random"), (2.0 ** 115, "rising"), (2.0 ** -60, "rising"),
         (2.0 ** -60, "random")]
sizes = pytest.mark.parametrize("size,rise", SIZES, ids=lambda x: x if isinstance(x, str) else f"2^{int(math.log2(x))}")


@sizes
@dims
@pytest.mark.parametrize("lens", [[40], [300, 33], [1500]], ids=str)
def test_prompts(lens, D, size, rise):
    g = torch.Generator().manual_seed(sum(lens))
    T = sum(lens)
    q, k, v, scale = case(g, rise, T, T, D)
    v = (v * size).to(BF)
    out, lse = attn().prefill(*to_gpu(q, k, v), cu_seqlens=offsets(lens).cuda(), scale=scale, return_lse=True)
    check(out, lse, R.prefill(q, k, v, lens, scale=scale), floor_of(T))


@sizes
@dims
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,L", [(1, 300), (1, 9000), (20, 300), (20, 5000)])
def test_over_the_cache(T, L, e4m3, D, size, rise):
    g = torch.Generator().manual_seed(T + L)
    page = 64
    pages = -(-L // page)
    q, k, v, scale = case(g, rise, T, pages * page, D)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    kind = E4M3 if e4m3 else BF
    paged = lambda x: torch.empty(pages, page, 1, D).index_copy_(0, table[0].long(), x.float().view(pages, page, 1, D))
    kc = paged(k).to(kind)
    vc = (paged(v) * 256).to(kind) if e4m3 else paged(v * size).to(kind)
    ks, vs = (torch.ones(1), torch.tensor([size / 256])) if e4m3 else (None, None)
    lens = i32(L - T)
    ref = R.decode(q[None], kc, vc, table, lens, scale=scale, k_scale=ks, v_scale=vs)
    qd, kd, vd, td, ld, ksd, vsd = to_gpu(q[None], kc, vc, table, lens, ks, vs)
    out, lse = attn().decode(qd, kd, vd, td, ld, scale=scale, k_scale=ksd, v_scale=vsd, return_lse=True)
    check(out, lse, ref, floor_of(pages * page))


def test_several_requests_of_large_values():
    # pieces of several contexts, empty slots and absent pages among them
    g = torch.Generator().manual_seed(2)
    lens, page, D = [3000, 5, 0, 7000], 64, 64
    table, rows, pages = pages_for(g, [x + 3 for x in lens], page)
    kc, vc, _, _ = cache_of(g, pages, page, 2, D, False)
    vc = (vc.float().clamp(-4, 4) * 2.0 ** 125).to(BF)
    table[rows[0], 7:9] = -1
    rows[1] = -1
    q = rand(g, 4, 3, 4, D, scale=1.4)
    ref = R.decode(q, kc, vc, table, i32(*lens), rows)
    qd, kd, vd, td, ld, rd = to_gpu(q, kc, vc, table, i32(*lens), rows)
    out, lse = attn().decode(qd, kd, vd, td, ld, rows=rd, return_lse=True)
    check(out, lse, ref, floor_of(8192))
