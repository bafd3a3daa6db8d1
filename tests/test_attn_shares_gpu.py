"""A value that is no number reaches every row that sees it, whatever its weight: also where the
waves of a workgroup, or the pieces of a cut context, have shared the keys out and one share's
scores are so far below the others' that its weight is zero."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, E4M3, attn, offsets, rand, to_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def lines(g, L, D, tops):
    """Keys, values and a scale with which a query of 16 along the first column scores 256 at the
    positions `tops` and 0 elsewhere (all exact in bf16 and e4m3)."""
    k = torch.zeros(L, 1, D)
    k[tops, 0, 0] = 128.0
    return k, rand(g, L, 1, D, scale=2.0).to(E4M3).float(), 0.125


# T tokens of H heads, and how long the context is: in a whole context four waves share the keys
# (up to 32 rows), a longer one is cut; the value at `at` is in another wave's or piece's share than `tops`
CASES = [(1, 4, 64, 3, [40]), (1, 4, 64, 40, [3]), (4, 4, 700, 650, [5, 6]), (1, 4, 6000, 3000, [10, 5900]),
         (1, 4, 6000, 10, [5900]), (1, 4, 6000, 5900, [10]), (20, 4, 6000, 3000, [10, 5900]), (20, 4, 6000, 10, [5900]),
         (20, 4, 6000, 5900, [10]), (1, 1, 60000, 31000, [10])]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,length,at,tops", CASES, ids=str)
def test_over_the_cache(T, H, length, at, tops, D, e4m3):
    g = torch.Generator().manual_seed(length + at)
    size = 64
    pages = -(-(length + T) // size)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    k, v, scale = lines(g, pages * size, D, tops)
    q = torch.zeros(1, T, H, D, dtype=BF)
    q[..., 0] = 16.0
    kind = E4M3 if e4m3 else BF
    paged = lambda x: torch.empty(pages, size, 1, D).index_copy_(0, table[0].long(), x.view(pages, size, 1, D)).to(kind)
    one = torch.ones(1) if e4m3 else None
    ref, lse_ref, mag, terms = R.decode(q, paged(k), paged(v), table, i32(length), scale=scale, k_scale=one, v_scale=one)
    v[at, 0, 7] = NAN
    if not e4m3:
        v[at, 0, 9] = INF
    qd, kd, vd, td, ld, od = to_gpu(q, paged(k), paged(v), table, i32(length), one)
    out, lse = (x.cpu() for x in attn().decode(qd, kd, vd, td, ld, scale=scale, k_scale=od, v_scale=od, return_lse=True))
    bad = [7] if e4m3 else [7, 9]
    assert torch.isnan(out[..., 7]).all() and not torch.isfinite(out[..., bad]).any()
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[..., bad] = False
    R.assert_out(out[keep], ref[keep], mag[keep])
    R.assert_lse(lse, lse_ref, terms, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length,at,tops", [(100, 3, [40]), (1100, 3, [40]), (1100, 40, [3]), (1100, 900, [10])])
def test_over_prompts(length, at, tops, D):
    g = torch.Generator().manual_seed(length + at)
    k, v, scale = lines(g, length, D, tops)
    q = torch.zeros(length, 2, D, dtype=BF)
    q[..., 0] = 16.0
    k, v = k.to(BF), v.to(BF)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, [length], scale=scale)
    v[at, 0, 7], v[at, 0, 9] = NAN, -INF
    out, lse = attn().prefill(*to_gpu(q, k, v), cu_seqlens=offsets([length]).cuda(), scale=scale, return_lse=True)
    out = out.cpu()
    assert torch.isnan(out[at:, :, 7]).all() and not torch.isfinite(out[at:, :, 9]).any()
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[at:, :, 7] = keep[at:, :, 9] = False
    R.assert_out(out[keep], ref[keep], mag[keep])
    R.assert_lse(lse.cpu(), lse_ref, terms, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,length", [(1, 64), (4, 700), (1, 6000), (20, 6000), (1, 60000)])
def test_behind_scores_of_minus_infinity(T, length, D):
    # all weights of a share are zero, and it has no maximum
    g = torch.Generator().manual_seed(length)
    size = 64
    pages = -(-(length + T) // size)
    k, v, q = rand(g, pages * size, 1, D), rand(g, pages * size, 1, D), rand(g, 1, T, 4, D)
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    k[:32, :, 0] = k[length // 4:length // 2, :, 0] = -INF
    at = 3 if length < 1000 else length // 3
    v[at, 0, 7], v[at, 0, 9] = NAN, INF
    table = torch.arange(pages, dtype=torch.int32)[None]
    paged = lambda x: x.view(pages, size, 1, D).cuda()
    out, _ = attn().decode(q.cuda(), paged(k), paged(v), table.cuda(), i32(length).cuda())
    assert torch.isnan(out[..., 7]).all() and not torch.isfinite(out[..., 9]).any()
    out[..., 7] = out[..., 9] = 0
    assert torch.isfinite(out).all()
