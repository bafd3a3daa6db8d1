"""Scores that are infinite: one of minus infinity is a weight of zero, one of plus infinity makes its row NaN."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, E4M3, attn, offsets, rand, to_gpu

pytestmark = pytest.mark.gpu
INF = float("inf")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(g, T, L, D, low, high):
    """Queries, keys, values; a first column that makes the scores of keys `low` minus infinity, of `high` plus
    infinity, and adds nothing to others."""
    q, k, v = rand(g, T, 2, D), rand(g, L, 1, D), rand(g, L, 1, D)
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    k[low, :, 0], k[high, :, 0] = -INF, INF
    return q, k, v


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [100, 1200])
@pytest.mark.parametrize("low", [[0], [0, 1, 31, 32, 64], list(range(0, 80)), list(range(5, 100, 2))], ids=lambda x: f"{len(x)}from{x[0]}")
def test_prompts(low, length, D):
    g = torch.Generator().manual_seed(length + len(low))
    q, k, v = case(g, length, length, D, low, [90])
    out, lse = (x.cpu() for x in attn().prefill(*to_gpu(q, k, v), cu_seqlens=offsets([length]).cuda(), return_lse=True))
    k = k.clone()
    k[..., 0] = 0.0
    seen = torch.ones(length, length, dtype=torch.bool).tril()
    seen[:, low] = False
    some = seen.any(1) & (torch.arange(length) < 90)
    for h in range(2):
        ref, lse_ref, mag, terms = R.attend(q[some, h], k[:, 0], v[:, 0], seen[some], D ** -0.5)
        R.assert_out(out[some, h], ref, mag)
        R.assert_lse(lse[some, h], lse_ref, terms, D)
    assert torch.isnan(out[90:]).all() and torch.isnan(lse[90:]).all()
    none = ~seen.any(1)
    assert torch.isnan(out[none]).all() and (lse[none] == -INF).all()  # (zero divided by zero)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,L", [(1, 300), (1, 5000), (20, 300), (20, 5000)])
@pytest.mark.parametrize("high", [False, True])
def test_over_the_cache(T, L, high, D):
    g = torch.Generator().manual_seed(T + L)
    page = 64
    pages = -(-L // page)
    for low in ([0], list(range(0, L - T, 2)), list(range(L))):
        q, k, v = case(g, T, pages * page, D, low, [77] if high else [])
        out, lse = (x.cpu() for x in attn().decode(*to_gpu(q[None], k.view(pages, page, 1, D), v.view(pages, page, 1, D),
                                                          torch.arange(pages, dtype=torch.int32)[None], i32(L - T)), return_lse=True))
        k = k.clone()
        k[..., 0] = 0.0
        seen = torch.ones(T, L, dtype=torch.bool).tril(L - T)
        seen[:, low] = False
        if high:
            assert torch.isnan(out).all() and torch.isnan(lse).all()
            continue
        for h in range(2):
            ref, lse_ref, mag, terms = R.attend(q[:, h], k[:L, 0], v[:L, 0], seen, D ** -0.5)
            assert torch.isfinite(out[0, :, h]).all()  # (zeros where all weights are)
            off = (out[0, :, h].double() - ref).abs()
            assert (off <= R.STEP * (mag + ref.abs()) * (1 + 2 ** -6) + 1e-30).all()
            R.assert_lse(lse[0, :, h], lse_ref, terms, D)
