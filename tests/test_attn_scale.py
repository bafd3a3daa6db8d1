"""The largest and the smallest scales of scores: those whose product with log2 e, of which the weights
are exponentials, leaves fp32 are refused, the others work."""
import pytest
import torch

import attn_reference as R
from test_attn_abi import INVALID, OK, prompt, step


@pytest.mark.parametrize("want,scale", [(OK, 1e-45), (OK, 2.0 ** -126), (OK, 2.0 ** 126), (OK, 2.0 ** 127), (INVALID, 2.4e38),
                                        (INVALID, 3.4e38)])
def test_checks(want, scale):
    assert prompt(scale=scale) == want
    assert step(scale=scale) == want


@pytest.mark.gpu
@pytest.mark.parametrize("scale,size", [(2.0 ** 126, 2.0 ** -62), (2.0 ** 127, 2.0 ** -64), (2.0 ** -126, 2.0 ** 62),
                                        (2.0 ** -126, 2.0 ** 58), (2.0 ** -126, 1.0)])
def test_scales(scale, size):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from kda_gated_delta_chunked_amd import attn
    g = torch.Generator().manual_seed(3)
    L, D = 200, 64
    q, k, v = (torch.randn(L, h, D, generator=g).to(torch.bfloat16) for h in (2, 1, 1))
    q, k = q * size, k * size
    ref, lse_ref, mag, terms = R.prefill(q, k, v, [L], scale=scale)
    ok = terms / scale < 2.0 ** 127  # (rows that see larger q . k have no defined output)
    assert ok.all() or size == 2.0 ** 62
    out, lse = attn.prefill(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=scale, return_lse=True)
    if ok.any():
        R.assert_out(out[0].cpu()[ok], ref[ok], mag[ok])
        R.assert_lse(lse[0].cpu()[ok], lse_ref[ok], terms[ok], D)
    # the last one's outputs over a cache
    ok = ok[-1:]
    table = torch.arange(13, dtype=torch.int32)[None]
    paged = lambda x: torch.cat([x, x.new_zeros(8, 1, D)]).view(13, 16, 1, D).cuda()
    out, lse = attn.decode(q[None, -1:].cuda(), paged(k), paged(v), table.cuda(), torch.tensor([L - 1], dtype=torch.int32).cuda(),
                           scale=scale, return_lse=True)
    if ok.any():
        R.assert_out(out[0].cpu()[ok], ref[-1:][ok], mag[-1:][ok])
        R.assert_lse(lse[0].cpu()[ok], lse_ref[-1:][ok], terms[-1:][ok], D)
