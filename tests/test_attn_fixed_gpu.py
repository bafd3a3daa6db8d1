"""Long prompts of one length, a batch with its own dimension, as columns of wider rows: the same outputs as
the packed batch has, and those of the definition in 64 bits at rows here and there."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import attn, offsets, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,H,KV", [(2, 1100, 2, 1), (3, 4097, 4, 2), (40, 1030, 2, 2), (1, 9000, 3, 3)])
def test_long_prompts_of_one_length(B, T, H, KV, D):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(B * T)
    rows = rand(g, B, T, (H + 2 * KV) * D + 16, scale=1.2)
    cut = lambda x, a, n: x[..., a * D:(a + n) * D].unflatten(-1, (n, D))
    parts = lambda x: (cut(x, 0, H), cut(x, H, KV), cut(x, H + KV, KV))
    d = rows.cuda()
    out, lse = attn().prefill(*parts(d), return_lse=True)
    packed, packed_lse = attn().prefill(*parts(d.flatten(0, 1)), cu_seqlens=offsets([T] * B).cuda(), return_lse=True)
    assert torch.equal(out.flatten(0, 1), packed) and torch.equal(lse.flatten(0, 1), packed_lse)
    q, k, v = parts(rows)
    at = torch.tensor(sorted({0, 31, 32, 127, 128, T // 2, T - 65, T - 1}))
    seen = torch.arange(T)[None] <= at[:, None]
    for b in {0, B // 2, B - 1}:
        for h in range(H):
            ref, lse_ref, mag, terms = R.attend(q[b, at, h], k[b, :, h * KV // H], v[b, :, h * KV // H], seen, D ** -0.5)
            R.assert_out(out[b, at, h].cpu(), ref, mag)
            R.assert_lse(lse[b, at, h].cpu(), lse_ref, terms, D)
