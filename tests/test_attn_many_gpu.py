"""Thousands of requests over the cache, every one of them against the definition in 64 bits."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import attn, cache_of, rand, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def short(q, kc, vc, table, lens, most, ks, vs):
    """Of requests with fewer than `most` tokens in all: outputs, logarithms, magnitudes and terms, chains of drafts."""
    N, T, H, D = q.shape
    size, KV = kc.shape[1:3]
    pos = torch.arange(most)
    page = table[:, pos // size].long()
    k, v = (c.double()[page, pos % size] for c in (kc, vc))              # [N, most, KV, D]
    if ks is not None:
        k, v = k * ks.double()[:, None], v * vs.double()[:, None]
    seen = pos[None, None] <= lens[:, None, None] + torch.arange(T)[None, :, None]
    k, v = (x.repeat_interleave(H // KV, 2).permute(0, 2, 1, 3) for x in (k, v))  # [N, H, most, D]
    x = q.double().permute(0, 2, 1, 3) * D ** -0.5                        # [N, H, T, D]
    s = (x @ k.transpose(-1, -2).contiguous()).masked_fill(~seen[:, None], -float("inf"))
    p = torch.softmax(s, -1)
    terms = (x.abs() @ k.abs().transpose(-1, -2).contiguous()).masked_fill(~seen[:, None], 0).amax(-1)
    back = lambda t: t.transpose(1, 2)
    return back(p @ v), back(torch.logsumexp(s, -1)), back(p @ v.abs()), back(terms)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N,T,W", [(20000, 1, 70), (20000, 1, 4), (900, 40, 70), (3000, 8, 70), (2500, 33, 6)])
def test_all_of_them(N, T, W, e4m3):
    # wide tables are cut into stretches, many requests each, narrow ones not
    g = torch.Generator().manual_seed(N + T)
    size, H, KV, D = 16, 2, 1, 64
    lens = torch.randint(0, 9, (N,), generator=g).to(torch.int32)
    long = {} if W < 70 else {3: 1000, N // 2: 300, N - 1: 900}
    for n, x in long.items():
        lens[n] = x
    kc, vc, ks, vs = cache_of(g, 200, size, KV, D, e4m3)
    table = torch.randint(0, 200, (N, W), generator=g).to(torch.int32)
    q = rand(g, N, T, H, D, scale=1.4)
    qd, kd, vd, td, ld, ksd, vsd = to_gpu(q, kc, vc, table, lens, ks, vs)
    out, lse = (x.cpu() for x in attn().decode(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd, return_lse=True))
    most = 8 + T
    for b in range(0, N, 2000):
        at = torch.tensor([n for n in range(b, min(b + 2000, N)) if n not in long])
        ref, lse_ref, mag, terms = short(q[at], kc, vc, table[at], lens[at], most, ks, vs)
        R.assert_out(out[at], ref, mag)
        R.assert_lse(lse[at], lse_ref, terms, D)
    if long:
        at = torch.tensor(sorted(long))
        ref, lse_ref, mag, terms = R.decode(q[at], kc, vc, table[at].contiguous(), lens[at], k_scale=ks, v_scale=vs)
        R.assert_out(out[at], ref, mag)
        R.assert_lse(lse[at], lse_ref, terms, D)
