"""Attention over the cache takes every batch whose launch has fewer than 2^32 threads, however many
rows of queries it has together."""
import pytest
import torch

import attn_reference as R
from kda_gated_delta_chunked_amd import attn as A
from test_attn_abi import OK, TOO_LARGE, cache, step


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=4096, T=64, H=128, c=cache(KV=8))),              # 2^25 rows, 2^18 workgroups
    (OK, dict(n=(1 << 24) - 1, T=1, H=128, c=cache(KV=1), ws_bytes=1 << 37)),  # 2^31 rows, a workgroup each request
    (OK, dict(n=(1 << 24) - 1, T=1, H=32, c=cache(KV=1))),
    (TOO_LARGE, dict(n=1 << 24, T=1, H=32, c=cache(KV=1))),
    (TOO_LARGE, dict(n=1 << 21, T=64, H=128, c=cache(KV=8))),
    (TOO_LARGE, dict(n=1 << 26, T=64, H=1, c=cache(KV=1)))])  # 2^32 tokens
def test_checks(want, kw):
    over = {x: (1 << 44) + (i << 42) for i, x in enumerate(["q", "kc", "vc", "table", "rows", "lens", "tree"])}
    assert step(**kw, **over, out=1 << 50, lse=1 << 51, ws=1 << 52) == want


@pytest.mark.gpu
def test_many_rows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N, T, H, D, size, W = 1 << 17, 4, 64, 64, 16, 3   # 2^25 rows
    g = torch.Generator().manual_seed(1)
    kc, vc = ((torch.randn(200, size, 1, D, generator=g)).to(torch.bfloat16) for _ in range(2))
    table = torch.randint(0, 200, (N, W), generator=g).to(torch.int32)
    lens = torch.randint(0, W * size - T + 1, (N,), generator=g).to(torch.int32)
    q = torch.empty(N, T, H, D, dtype=torch.bfloat16, device="cuda")
    torch.manual_seed(2)
    for b in range(0, N, 1 << 13):
        q[b:b + (1 << 13)] = torch.randn(1 << 13, T, H, D, device="cuda")
    kd, vd, td, ld = (x.cuda() for x in (kc, vc, table, lens))
    out, lse = A.decode(q, kd, vd, td, ld, return_lse=True)
    at = torch.tensor([0, 1, 65535, 65536, 100000, N - 1])
    ref, lse_ref, mag, terms = R.decode(q[at.cuda()].cpu(), kc, vc, table[at].contiguous(), lens[at])
    R.assert_out(out[at.cuda()].cpu(), ref, mag)
    R.assert_lse(lse[at.cuda()].cpu(), lse_ref, terms, D)
    # a request's outputs are its own, in any batch (short contexts are not cut)
    for b in range(0, N, 1 << 13):
        part, part_lse = A.decode(q[b:b + 999], kd, vd, td[b:b + 999].clone(), ld[b:b + 999].clone(), return_lse=True)
        assert torch.equal(out[b:b + 999], part) and torch.equal(lse[b:b + 999], part_lse)
