"""What no row can see costs next to nothing, also where it is NaN: rows of a page behind a request's end, as an
allocation or an earlier request has left them, and what is read in the place of absent pages; later tokens of
a prompt, which are NaN in a padded batch, cost little more."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, E4M3, attn, cache_of, pages_for, rand, to_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def microseconds(call, n=5):
    call()
    best = float("inf")
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1e3)
    return best


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,H,KV", [(1, 32, 8), (32, 32, 4)])
def test_rest_of_a_page(T, H, KV, e4m3):
    # (looked over one by one, contexts like these took 22 and 35 times as long)
    g = torch.Generator().manual_seed(T)
    N, size, W, D = 32, 64, 128, 128
    lens = torch.randint(1, W * size - T, (N,), generator=g).to(torch.int32)
    table = torch.randperm(N * W, generator=g).view(N, W).to(torch.int32)
    kind = E4M3 if e4m3 else BF
    kd, vd = (torch.randn(N * W, size, KV, D, device="cuda").to(kind) for _ in range(2))
    q, ld, td = rand(g, N, T, H, D).cuda(), lens.cuda(), table.cuda()
    one = dict(k_scale=torch.ones(KV).cuda(), v_scale=torch.ones(KV).cuda()) if e4m3 else {}
    run = lambda: attn().decode(q, kd, vd, td, ld, **one)
    clean, us = run()[0].clone(), microseconds(run)
    pos = torch.arange(W * size)[None]
    slots = (table.long().repeat_interleave(size, 1) * size + pos % size)[pos >= lens[:, None] + T].cuda()
    for c in (kd, vd):
        c.view(torch.uint8).view(N * W * size, -1)[slots] = 0x7f if e4m3 else 0xff
    assert torch.equal(run()[0], clean)
    assert microseconds(run) <= 2 * us + 20


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,H", [(1, 4), (20, 4)])
@pytest.mark.parametrize("N", [1, 2, 3])
def test_tiles_with_rows_that_are_not_there(N, T, H, e4m3):
    # absent pages here and there (page 0, which is read in their place, is NaN), a hidden token, and the page's rest;
    # contexts of more than 64 tiles a wave, values that are seen as well
    g = torch.Generator().manual_seed(T + N)
    size, D, KV = 16, 64, 1
    lens = [9000, 2100, 35000][:N]
    table, rows, pages = pages_for(g, [x + T for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages + 1, size, KV, D, e4m3)
    table[table >= 0] += 1
    vc = vc.float()
    vc[0] = NAN
    for r, n in zip(rows.tolist(), lens):
        table[r, 5::97] = -1
        last = (n + T - 1) // size
        vc[table[r, last], (n + T - 1) % size + 1:] = NAN
    vc = vc.to(E4M3 if e4m3 else BF)
    q = rand(g, N, T, H, D, scale=1.4)
    # (its reference, from a cache in which page 0 is zeros)
    clean = torch.where(torch.isnan(vc.float()), 0.0, vc.float()).to(vc.dtype)
    ref, lse_ref, mag, terms = R.decode(q, kc, clean, table, i32(*lens), rows, k_scale=ks, v_scale=vs)
    seen = 64 * 130 - 3 if lens[0] > 8400 else 70
    page = table[rows[0], seen // size]
    assert page > 0
    vc = vc.float()
    vc[page, seen % size, 0, 7] = NAN
    vc = vc.to(kc.dtype)
    qd, kd, vd, td, ld, rd, ksd, vsd = to_gpu(q, kc, vc, table, i32(*lens), rows, ks, vs)
    out, lse = (x.cpu() for x in attn().decode(qd, kd, vd, td, ld, rows=rd, k_scale=ksd, v_scale=vsd, return_lse=True))
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[0, ..., 7] = False
    assert torch.isnan(out[0, ..., 7]).all()
    R.assert_out(out[keep], ref[keep], mag[keep])
    R.assert_lse(lse, lse_ref, terms, D)


@pytest.mark.parametrize("H,KV,D", [(8, 2, 128), (16, 2, 64)])
def test_a_batch_padded_with_values_that_are_no_numbers(H, KV, D):
    # (looked over one by one, all keys ahead of a padded token, these took 39 and 20 times as long)
    g = torch.Generator().manual_seed(D)
    B, T = 8, 4096
    real = [4096, 3000, 17, 2048, 1, 4000, 1000, 2500]
    q, k, v = (rand(g, B, T, h, D).cuda() for h in (H, KV, KV))
    run = lambda: attn().prefill(q, k, v)
    us = microseconds(run)
    for x in (k, v):
        for b, n in enumerate(real):
            x[b, n:] = NAN
    out = run()[0]
    qc, kc, vc, scale = q.cpu(), k.cpu(), v.cpu(), D ** -0.5
    for b, n in enumerate(real):
        assert torch.isfinite(out[b, :n]).all() and torch.isnan(out[b, n:]).all()
        rows = torch.tensor(sorted({0, n // 3, n // 2, max(0, n - 33), max(0, n - 2), n - 1}))
        seen = torch.arange(n)[None] <= rows[:, None]
        for h in range(H):  # (last bits may differ: rows side by side take their maxima together)
            ref, _, mag, _ = R.attend(qc[b, rows, h], kc[b, :n, h * KV // H], vc[b, :n, h * KV // H], seen, scale)
            R.assert_out(out[b, rows, h].cpu(), ref, mag)
    assert microseconds(run) <= 8 * us + 20
