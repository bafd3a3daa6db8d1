"""Edges of softmax attention over prompts and over the paged cache: what masks hide,
values that are no numbers, far scores, cut contexts, offsets past 32 bits."""
import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, assign_case, attn, cache_of, check_assign, check_decode, offsets, pages_for, rand, to_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


caches = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
dims = pytest.mark.parametrize("D", [64, 128])


# ---------------------------------------------------------------------------
# prompts

def prompts(lens, D, seed, H=4, KV=2, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    return rand(g, T, H, D, scale=scale), rand(g, T, KV, D, scale=scale), rand(g, T, KV, D)


def run_prompts(q, k, v, lens, **kw):
    out, lse = attn().prefill(*to_gpu(q, k, v), cu_seqlens=offsets(lens).cuda(), return_lse=True, **kw)
    return out.cpu(), lse.cpu()


@dims
@pytest.mark.parametrize("at", [0, 31, 32, 63, 64, 100, 127, 128, 200, 299])
def test_a_value_that_is_infinite_is_seen_by_later_rows_only(at, D):
    lens = [300, 40]
    q, k, v = prompts(lens, D, at)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    v[at, 1, 5], v[at, 1, 9] = INF, NAN
    out, lse = run_prompts(q, k, v, lens)
    R.assert_lse(lse, lse_ref, terms, D)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[at:300, 2:, 5] = hit[at:300, 2:, 9] = True
    assert (out[at:300, 2:, 5] == INF).all() and torch.isnan(out[at:300, 2:, 9].float()).all()
    keep = ~hit
    R.assert_out(out[keep], ref[keep], mag[keep])


@dims
@pytest.mark.parametrize("at", [0, 40, 64, 255, 299])
def test_keys_and_queries_that_are_nan(at, D):
    lens = [300, 40]
    q, k, v = prompts(lens, D, at)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    k[at, 0, D - 1] = NAN
    q[at // 2, 3, 0] = NAN
    q[310, 0, 1] = NAN
    out, lse = run_prompts(q, k, v, lens)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool)
    hit[at:300, :2] = hit[at // 2, 3] = hit[310, 0] = True
    assert torch.isnan(out[hit].float()).all() and torch.isnan(lse[hit]).all()
    R.assert_out(out[~hit], ref[~hit], mag[~hit])
    R.assert_lse(lse[~hit], lse_ref[~hit], terms[~hit], D)


@dims
@pytest.mark.parametrize("length", [90, 300])
@pytest.mark.parametrize("slope", [1e-3, 0.3, -0.3, 30.0, -30.0])
def test_scores_that_rise_and_fall_along_the_keys(slope, length, D):
    # the keys lie along one direction, more and more of it
    g = torch.Generator().manual_seed(length)
    u = torch.randn(D, generator=g)
    k = (torch.arange(length)[:, None, None] * u * slope / (u @ u) ** 0.5 + torch.randn(length, 1, D, generator=g) * 0.1).to(BF)
    q = (u / (u @ u) ** 0.5 * torch.tensor([1.0, -1.0, 3.0])[None, :, None] + torch.zeros(length, 3, D)).to(BF)
    v = rand(g, length, 1, D)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, [length], scale=1.0)
    out, lse = run_prompts(q, k, v, [length], scale=1.0)
    # an exponent off by d makes a weight off by d of it, the outputs by 2 d mag: scores up to 3 slope length
    d = (D + 8) * 2.0 ** -24 * terms[..., None]
    off = (out.double() - ref).abs()
    assert (off <= (R.STEP * (1 + 2 ** -6) + 2 * d) * (mag + ref.abs()) + 1e-30).all()
    R.assert_lse(lse, lse_ref, terms, D)


@dims
def test_scores_far_apart_take_one_value(D):
    lens = [200, 130]
    q, k, v = prompts(lens, D, 3, scale=1e9)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    out, lse = run_prompts(q, k, v, lens)
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, D)


@dims
def test_keys_of_the_lowest_value(D):
    # scores of -1e38 and so on are numbers, not masks
    lens = [70]
    q, k, v = prompts(lens, D, 4)
    q[:] = 0
    q[..., 0] = 1.0
    k[:] = 0
    k[:, :, 0] = torch.finfo(BF).min
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens, scale=0.5)
    out, lse = run_prompts(q, k, v, lens, scale=0.5)
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, D)


def test_a_batch_padded_with_short_sequences_and_one_long():
    lens = [1] * 130 + [777] + [0] * 50 + [2, 3]
    q, k, v = prompts(lens, 64, 6, H=2, KV=1)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    out, lse = run_prompts(q, k, v, lens)
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, 64)


# Few workgroups of long rows: two sides of one share a row's keys.

@dims
@pytest.mark.parametrize("H,KV,lens", [(2, 1, [1024]), (3, 3, [1, 2047]), (2, 2, [1301, 0, 1900]), (1, 1, [4200])], ids=str)
def test_long_rows(H, KV, lens, D):
    q, k, v = prompts(lens, D, sum(lens), H=H, KV=KV, scale=1.4)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    out, lse = run_prompts(q, k, v, lens)
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, D)


@dims
@pytest.mark.parametrize("at", [0, 33, 1000, 1099])
def test_long_rows_with_values_and_keys_that_are_no_numbers(at, D):
    lens = [1100]
    q, k, v = prompts(lens, D, at, H=2, KV=1)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    bad = v.clone()
    bad[at, 0, 3], bad[at, 0, 7] = -INF, NAN
    out, lse = run_prompts(q, k, bad, lens)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[at:, :, 3] = hit[at:, :, 7] = True
    assert (out[at:, :, 3] == -INF).all() and torch.isnan(out[at:, :, 7].float()).all()
    R.assert_out(out[~hit], ref[~hit], mag[~hit])
    R.assert_lse(lse, lse_ref, terms, D)
    k[at, 0, D - 1] = NAN
    out, lse = run_prompts(q, k, v, lens)
    assert torch.isnan(out[at:].float()).all() and torch.isnan(lse[at:]).all()
    if at:
        R.assert_out(out[:at], ref[:at], mag[:at])
        R.assert_lse(lse[:at], lse_ref[:at], terms[:at], D)


@dims
def test_long_rows_with_scores_far_apart(D):
    q, k, v = prompts([1200], D, 3, H=2, KV=1, scale=1e9)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, [1200])
    out, lse = run_prompts(q, k, v, [1200])
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, D)


# ---------------------------------------------------------------------------
# the cache

@caches
@dims
@pytest.mark.parametrize("T,H", [(1, 4), (5, 4), (20, 4)])
def test_what_no_token_sees_may_hold_anything(T, H, D, e4m3):
    g = torch.Generator().manual_seed(T + D)
    size, lens = 16, [0, 7, 16, 130, 259]
    table, rows, pages = pages_for(g, [x + T for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages, size, 2, D, e4m3)
    kc, vc = kc.float(), vc.float()
    used = torch.zeros(pages, size, dtype=torch.bool)
    for r, n in zip(rows.tolist(), lens):
        for x in range(n + T):
            used[table[r, x // size], x % size] = True
    kc[~used], vc[~used] = NAN, NAN if e4m3 else INF
    words = torch.full((T,), -1, dtype=torch.int64)
    if T > 2:  # the request's token 1 is seen by itself alone
        words[:] = ~2
        words[1] = 2
        for r, n in zip(rows.tolist(), lens):
            vc[table[r, (n + 1) // size], (n + 1) % size, :, 3] = NAN
    kc, vc = kc.to(torch.float8_e4m3fn if e4m3 else BF), vc.to(torch.float8_e4m3fn if e4m3 else BF)
    q = rand(g, len(lens), T, H, D)
    clean = torch.where(torch.isnan(vc.float()), 0.0, vc.float()).to(vc.dtype)
    ref, lse_ref, mag, terms = R.decode(q, kc, clean, table, i32(*lens), rows, words, k_scale=ks, v_scale=vs)
    qd, kd, vd, td, ld, rd, wd, ksd, vsd = to_gpu(q, kc, vc, table, i32(*lens), rows, words, ks, vs)
    out, lse = (x.cpu() for x in attn().decode(qd, kd, vd, td, ld, rows=rd, tree=wd, k_scale=ksd, v_scale=vsd, return_lse=True))
    keep = torch.ones(out.shape, dtype=torch.bool)
    if T > 2:
        assert torch.isnan(out[:, 1, :, 3].float()).all()
        keep[:, 1, :, 3] = False
    R.assert_out(out[keep], ref[keep], mag[keep])
    R.assert_lse(lse, lse_ref, terms, D)


@caches
def test_rows_without_a_key(e4m3):
    # empty contexts and a tree that hides all: zeros and -inf, whatever is in the page
    g = torch.Generator().manual_seed(2)
    table, rows, pages = pages_for(g, [3, 43], 16)
    kc, vc, ks, vs = cache_of(g, pages, 16, 2, 64, e4m3)
    vc = vc.float().fill_(NAN).to(vc.dtype)
    words = torch.zeros(2, 3, dtype=torch.int64)
    qd, kd, vd, td, ld, rd, wd, ksd, vsd = to_gpu(rand(g, 2, 3, 4, 64), kc, vc, table, i32(0, 40), rows, words, ks, vs)
    out, lse = attn().decode(qd, kd, vd, td, ld, rows=rd, tree=wd, k_scale=ksd, v_scale=vsd, return_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -INF).all()
    assert torch.isnan(out[1]).all() and torch.isfinite(lse[1]).all()


@caches
@dims
@pytest.mark.parametrize("T,H,KV", [(1, 2, 1), (3, 8, 2), (9, 8, 1), (40, 8, 2)])
@pytest.mark.parametrize("lens", [[5000], [3000, 5, 0, 7000], [0] * 9 + [2500, 128, 127, 129, 1] * 3], ids=["one", "four", "more"])
def test_cut_contexts(lens, T, H, KV, D, e4m3):
    if T * len(lens) > 160:
        lens = lens[:5] + lens[-6:]
    g = torch.Generator().manual_seed(T + len(lens))
    size = 64
    table, rows, pages = pages_for(g, [x + T for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages, size, KV, D, e4m3)
    rows[len(lens) // 2] = -1 if len(lens) > 3 else rows[len(lens) // 2]
    if len(lens) > 1:
        table[rows[0], 7:9] = -1
    q = rand(g, len(lens), T, H, D, scale=1.4)
    out, lse = check_decode(q, kc, vc, table, i32(*lens), rows, None, ks, vs)
    again = attn().decode(*to_gpu(q, kc, vc, table, i32(*lens)), rows=rows.cuda(), return_lse=True,
                          **({} if ks is None else dict(k_scale=ks.cuda(), v_scale=vs.cuda())))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # (no sum in the order of arrival)


@caches
@dims
@pytest.mark.parametrize("T,H,KV,lens", [(64, 12, 2, [0, 33]), (50, 9, 3, [100, 1, 64, 5]), (64, 4, 1, [2000, 100]), (2, 128, 1, [40, 300])],
                         ids=str)
def test_more_rows_than_a_workgroup_takes(T, H, KV, lens, D, e4m3):
    g = torch.Generator().manual_seed(T * H)
    table, rows, pages = pages_for(g, [x + T for x in lens], 32)
    kc, vc, ks, vs = cache_of(g, pages, 32, KV, D, e4m3)
    words = torch.randint(-2 ** 62, 2 ** 62, (len(lens), T), generator=g) if T > 2 else None
    check_decode(rand(g, len(lens), T, H, D, scale=1.4), kc, vc, table, i32(*lens), rows, words, ks, vs)


@caches
@pytest.mark.parametrize("T", [1, 12])
def test_more_requests_than_threads_cut(T, e4m3):
    g = torch.Generator().manual_seed(T)
    lens = torch.randint(0, 40, (300,), generator=g).tolist()
    lens[17], lens[255], lens[256], lens[299] = 1900, 700, 0, 1100
    if T > 1:
        lens = lens[:18] + lens[250:258]
    table, rows, pages = pages_for(g, [x + T for x in lens], 16)
    kc, vc, ks, vs = cache_of(g, pages, 16, 1, 64, e4m3)
    check_decode(rand(g, len(lens), T, 4, 64), kc, vc, table, i32(*lens), rows, None, ks, vs)


@caches
@pytest.mark.parametrize("T", [1, 20])
def test_cut_contexts_with_values_that_are_no_numbers(T, e4m3):
    g = torch.Generator().manual_seed(T)
    lens, size, D = [6000, 100], 32, 64
    table, rows, pages = pages_for(g, [x + T for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages, size, 1, D, e4m3)
    ref, lse_ref, mag, terms = R.decode(q := rand(g, 2, T, 4, D), kc, vc, table, i32(*lens), rows, k_scale=ks, v_scale=vs)
    vc = vc.float()
    vc[table[rows[0], 3000 // size], 3000 % size, 0, 7] = NAN
    vc = vc.to(kc.dtype)
    qd, kd, vd, td, ld, rd, ksd, vsd = to_gpu(q, kc, vc, table, i32(*lens), rows, ks, vs)
    out, lse = (x.cpu() for x in attn().decode(qd, kd, vd, td, ld, rows=rd, k_scale=ksd, v_scale=vsd, return_lse=True))
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[0, ..., 7] = False
    assert torch.isnan(out[0, ..., 7].float()).all()
    R.assert_out(out[keep], ref[keep], mag[keep])
    R.assert_lse(lse, lse_ref, terms, D)
    kc = kc.float()
    kc[table[rows[0], 3000 // size], 3000 % size, 0, 7] = NAN  # a piece whose sum is none
    out, lse = (x.cpu() for x in attn().decode(qd, kc.to(vc.dtype).cuda(), vd, td, ld, rows=rd, k_scale=ksd, v_scale=vsd,
                                               return_lse=True))
    assert torch.isnan(out[0].float()).all() and torch.isnan(lse[0]).all()
    R.assert_out(out[1], ref[1], mag[1])


@caches
def test_far_scores_over_the_cache(e4m3):
    g = torch.Generator().manual_seed(5)
    lens = [1500, 33]
    table, rows, pages = pages_for(g, [x + 2 for x in lens], 64)
    kc, vc, ks, vs = cache_of(g, pages, 64, 2, 128, e4m3)
    if e4m3:
        ks = ks * 1e12
    else:
        kc = (kc.float() * 1e9).to(BF)
    check_decode(rand(g, 2, 2, 4, 128, scale=1e9), kc, vc, table, i32(*lens), rows, None, ks, vs)


def test_lengths_beyond_the_table_and_a_shared_row():
    g = torch.Generator().manual_seed(8)
    table, _, pages = pages_for(g, [48, 40, 9], 16)
    kc, vc, _, _ = cache_of(g, pages, 16, 1, 64, False)
    lens = i32(2 ** 31 - 1, 2 ** 31 - 60, 20, 31)
    check_decode(rand(g, 4, 5, 2, 64), kc, vc, table, lens, i32(0, 1, 2, 2))


@caches
@pytest.mark.parametrize("T", [1, 9])
def test_a_cache_of_more_than_32_bits(T, e4m3):
    size, KV, D, H = 64, 8, 128, 8 if T == 1 else 64
    pages = (2 ** 32 // (size * KV * D)) + 70
    dtype = torch.float8_e4m3fn if e4m3 else BF
    both = torch.empty(pages, 2, size, KV, D, dtype=dtype, device="cuda")  # elements past 2^33, bytes past 2^34
    kd, vd = both.unbind(1)
    g = torch.Generator().manual_seed(3)
    length = 300
    ids = torch.tensor([0, pages - 1, pages // 2 + 1, 5, pages - 30][:-(-(length + T) // size)], dtype=torch.int32)
    kc, vc, ks, vs = cache_of(g, len(ids), size, KV, D, e4m3)
    kd[ids.long().cuda()], vd[ids.long().cuda()] = kc.cuda(), vc.cuda()
    q = rand(g, 1, T, H, D)
    local = torch.arange(len(ids), dtype=torch.int32)[None]
    ref, lse_ref, mag, terms = R.decode(q, kc, vc, local, i32(length), k_scale=ks, v_scale=vs)
    qd, td, ld, ksd, vsd = to_gpu(q, ids[None], i32(length), ks, vs)
    out, lse = attn().decode(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd, return_lse=True)
    R.assert_out(out.cpu(), ref, mag)
    R.assert_lse(lse.cpu(), lse_ref, terms, D)
    # stored into as well
    slots = torch.tensor([pages * size - 1, pages * size, -1, (pages // 2 + 1) * size + 3, 7], device="cuda")
    k, v = rand(g, 5, KV, D).cuda(), rand(g, 5, KV, D).cuda()
    before = both[5].clone()
    attn().store(k, v, kd, vd, slots, k_scale=ksd, v_scale=vsd)
    for i, (p, x) in [(0, (pages - 1, size - 1)), (3, (pages // 2 + 1, 3)), (4, (0, 7))]:
        for c, t, s in ((kd, k, ksd), (vd, v, vsd)):
            want = t[i] if s is None else (t[i].float() / s[:, None]).clamp(-448, 448).to(dtype)
            assert torch.equal(c[p, x].view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(both[5].view(torch.uint8), before.view(torch.uint8))


# ---------------------------------------------------------------------------
# many of everything

def test_thousands_of_prompts():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 4, (3000,), generator=g).tolist()
    lens[1234] = 150
    q, k, v = prompts(lens, 64, 4, H=2, KV=1)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    out, lse = run_prompts(q, k, v, lens)
    R.assert_out(out, ref, mag)
    R.assert_lse(lse, lse_ref, terms, 64)


@caches
@pytest.mark.parametrize("T", [1, 40])
def test_thousands_of_requests(T, e4m3):
    g = torch.Generator().manual_seed(T)
    N, size, W = 20000 if T == 1 else 900, 16, 70
    lens = torch.randint(0, 5, (N,), generator=g).to(torch.int32)
    some = [0, 1, 255, 256, 700, N // 2, N - 2, N - 1]
    lens[some[3]], lens[some[5]], lens[N - 1] = 1000, 300, 900
    kc, vc, ks, vs = cache_of(g, 200, size, 1, 64, e4m3)
    table = torch.randint(0, 200, (N, W), generator=g).to(torch.int32)
    q = rand(g, N, T, 2, 64, scale=1.4)
    qd, kd, vd, td, ld, ksd, vsd = to_gpu(q, kc, vc, table, lens, ks, vs)
    out, lse = attn().decode(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd, return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    at = torch.tensor(some)
    ref, lse_ref, mag, terms = R.decode(q[at], kc, vc, table[at].contiguous(), lens[at], k_scale=ks, v_scale=vs)
    R.assert_out(out.cpu()[at], ref, mag)
    R.assert_lse(lse.cpu()[at], lse_ref, terms, 64)
    # and all of them against the same requests, a hundred at a time
    for b in range(0, N, 4000):
        part, _ = attn().decode(qd[b:b + 100], kd, vd, td[b:b + 100], ld[b:b + 100], k_scale=ksd, v_scale=vsd)
        assert (out[b:b + 100].float() - part.float()).abs().max() <= 2 * R.STEP * 2 * vc.float().abs().max() * (1 if vs is None else vs.max())


@caches
@pytest.mark.parametrize("KV,size,length", [(128, 16, 1500), (2, 1024, 3000), (200, 64, 1200)])
def test_many_heads_and_large_pages(KV, size, length, e4m3):
    g = torch.Generator().manual_seed(KV)
    lens = [length, 20]
    table, rows, pages = pages_for(g, [x + 1 for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages, size, KV, 64, e4m3)
    check_decode(rand(g, 2, 1, KV, 64, scale=1.4), kc, vc, table, i32(*lens), rows, None, ks, vs)


def test_thousands_of_requests_get_pages():
    g = torch.Generator().manual_seed(6)
    old, rows, cu, table, free = assign_case(g, 5000, 60, 5, 16)
    rows[::7] = -1
    check_assign(old, rows, cu, table, free, 0, 16, int(cu[-1]) + 300)


# ---------------------------------------------------------------------------
# refusals of the binding

def test_refusals():
    A = attn()
    e = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")
    f8, f32, it = torch.float8_e4m3fn, torch.float32, torch.int32
    q, c, t, n = e(2, 1, 4, 64), e(3, 16, 2, 64), e(2, 4, dtype=it), e(2, dtype=it)
    with pytest.raises(ValueError, match="on a cuda"):
        A.prefill(q[0].cpu(), q[0].cpu(), q[0].cpu())
    with pytest.raises(TypeError, match="k must be"):
        A.prefill(q, q.float(), q)
    with pytest.raises(ValueError, match="v must have shape"):
        A.prefill(q, q, q[:, :, :2])
    with pytest.raises(ValueError, match="k and v must be"):
        A.prefill(q, q[0], q[0])
    with pytest.raises(Exception, match="kda_attn_prefill"):
        A.prefill(e(4, 3, 64), e(4, 2, 64), e(4, 2, 64))  # 2 does not divide 3
    with pytest.raises(Exception, match="kda_attn_prefill"):
        A.prefill(e(4, 2, 96), e(4, 2, 96), e(4, 2, 96))
    with pytest.raises(ValueError, match="same strides"):
        A.decode(q, c, e(3, 16, 4, 64)[:, :, :2], t, n)
    with pytest.raises(ValueError, match="last 2 dimensions"):
        A.decode(q, e(3, 16, 64, 2).transpose(2, 3), c, t, n)
    with pytest.raises(TypeError, match="bfloat16 or float8"):
        A.decode(q, c.half(), c.half(), t, n)
    with pytest.raises(ValueError, match="needs k_scale"):
        A.decode(q, c.to(f8), c.to(f8), t, n)
    with pytest.raises(ValueError, match="v_scale is for"):
        A.store(c[0], c[0], c, c.clone(), e(16, dtype=torch.int64), v_scale=e(2, dtype=f32))
    with pytest.raises(ValueError, match="heads of 64, q of 128"):
        A.decode(e(2, 1, 4, 128), c, c, t, n)
    with pytest.raises(TypeError, match="table must be"):
        A.decode(q, c, c, t.long(), n)
    with pytest.raises(ValueError, match="lens must have shape"):
        A.decode(q, c, c, t, e(3, dtype=it))
    with pytest.raises(TypeError, match="tree must be"):
        A.decode(q, c, c, t, n, tree=n)
    with pytest.raises(Exception, match="kda_attn_decode"):
        A.decode(e(2, 65, 4, 64), c, c, t, n)
    with pytest.raises(Exception, match="kda_attn_decode"):
        A.decode(q, c, c, e(2, 4096, dtype=it), n, workspace=e(64, dtype=torch.uint8))  # too small
    with pytest.raises(ValueError, match="slots must have shape"):
        A.store(c[0], c[0], c, c.clone(), e(15, dtype=torch.int64))
    with pytest.raises(Exception, match="kda_kv_store"):
        A.store(c[0], c[0], c, c, e(16, dtype=torch.int64))  # keys and values into the same cache
    with pytest.raises(ValueError, match="packed batch needs"):
        A.assign_pages(n, t, n, e(1, dtype=it), page_size=16, cu_seqlens=e(3, dtype=it))
    with pytest.raises(ValueError, match="cu_seqlens must have 3"):
        A.assign_pages(n, t, n, e(1, dtype=it), page_size=16, cu_seqlens=e(4, dtype=it), total_tokens=3)
    with pytest.raises(Exception, match="kda_kv_assign"):
        A.assign_pages(n, t, n, e(1, dtype=it), page_size=24)
    with pytest.raises(Exception, match="kda_kv_assign"):
        A.assign_pages(n, t, n, e(1, dtype=it), page_size=16, lens_out=n)
    torch.cuda.synchronize()
