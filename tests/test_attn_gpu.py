"""Softmax attention, its paged cache and tables against plain torch in 64 bits
(tests/attn_reference.py, which states the error bounds)."""
import pytest
import torch

import attn_reference as R

pytestmark = pytest.mark.gpu
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
SENTINEL = 12345.0


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def attn():
    from kda_gated_delta_chunked_amd import attn as a
    return a


def rand(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def offsets(lens, dtype=torch.int32):
    cu = torch.zeros(len(lens) + 1, dtype=dtype)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    return cu


# ---------------------------------------------------------------------------
# prompts

HEADS = [(1, 1), (4, 2), (6, 1), (3, 3), (10, 2)]
LENS = [[1], [37], [64], [65], [127, 1, 128], [129], [0, 5, 0, 0, 200, 33, 0], [300], [2] * 70]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_packed_prompts(lens, heads, D):
    H, KV = heads
    g = torch.Generator().manual_seed(sum(lens) + H)
    T = sum(lens)
    q, k, v = rand(g, T, H, D, scale=1.4), rand(g, T, KV, D, scale=1.4), rand(g, T, KV, D)
    ref, lse_ref, mag, terms = R.prefill(q, k, v, lens)
    cu = offsets(lens, torch.int64 if H % 2 else torch.int32)
    out, lse = attn().prefill(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu.cuda(), return_lse=True)
    R.assert_out(out.cpu(), ref, mag)
    R.assert_lse(lse.cpu(), lse_ref, terms, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 96), (3, 130), (5, 17)])
def test_fixed_prompts_and_scale(B, T, D):
    g = torch.Generator().manual_seed(B * T)
    q, k, v = rand(g, B, T, 4, D), rand(g, B, T, 2, D), rand(g, B, T, 2, D)
    ref, lse_ref, mag, terms = R.prefill(*(x.flatten(0, 1) for x in (q, k, v)), [T] * B, scale=0.3)
    out, lse = attn().prefill(q.cuda(), k.cuda(), v.cuda(), scale=0.3, return_lse=True)
    R.assert_out(out.cpu().flatten(0, 1), ref, mag)
    R.assert_lse(lse.cpu().flatten(0, 1), lse_ref, terms, D)


@pytest.mark.parametrize("D", [64, 128])
def test_columns_of_one_row_and_rows_behind_the_last_sequence(D):
    lens, H, KV, pad = [70, 0, 131], 6, 2, 60
    g = torch.Generator().manual_seed(5)
    T = sum(lens)
    rows = rand(g, T + pad, (H + 2 * KV) * D + 64)
    rows[T:] = float("nan")
    cut = lambda x, a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
    q, k, v = cut(rows, 0, H), cut(rows, H, KV), cut(rows, H + KV, KV)
    ref, lse_ref, mag, terms = R.prefill(q[:T], k[:T], v[:T], lens)
    d = rows.cuda()
    wide = torch.full((T + pad, H * D + 128), SENTINEL, dtype=BF).cuda()
    lse = torch.full((T + pad, H), SENTINEL).cuda()
    out = wide[:, 64:64 + H * D].unflatten(1, (H, D))
    attn().prefill(cut(d, 0, H), cut(d, H, KV), cut(d, H + KV, KV), cu_seqlens=offsets(lens).cuda(), out=out, lse=lse)
    R.assert_out(out[:T].cpu(), ref, mag)
    R.assert_lse(lse[:T].cpu(), lse_ref, terms, D)
    assert (wide[T:] == SENTINEL).all() and (wide[:, :64] == SENTINEL).all() and (wide[:, 64 + H * D:] == SENTINEL).all()
    assert (lse[T:] == SENTINEL).all()


def test_no_tokens():
    z = torch.zeros(0, 4, 64, dtype=BF).cuda()
    out, lse = attn().prefill(z, z, z, cu_seqlens=torch.zeros(3, dtype=torch.int32).cuda(), return_lse=True)
    assert out.shape == z.shape and lse.shape == (0, 4)


# ---------------------------------------------------------------------------
# the cache

def pages_for(g, lens, size, R_extra=2, spare=3):
    """A shuffled block table: [R, W], rows of the requests, pages."""
    n = len(lens)
    counts = [-(-x // size) for x in lens]
    W = max(counts + [1]) + 1
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    rows = torch.randperm(n + R_extra, generator=g)[:n].to(torch.int32)
    table = torch.full((n + R_extra, W), -1, dtype=torch.int32)
    at = 0
    for r, c in zip(rows.tolist(), counts):
        table[r, :c] = order[at:at + c]
        at += c
    return table, rows, pages


def cache_of(g, pages, size, KV, D, e4m3):
    if not e4m3:
        return rand(g, pages, size, KV, D, scale=1.4), rand(g, pages, size, KV, D), None, None
    kc, vc = ((torch.randn((pages, size, KV, D), generator=g) * 60).to(E4M3) for _ in range(2))
    return kc, vc, torch.rand(KV, generator=g) * 0.02 + 0.01, torch.rand(KV, generator=g) * 0.02 + 0.01


def to_gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_decode(q, kc, vc, table, lens, rows=None, tree=None, ks=None, vs=None, **kw):
    ref, lse_ref, mag, terms = R.decode(q, kc, vc, table, lens, rows, tree, k_scale=ks, v_scale=vs)
    qd, kd, vd, td, ld, rd, trd, ksd, vsd = to_gpu(q, kc, vc, table, lens, rows, tree, ks, vs)
    out, lse = attn().decode(qd, kd, vd, td, ld, rows=rd, tree=trd, k_scale=ksd, v_scale=vsd, return_lse=True, **kw)
    R.assert_out(out.cpu(), ref, mag)
    R.assert_lse(lse.cpu(), lse_ref, terms, q.shape[-1])
    empty = lse_ref == -float("inf")
    assert (out.cpu()[empty] == 0).all()
    return out, lse


CONTEXTS = [[0], [1, 30, 31], [32, 33, 127, 128, 129, 0], [500, 3, 1000]]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [16, 32, 64, 256])
@pytest.mark.parametrize("lens", CONTEXTS, ids=str)
def test_single_tokens(lens, size, D, e4m3):
    H, KV = (6, 2) if D == 64 else (4, 1)
    g = torch.Generator().manual_seed(sum(lens) + size)
    table, rows, pages = pages_for(g, [x + 1 for x in lens], size)
    kc, vc, ks, vs = cache_of(g, pages, size, KV, D, e4m3)
    check_decode(rand(g, len(lens), 1, H, D, scale=1.4), kc, vc, table, torch.tensor(lens, dtype=torch.int32), rows,
                 None, ks, vs)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,KV", [(2, 2, 2), (5, 6, 1), (4, 8, 1), (33, 3, 3), (64, 2, 1), (17, 10, 2)])
@pytest.mark.parametrize("tree", ["chain", "shared", "each"])
def test_drafts(T, H, KV, D, tree, e4m3):
    lens = [0, 19, 260]
    g = torch.Generator().manual_seed(T * H + D)
    table, rows, pages = pages_for(g, [x + T for x in lens], 32)
    kc, vc, ks, vs = cache_of(g, pages, 32, KV, D, e4m3)
    words = None
    if tree != "chain":
        shape = (T,) if tree == "shared" else (3, T)
        words = torch.randint(-2 ** 62, 2 ** 62, shape, generator=g) << 1 | torch.randint(0, 2, shape, generator=g)
        words[..., 0] = 0  # a token that sees none of its request's own: nothing at all where the context is empty
        words[..., T - 1] = -1
    check_decode(rand(g, 3, T, H, D, scale=1.4), kc, vc, table, torch.tensor(lens, dtype=torch.int32), rows, words, ks, vs)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_empty_slots_absent_pages_and_narrow_tables(e4m3):
    g = torch.Generator().manual_seed(9)
    size, KV, H, D, T = 16, 2, 4, 128, 3
    lens = torch.tensor([100, 40, 70, 20, -5, 90], dtype=torch.int32)
    table, rows, pages = pages_for(g, [105] * 6, size)
    kc, vc, ks, vs = cache_of(g, pages, size, KV, D, e4m3)
    rows[1], rows[3] = -1, 1000
    table[rows[0], 2], table[rows[0], 3] = -1, pages  # absent in the middle of a context
    table[rows[2]] = -7                               # nothing at all is there
    check_decode(rand(g, 6, T, H, D), kc, vc, table, lens, rows, None, ks, vs)
    # a table that ends inside the contexts
    check_decode(rand(g, 6, T, H, D), kc, vc, table[:, :3].contiguous(), lens, rows, None, ks, vs)
    # rows by the requests' own order, more requests than rows
    check_decode(rand(g, 6, T, H, D), kc, vc, table[:4].contiguous(), lens, None, None, ks, vs)


def test_no_requests():
    z = torch.zeros(0, 2, 4, 64, dtype=BF).cuda()
    c = torch.zeros(1, 16, 2, 64, dtype=BF).cuda()
    e = torch.zeros(0, dtype=torch.int32).cuda()
    out, lse = attn().decode(z, c, c, torch.zeros(1, 1, dtype=torch.int32).cuda(), e, return_lse=True)
    assert out.shape == z.shape and lse.shape == (0, 2, 4)


@pytest.mark.parametrize("layout", ["pages", "tokens"])
def test_halves_of_one_buffer(layout):
    g = torch.Generator().manual_seed(11)
    size, KV, H, D = 32, 2, 6, 64
    lens = torch.tensor([77, 5], dtype=torch.int32)
    table, rows, pages = pages_for(g, [78, 6], size)
    both = rand(g, pages, 2, size, KV, D) if layout == "pages" else rand(g, pages, size, 2, KV, D)
    axis = 1 if layout == "pages" else 2
    kc, vc = both.unbind(axis)
    q = rand(g, 2, 1, H, D)
    ref, lse_ref, mag, terms = R.decode(q, kc, vc, table, lens, rows)
    kd, vd = both.cuda().unbind(axis)
    out, _ = attn().decode(q.cuda(), kd, vd, table.cuda(), lens.cuda(), rows=rows.cuda())
    R.assert_out(out.cpu(), ref, mag)
    # and stored into
    k, v = rand(g, 3, KV, D), rand(g, 3, KV, D)
    slots = torch.tensor([5, -1, 40])
    attn().store(k.cuda(), v.cuda(), kd, vd, slots.cuda())
    for c, x in ((kc, k), (vc, v)):
        c[0, 5], c[1, 8] = x[0], x[2]
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


def test_rows_of_wider_tensors_and_in_place():
    g = torch.Generator().manual_seed(12)
    size, KV, H, D, T = 16, 1, 5, 64, 2
    lens = torch.tensor([33, 0, 12], dtype=torch.int32)
    table, rows, pages = pages_for(g, [35, 2, 14], size)
    kc, vc, _, _ = cache_of(g, pages, size, KV, D, False)
    wide = rand(g, 3, T, H * D + 64)
    q = wide[..., 64:].unflatten(2, (H, D))
    ref, _, mag, _ = R.decode(q, kc, vc, table, lens, rows)
    d = wide.cuda()
    qd = d[..., 64:].unflatten(2, (H, D))
    out, lse = attn().decode(qd, *to_gpu(kc, vc, table, lens), rows=rows.cuda(), out=qd)
    assert out is qd and lse is None
    R.assert_out(qd.cpu(), ref, mag)
    assert torch.equal(d[..., :64].cpu(), wide[..., :64])


# ---------------------------------------------------------------------------
# store

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,KV", [(0, 2), (1, 1), (7, 3), (100, 2), (513, 1)])
@pytest.mark.parametrize("sliced", [False, True])
def test_store(T, KV, D, sliced, e4m3):
    g = torch.Generator().manual_seed(T + KV + D)
    size, pages = 16, -(-T // 16) + 2
    kc, vc, ks, vs = cache_of(g, pages, size, KV, D, e4m3)
    rows = rand(g, T, 2 * KV * D + 64, scale=3.0)
    k, v = rows[:, :KV * D].unflatten(1, (KV, D)), rows[:, KV * D:2 * KV * D].unflatten(1, (KV, D))
    if T:
        k[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3e38], dtype=BF)
        v[T - 1, KV - 1, -3:] = torch.tensor([-0.0, 1e-30, -3e38], dtype=BF)
    slots = torch.randperm(pages * size, generator=g)[:T]
    slots[::5] = -1
    slots[3::11] = pages * size
    d = rows.cuda()
    kd, vd = d[:, :KV * D].unflatten(1, (KV, D)), d[:, KV * D:2 * KV * D].unflatten(1, (KV, D))
    if not sliced:
        kd, vd = kd.contiguous(), vd.contiguous()
    kcd, vcd, ksd, vsd, sd = to_gpu(kc, vc, ks, vs, slots)
    attn().store(kd, vd, kcd, vcd, sd, k_scale=ksd, v_scale=vsd)
    put = (slots >= 0) & (slots < pages * size)
    for c, x, s in ((kc, k, ks), (vc, v, vs)):
        x = x[put]
        if s is not None:
            x = (x.float() / s[:, None]).clamp(-448, 448).to(E4M3)
        c.view(torch.uint8).flatten(0, 1)[slots[put]] = x.contiguous().view(torch.uint8)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if e4m3:  # (a NaN's sign is not kept)
        nan = lambda x: torch.isnan(x.float())
        assert torch.equal(nan(kcd.cpu()), nan(kc))
        kc, kcd = (x.float().nan_to_num(7.0) for x in (kc, kcd.cpu()))
        vc, vcd = (x.float().nan_to_num(7.0) for x in (vc, vcd.cpu()))
        assert torch.equal(kcd, kc) and torch.equal(vcd, vc)
    else:
        assert same(kcd.cpu(), kc) and same(vcd.cpu(), vc)


# ---------------------------------------------------------------------------
# tables and slots

def check_assign(lens, rows, cu, table, free, head, size, total, **kw):
    want = R.assign(lens, rows, cu, table, free, head, size)
    ld, rd, td, fd, hd = to_gpu(lens, rows, table, free, torch.tensor([head], dtype=torch.int32))
    cud = cu.cuda() if kw.pop("packed", True) else None
    if cud is not None:
        kw["total_tokens"] = total
    slots, lens_out, head_out = attn().assign_pages(ld, td, fd, hd, page_size=size, rows=rd, cu_seqlens=cud, **kw)
    assert slots.cpu().tolist() == want[0] + [-1] * (total - len(want[0]))
    assert lens_out.cpu().tolist() == want[1] and int(head_out) == want[2]
    assert torch.equal(td.cpu(), want[3])
    assert torch.equal(ld.cpu(), lens) and int(hd) == head  # (inputs stay)


def assign_case(g, n, most_old, most_new, size, spare=4):
    old = torch.randint(0, most_old + 1, (n,), generator=g).to(torch.int32)
    new = torch.randint(0, most_new + 1, (n,), generator=g)
    table, rows, pages = pages_for(g, [int(x) for x in old], size)
    W = -(-(most_old + most_new) // size) + 1
    table = torch.nn.functional.pad(table, (0, max(0, W - table.shape[1])), value=-1)
    free = torch.randperm(int(new.sum()) // size + n + spare, generator=g).to(torch.int32) + pages
    return old, rows, offsets(new.tolist()), table.contiguous(), free


@pytest.mark.parametrize("size", [16, 64, 1024])
@pytest.mark.parametrize("n,most_old,most_new,pad", [(1, 0, 1, 0), (1, 100, 300, 9), (5, 50, 700, 0), (300, 40, 3, 0),
                                                     (700, 90, 9, 5), (40, 2000, 2000, 1500), (1000, 0, 0, 3)])
def test_assign_packed(n, most_old, most_new, pad, size):
    g = torch.Generator().manual_seed(n + most_new + size)
    old, rows, cu, table, free = assign_case(g, n, most_old, most_new, size)
    if n > 4:
        rows[n // 2], rows[1] = -1, 1 << 20
    if n % 2:
        cu = cu.to(torch.int64)
    check_assign(old, rows, cu, table, free, 3, size, int(cu[-1]) + pad)


@pytest.mark.parametrize("n,T", [(1, 1), (6, 4), (1024, 1), (2000, 2), (3, 0)])
def test_assign_equal_lengths(n, T):
    g = torch.Generator().manual_seed(n + T)
    old = torch.randint(0, 200, (n,), generator=g).to(torch.int32)
    old[0] = -4
    table, _, pages = pages_for(g, [220] * n, 16, R_extra=0)
    table[:] = torch.randint(0, pages, table.shape, generator=g)
    free = torch.randperm(n + 9, generator=g).to(torch.int32) + pages
    check_assign(old, None, offsets([T] * n), table, free, 0, 16, n * T, packed=False, tokens_per_seq=T)


def test_assign_runs_out_of_pages_and_of_width():
    g = torch.Generator().manual_seed(21)
    old, rows, cu, table, free = assign_case(g, 30, 60, 90, 16)
    check_assign(old, rows, cu, table, free[:20].contiguous(), 5, 16, int(cu[-1]))   # too few
    check_assign(old, rows, cu, table, free[:0].contiguous(), 0, 16, int(cu[-1]))    # none
    check_assign(old, rows, cu, table, free, len(free) + 3, 16, int(cu[-1]))         # past the end already
    check_assign(old, rows, cu, table[:, :4].contiguous(), free, 0, 16, int(cu[-1]))  # too narrow
    free[7] = -2                                                                     # not a page
    check_assign(old, rows, cu, table, free, 0, 16, int(cu[-1]))
