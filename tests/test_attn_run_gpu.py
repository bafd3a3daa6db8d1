"""Prompt attention, the paged cache and attention over it as a program runs them: one after
the other over a serving run, captured in graphs and replayed, on other streams, two
at once.  References in 64 bits (tests/attn_reference.py, which states the error bounds)."""
from types import SimpleNamespace

import pytest
import torch

import attn_reference as R
from test_attn_gpu import BF, E4M3, attn, offsets, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Serving:
    """A cache and its tables on the GPU; what the requests have stored, on the CPU."""

    def __init__(self, slots, D, e4m3, seed, H=6, KV=2, size=16, pages=120, width=40):
        self.g = torch.Generator().manual_seed(seed)
        self.H, self.KV, self.D, self.size = H, KV, D, size
        dtype = E4M3 if e4m3 else BF
        both = torch.zeros(pages, 2, size, KV, D, dtype=dtype).view(torch.uint8).fill_(0x7f).view(dtype)  # (NaNs)
        self.kc, self.vc = both.cuda().unbind(1)
        self.scales = {}
        if e4m3:
            self.scales = dict(k_scale=torch.tensor([0.011, 0.02]).cuda(), v_scale=torch.tensor([0.013, 0.009]).cuda())
        self.table = torch.full((slots + 3, width), -1, dtype=torch.int32).cuda()
        self.rows = torch.randperm(slots + 3, generator=self.g)[:slots].to(torch.int32).cuda()
        self.lens = torch.zeros(slots, dtype=torch.int32).cuda()
        self.free = torch.randperm(pages, generator=self.g).to(torch.int32).cuda()
        self.head = torch.zeros(1, dtype=torch.int32).cuda()
        self.past = [(torch.zeros(0, KV, D, dtype=torch.float64),) * 2 for _ in range(slots)]

    def project(self, *lead):
        """Queries, keys and values, columns of one tensor."""
        H, KV, D = self.H, self.KV, self.D
        x = rand(self.g, *lead, (H + 2 * KV) * D, scale=1.2).cuda()
        return (x[..., :H * D].unflatten(-1, (H, D)), x[..., H * D:(H + KV) * D].unflatten(-1, (KV, D)),
                x[..., (H + KV) * D:].unflatten(-1, (KV, D)))

    def held(self, k, name):
        """What the cache has of these rows."""
        k = k.cpu()
        if not self.scales:
            return k.double()
        s = self.scales[name].cpu()[:, None]
        return (k.float() / s).clamp(-448, 448).to(E4M3).double() * s.double()

    def expect(self, n, q, k, v):
        """Of a request's new tokens, a chain behind its past."""
        ks, vs = (torch.cat([p, x]) for p, x in zip(self.past[n], (k, v)))
        T, L = q.shape[0], ks.shape[0]
        seen = torch.ones(T, L, dtype=torch.bool).tril(L - T)
        per_head = [R.attend(q[:, h].cpu(), ks[:, h // (self.H // self.KV)], vs[:, h // (self.H // self.KV)], seen, self.D ** -0.5)
                    for h in range(self.H)]
        return [torch.stack(x, 1) for x in zip(*per_head)]

    def step(self, T, keep=None):
        """T new tokens of every request, `keep` of which stay."""
        A, N = attn(), len(self.past)
        keep = T if keep is None else keep
        q, k, v = self.project(N, T)
        slots, after, self.head = A.assign_pages(self.lens, self.table, self.free, self.head, page_size=self.size,
                                                 rows=self.rows, tokens_per_seq=T)
        A.store(k.flatten(0, 1), v.flatten(0, 1), self.kc, self.vc, slots, **self.scales)
        out, lse = A.decode(q, self.kc, self.vc, self.table, self.lens, rows=self.rows, return_lse=True, **self.scales)
        hk, hv = self.held(k, "k_scale"), self.held(v, "v_scale")
        for n, row in enumerate(self.rows.tolist()):
            if row < 0:
                assert (out[n] == 0).all() and (lse[n] == -float("inf")).all()
                continue
            ref, lse_ref, mag, terms = self.expect(n, q[n], hk[n], hv[n])
            R.assert_out(out[n].cpu(), ref, mag)
            R.assert_lse(lse[n].cpu(), lse_ref, terms, self.D)
            self.past[n] = tuple(torch.cat([p, x[n, :keep]]) for p, x in zip(self.past[n], (hk, hv)))
        self.lens = after if keep == T else torch.where(self.rows >= 0, after - (T - keep), after).to(torch.int32)

    def prompts(self, lens, pad=0):
        A = attn()
        T = sum(lens)
        q, k, v = self.project(T + pad)
        cu = offsets(lens).cuda()
        slots, self.lens, self.head = A.assign_pages(self.lens, self.table, self.free, self.head, page_size=self.size,
                                                     rows=self.rows, cu_seqlens=cu, total_tokens=T + pad)
        A.store(k, v, self.kc, self.vc, slots, **self.scales)
        out, lse = A.prefill(q, k, v, cu_seqlens=cu, return_lse=True)
        ref, lse_ref, mag, terms = R.prefill(q[:T].cpu(), k[:T].cpu(), v[:T].cpu(), lens)
        R.assert_out(out[:T].cpu(), ref, mag)
        R.assert_lse(lse[:T].cpu(), lse_ref, terms, self.D)
        at = 0
        for n, length in enumerate(lens):
            new = (self.held(k[at:at + length], "k_scale"), self.held(v[at:at + length], "v_scale"))
            self.past[n] = tuple(torch.cat([p, x]) for p, x in zip(self.past[n], new))
            at += length


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_serving_run(D, e4m3):
    s = Serving(5, D, e4m3, seed=D)
    s.prompts([37, 0, 200, 64, 5], pad=11)
    for _ in range(3):
        s.step(1)
    s.step(4, keep=2)      # drafts, the last two not taken
    s.step(1)
    s.rows[2] = -1         # a request leaves
    s.step(1)
    s.step(20, keep=17)    # more rows than a wave has
    s.step(1)
    assert int(s.head) <= s.free.numel()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,width", [(1, 40), (3, 200), (16, 200)])
def test_a_step_in_a_graph(T, width, e4m3):
    # width: contexts are cut where the table has room for long ones
    A, D = attn(), 64
    s = Serving(4, D, e4m3, seed=T, width=width)
    s.prompts([37, 130, 200, 64])
    q, k, v = (x.contiguous() for x in s.project(4, T))
    state = [s.lens, s.head, s.table, s.kc, s.vc]
    lens, head = s.lens.clone(), s.head.clone()

    def step(q, k, v, lens, head, table, kc, vc):
        slots, after, top = A.assign_pages(lens, table, s.free, head, page_size=s.size, rows=s.rows, tokens_per_seq=T)
        A.store(k.flatten(0, 1), v.flatten(0, 1), kc, vc, slots, **s.scales)
        out, lse = A.decode(q, kc, vc, table, lens, rows=s.rows, return_lse=True, **s.scales)
        lens.copy_(after)
        head.copy_(top)
        return out, lse, slots

    mirror = [lens, head, s.table.clone(), s.kc.clone(), s.vc.clone()]  # for the eager steps
    step(q, k, v, *[x.clone() for x in state])  # (the library is loaded ahead of the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(q, k, v, *state)
    for turn in range(4):
        for x, new in zip((q, k, v), s.project(4, T)):
            x.copy_(new)
        want = step(q, k, v, *mirror)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn
        for a, b in zip(state, mirror):
            assert torch.equal(a.view(torch.uint8) if a.dtype == E4M3 else a.nan_to_num(3.0),
                               b.view(torch.uint8) if b.dtype == E4M3 else b.nan_to_num(3.0)), turn


@pytest.mark.parametrize("lens", [[300, 5, 77], [1500]], ids=str)
def test_prompts_in_a_graph(lens):
    A, T = attn(), sum(lens)
    g = torch.Generator().manual_seed(T)
    q, k, v = rand(g, T, 4, 64).cuda(), rand(g, T, 2, 64).cuda(), rand(g, T, 2, 64).cuda()
    cu = offsets(lens).cuda()
    A.prefill(q, k, v, cu_seqlens=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = A.prefill(q, k, v, cu_seqlens=cu, return_lse=True)
    for turn in range(3):
        for x in (q, k, v):
            x.copy_(rand(g, *x.shape).cuda())
        if len(lens) == 3:  # lengths move too
            cu[1] += 19
            cu[2] += 7
        want = A.prefill(q, k, v, cu_seqlens=cu, return_lse=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), turn


def long_context(seed, T=1, length=4000):
    g = torch.Generator().manual_seed(seed)
    pages = -(-(length + T) // 64)
    kc, vc = rand(g, pages, 64, 2, 64).cuda(), rand(g, pages, 64, 2, 64).cuda()
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    return rand(g, 1, T, 4, 64).cuda(), kc, vc, table, torch.tensor([length], dtype=torch.int32).cuda()


def test_two_graphs_on_one_workspace():
    A = attn()
    args = [long_context(s) for s in (1, 2)]
    want = [A.decode(*a) for a in args]
    q, kc, _, table, _ = args[0]
    need = A.decode_workspace_size(A.DecodeProblem(1, 1, 4, 0.125, 1, table.shape[1], 0, 0, 0,
                                                   A.KvCache(2, 64, 0, 64, kc.shape[0], 0, 0)))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for a in args:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(A.decode(*a, workspace=ws)[0])
    for _ in range(3):
        for i in (1, 0):
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(got[i], want[i][0])
        got[0].zero_()
        ws.fill_(255)


def test_two_calls_at_once():
    A = attn()
    args = [long_context(s, T, 9000) for s, T in ((1, 1), (2, 1), (3, 20), (4, 20))]
    want = [A.decode(*a, return_lse=True) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(5):
        got = [A.decode(*a, return_lse=True, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_behind_queued_work_of_another_stream():
    A = attn()
    s = Serving(3, 64, False, seed=1)
    s.prompts([20, 60, 100])
    q, k, v = s.project(3, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.zeros_like(x.contiguous()) for x in (q, k, v)]
    lens, table = torch.zeros_like(s.lens), torch.full_like(s.table, -1)
    kc, vc = torch.zeros_like(s.kc), torch.zeros_like(s.vc)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # inputs come late
        for a, b in zip((*late, lens, table, kc, vc), (q, k, v, s.lens, s.table, s.kc, s.vc)):
            a.copy_(b)
    slots, after, head = A.assign_pages(lens, table, s.free, s.head, page_size=s.size, rows=s.rows, tokens_per_seq=2,
                                        stream=side)
    A.store(late[1].flatten(0, 1), late[2].flatten(0, 1), kc, vc, slots, stream=side)
    out, lse = A.decode(late[0], kc, vc, table, lens, rows=s.rows, return_lse=True, stream=side)
    one, _ = A.prefill(late[0], late[1], late[2], stream=side)
    side.synchronize()
    want = A.assign_pages(s.lens, s.table, s.free, s.head, page_size=s.size, rows=s.rows, tokens_per_seq=2)
    A.store(k.flatten(0, 1), v.flatten(0, 1), s.kc, s.vc, want[0])
    eager = A.decode(q, s.kc, s.vc, s.table, s.lens, rows=s.rows, return_lse=True)
    assert torch.equal(slots, want[0]) and torch.equal(after, want[1]) and torch.equal(head, want[2])
    assert torch.equal(table, s.table) and torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    assert torch.equal(one, A.prefill(q, k, v)[0])


def calls():
    e = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda:0")
    i32 = torch.int32
    q, kv = e(2, 3, 4, 64), e(2, 3, 2, 64)
    kc, vc, table, lens = e(3, 16, 2, 64), e(3, 16, 2, 64), e(2, 4, dtype=i32), e(2, dtype=i32)
    A = attn()
    return {
        "prefill": lambda s: A.prefill(q, kv, kv, stream=s),
        "decode": lambda s: A.decode(q, kc, vc, table, lens, stream=s),
        "store": lambda s: A.store(kv[0], kv[0], kc, vc, torch.arange(3, device="cuda:0"), stream=s),
        "assign_pages": lambda s: A.assign_pages(lens, table, lens, lens[:1].clone(), page_size=16, stream=s),
    }


@pytest.mark.parametrize("name", ["prefill", "decode", "store", "assign_pages"])
def test_another_devices_stream_is_refused(name):
    call = calls()[name]
    side = torch.cuda.Stream(torch.device("cuda", 0))
    torch.cuda.synchronize()
    call(side)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(SimpleNamespace(device=torch.device("cuda", 1)))
    torch.cuda.synchronize()
