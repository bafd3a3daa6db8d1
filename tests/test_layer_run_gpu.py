"""The layer operators as a program runs them: one after the other in a layer,
prompts then single tokens, captured in graphs and replayed, on other streams,
on many sequences and on buffers past 32-bit offsets.  References in 64 bits
(tests/layer_reference.py, which states the error bounds)."""
import pytest
import torch

import layer_reference as R
from test_layer_gpu import BF, K, NAN, cuda, offsets, on_gpu, rand, scan_args, scan_case, scan_ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---------------------------------------------------------------------------
# a layer: residual norm, projection, convolution, scan, gated output, norm

class Layer:
    H, G, P, N, W, hidden = 4, 2, 64, 128, 4, 256

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.inner, self.bc = self.H * self.P, self.G * self.N
        self.D = self.inner + 2 * self.bc
        self.norm_w = rand(g, self.hidden, scale=0.1) + 1
        self.proj = rand(g, self.hidden, self.D + self.inner + 8, scale=self.hidden ** -0.5)
        self.conv_w, self.conv_b = rand(g, self.D, self.W, scale=0.4), rand(g, self.D, scale=0.1)
        self.A = -(torch.rand(self.H, generator=g) * 4 + 0.5)
        self.skip, self.dt_bias = torch.rand(self.H, generator=g), torch.randn(self.H, generator=g) - 2
        self.out_w = rand(g, self.inner, scale=0.1) + 1

    def cuda(self):
        for k, v in vars(self).items():
            if torch.is_tensor(v):
                setattr(self, k, v.cuda())
        return self

    def project(self, h):
        """Columns of one product, its rows a multiple of 8 long: the convolution's
        input, the gate and the steps."""
        u = (h.float() @ self.proj.float()).to(BF)
        return u[..., :self.D], u[..., self.D:self.D + self.inner], u[..., -8:][..., :self.H].float()

    def columns(self, c):
        at = self.inner + self.bc
        return (c[..., :self.inner].unflatten(-1, (self.H, self.P)),
                c[..., self.inner:at].unflatten(-1, (self.G, self.N)),
                c[..., at:].unflatten(-1, (self.G, self.N)))

    def scan_kw(self, z):
        return dict(D=self.skip, z=z.unflatten(-1, (self.H, self.P)), dt_bias=self.dt_bias, dt_softplus=True)

    def prompt(self, x, res, cu, conv0, ssm0, **kw):
        k = K()
        h, res, _ = k.add_rmsnorm(x, self.norm_w, residual=res)
        u, z, dt = self.project(h)
        c, conv1 = k.conv_prefill(u, self.conv_w, self.conv_b, cu_seqlens=cu, initial_state=conv0)
        xs, B, C = self.columns(c)
        y, ssm1 = k.ssm_prefill(xs, dt, self.A, B, C, cu_seqlens=cu, initial_state=ssm0, **self.scan_kw(z), **kw)
        q, _, s = k.add_rmsnorm(y.flatten(-2), self.out_w, out_dtype=E4M3, scale_group=128)
        return dict(h=h, res=res, u=u, z=z, dt=dt, c=c, y=y, q=q, s=s, conv=conv1, ssm=ssm1)

    def step(self, x, res, conv, ssm, idx):
        k = K()
        h, res, _ = k.add_rmsnorm(x, self.norm_w, residual=res)
        u, z, dt = self.project(h)
        c = k.conv_decode(u, self.conv_w, self.conv_b, conv, idx)
        xs, B, C = self.columns(c)
        y = k.ssm_decode(xs, dt, self.A, B, C, ssm, idx, **self.scan_kw(z))
        q, _, s = k.add_rmsnorm(y.flatten(-2), self.out_w, out_dtype=E4M3, scale_group=128)
        return dict(h=h, res=res, u=u, z=z, dt=dt, c=c, y=y, q=q, s=s)


def check_layer(m, x, res, r, conv0, ssm0, lens):
    """Each operator's output against its formula on the operator's own input."""
    c = {k: v.cpu() if torch.is_tensor(v) else v for k, v in r.items()}
    p = {k: v.cpu() if torch.is_tensor(v) else v for k, v in vars(m).items()}
    ref, s = R.norm(x.cpu(), res.cpu(), p["norm_w"], 1e-6)
    R.assert_norm(c["h"], None, ref, 0)
    assert torch.equal(c["res"], (x.cpu().float() + res.cpu().float()).to(BF))
    ref, conv1, mag = R.conv(c["u"], p["conv_w"], p["conv_b"], "silu", conv0.cpu(), lens)
    R.assert_conv(c["c"], ref, mag, "silu")
    xs, B, C = m.columns(c["c"])
    ref, ssm1, mag, smag = R.scan(xs, R.steps(c["dt"], p["dt_bias"], True), p["A"], B, C, p["skip"],
                                  c["z"].unflatten(-1, (m.H, m.P)), ssm0.cpu(), lens)
    R.assert_scan_out(c["y"], ref, mag)
    ref, _ = R.norm(c["y"].flatten(-2), None, p["out_w"], 1e-6)
    R.assert_norm(c["q"], c["s"], ref, 128)
    return conv1, ssm1, smag


@pytest.mark.parametrize("piece", [0, 64])
def test_layer_on_prompts(piece):
    m, lens = Layer(1).cuda(), [150, 0, 1, 77]
    g = torch.Generator().manual_seed(11)
    x, res = rand(g, sum(lens), m.hidden).cuda(), rand(g, sum(lens), m.hidden).cuda()
    conv0, ssm0 = rand(g, 4, 3, m.D).cuda(), rand(g, 4, m.H, m.N, m.P, dtype=torch.float32).cuda()
    r = m.prompt(x, res, offsets(lens).cuda(), conv0, ssm0, piece_tokens=piece)
    conv1, ssm1, smag = check_layer(m, x, res, r, conv0, ssm0, lens)
    assert torch.equal(r["conv"].cpu().to(R.F64), conv1)
    R.assert_state(r["ssm"].cpu(), ssm1, smag)


@pytest.mark.parametrize("T", [1, 3])
def test_layer_prompt_then_single_tokens(T):
    # three requests of 70 tokens: 70 - 2 T as prompts, then twice T tokens on
    # pools; the convolution's rows are those of the whole prompt bit for bit
    m, N, L = Layer(2).cuda(), 3, 70
    g = torch.Generator().manual_seed(12)
    x, res = rand(g, N, L, m.hidden).cuda(), rand(g, N, L, m.hidden).cuda()
    conv0 = torch.zeros(N, 3, m.D, dtype=BF).cuda()
    ssm0 = torch.zeros(N, m.H, m.N, m.P).cuda()
    rows = [t[:, :L - 2 * T].flatten(0, 1) for t in (x, res)]
    head = L - 2 * T
    r = m.prompt(*rows, offsets([head] * N).cuda(), None, None)
    check_layer(m, *rows, r, conv0, ssm0, [head] * N)
    idx = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    conv, ssm = rand(g, 6, 3, m.D).cuda(), rand(g, 6, m.H, m.N, m.P, dtype=torch.float32).cuda()
    conv[idx.long()], ssm[idx.long()] = r["conv"], r["ssm"]
    parts = [r["c"].unflatten(0, (N, head))]
    us = [r["u"].unflatten(0, (N, head))]
    for at in (head, head + T):
        xt, rt = x[:, at:at + T].contiguous(), res[:, at:at + T].contiguous()
        before = conv[idx.long()].clone(), ssm[idx.long()].clone()
        r = m.step(xt, rt, conv, ssm, idx)
        flat = {k: v.flatten(0, 1) if torch.is_tensor(v) else v for k, v in r.items()}
        conv1, ssm1, smag = check_layer(m, xt.flatten(0, 1), rt.flatten(0, 1), flat, *before, [T] * N)
        assert torch.equal(conv[idx.long()].cpu().to(R.F64), conv1)
        R.assert_state(ssm[idx.long()].cpu(), ssm1, smag)
        parts.append(r["c"])
        us.append(r["u"])
    whole, _ = K().conv_prefill(torch.cat(us, 1), m.conv_w, m.conv_b)
    assert torch.equal(torch.cat(parts, 1), whole)


def test_convolution_feeds_the_delta_rule_prefill():
    # q, k and v of the delta-rule attention from one convolution, then two more
    # tokens by the two state-pool steps
    k = K()
    H, Dh, L = 2, 128, 90
    g = torch.Generator().manual_seed(13)
    D = 3 * H * Dh
    u, w = rand(g, 1, L, D, scale=0.3).cuda(), rand(g, D, 4, scale=0.4).cuda()
    decay = (-torch.rand(1, L, H, Dh, generator=g) * 0.2).cuda()
    beta = torch.rand(1, L, H, generator=g).cuda()

    def heads(c):
        q, kk, v = (t.unflatten(-1, (H, Dh)).contiguous() for t in c.chunk(3, -1))
        return q, (kk.float() / kk.float().norm(dim=-1, keepdim=True).clamp(min=1e-3)).to(BF), v

    c, _ = k.conv_prefill(u, w)
    whole, _ = k.prefill(*heads(c), decay, beta)
    cut = L - 2
    c1, rows = k.conv_prefill(u[:, :cut], w)
    assert torch.equal(c1, c[:, :cut])
    _, S = k.prefill(*heads(c1), decay[:, :cut].contiguous(), beta[:, :cut].contiguous())
    idx = torch.zeros(1, dtype=torch.int32).cuda()
    c2 = k.conv_decode(u[:, cut:], w, None, rows, idx)
    assert torch.equal(c2, c[:, cut:])
    out = k.decode(*heads(c2), decay[:, cut:].contiguous(), beta[:, cut:].contiguous(), S.contiguous(), idx)
    out = out[0] if isinstance(out, tuple) else out
    a, b = out.float(), whole[:, cut:].float()
    # both are within 1e-2 of the recurrence (the prefill's own bound)
    assert (a - b).norm() <= 2e-2 * b.norm()


# ---------------------------------------------------------------------------
# graphs and streams

def operators(seed):
    """name -> (inputs that change from replay to replay, call(inputs) -> outputs)"""
    k = K()
    g = torch.Generator().manual_seed(seed)
    w, b = rand(g, 136, 4).cuda(), rand(g, 136).cuda()
    cu, idx = offsets([70, 0, 3, 200]).cuda(), torch.tensor([3, -1, 0], dtype=torch.int32).cuda()
    c = on_gpu(scan_case(g, 273, 4, 1, 64, 128, z=True, softplus=True, skip=True))
    f = on_gpu(scan_case(g, 2048, 2, 1, 128, 128, z=False, softplus=False, skip=False))
    f = {n: v[None] if n in ("x", "B", "C", "dt") else v for n, v in f.items()}
    s = on_gpu(scan_case(g, 6, 4, 1, 64, 128, z=True, softplus=True, skip=True))
    s = {n: v.unflatten(0, (3, 2)) if n in ("x", "B", "C", "z", "dt") else v for n, v in s.items()}

    def scan(d, **more):
        a, kw = scan_args(d)
        return lambda x, s0: k.ssm_prefill(x, *a[1:], **kw, initial_state=s0, **more)

    def scan_step(x, pool):
        a, kw = scan_args(s)
        pool = pool.clone()
        return k.ssm_decode(x, *a[1:], pool, idx, **kw), pool

    def conv_step(x, pool):
        pool = pool.clone()
        return k.conv_decode(x, w, b, pool, idx), pool

    nw = rand(g, 520).cuda()
    return {
        "conv": ([rand(g, 273, 136).cuda(), rand(g, 4, 3, 136).cuda()],
                 lambda x, s0: k.conv_prefill(x, w, b, cu_seqlens=cu, initial_state=s0)),
        "conv_step": ([rand(g, 3, 2, 136).cuda(), rand(g, 5, 3, 136).cuda()], conv_step),
        "scan": ([c["x"].clone(), rand(g, 4, 4, 128, 64, dtype=torch.float32).cuda()], scan(c, cu_seqlens=cu)),
        "scan_pieces": ([c["x"].clone(), rand(g, 4, 4, 128, 64).cuda()], scan(c, cu_seqlens=cu, piece_tokens=64)),
        "scan_auto": ([f["x"].clone(), rand(g, 1, 2, 128, 128, dtype=torch.float32).cuda()], scan(f)),
        "scan_step": ([s["x"].clone(), rand(g, 5, 4, 128, 64, dtype=torch.float32).cuda()], scan_step),
        "norm": ([rand(g, 33, 520).cuda(), rand(g, 33, 520).cuda()],
                 lambda x, r: k.add_rmsnorm(x, nw, residual=r)[:2]),
        "norm_e4m3": ([rand(g, 33, 520).cuda(), rand(g, 33, 520).cuda()],
                      lambda x, r: tuple(t.view(torch.uint8) if t.dtype == E4M3 else t for t in
                                         k.add_rmsnorm(x, nw, residual=r, out_dtype=E4M3, scale_group=128))),
    }


NAMES = ["conv", "conv_step", "scan", "scan_pieces", "scan_auto", "scan_step", "norm", "norm_e4m3"]


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays_give_the_eager_results(name):
    inputs, call = operators(21)[name]
    g = torch.Generator().manual_seed(22)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):  # no warm-up call
        got = call(*inputs)
    for _ in range(4):
        for t in inputs:
            t.copy_(rand(g, *t.shape, scale=0.7, dtype=t.dtype))
        want = [t.clone() for t in call(*inputs)]  # eager work between the replays
        for t in got:
            t.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_split_scans_replayed_in_turn():
    # each capture took a workspace of its own: replays in any order, and at the
    # same time on two streams, give the eager results
    graphs = []
    for seed in (31, 32):
        inputs, call = operators(seed)["scan_auto"]
        want = [t.clone() for t in call(*inputs)]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = call(*inputs)
        graphs.append((graph, got, want, inputs, call))  # a graph reads its inputs where they were
    side = torch.cuda.Stream()
    for both in (False, True, False):
        for _, got, *_ in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        graphs[0][0].replay()
        if both:
            with torch.cuda.stream(side):
                graphs[1][0].replay()
        else:
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, got, want, *_ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_other_streams(name):
    inputs, call = operators(41)[name]
    want = [t.clone() for t in call(*inputs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(*inputs)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stream_argument_and_two_scans_in_flight():
    # the operators' own buffers (results and workspaces) stay theirs until the
    # given stream is done with them
    inputs, _ = operators(51)["scan_auto"]
    k = K()
    g = torch.Generator().manual_seed(52)
    f = on_gpu(scan_case(g, 2048, 2, 1, 128, 128, z=False, softplus=False, skip=False))
    a, kw = scan_args({n: v[None] if n in ("x", "B", "C", "dt") else v for n, v in f.items()})
    want = k.ssm_prefill(*a, **kw, initial_state=inputs[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [k.ssm_prefill(*a, **kw, initial_state=inputs[1], stream=s) for s in streams]
        junk = [torch.full((1 << 20,), NAN, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        for r in got:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_change_from_call_to_call(name):
    inputs, call = operators(61)[name]
    first = [t.clone() for t in call(*inputs)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(*inputs), first))


# ---------------------------------------------------------------------------
# sizes

@pytest.mark.parametrize("cu", [torch.int32, torch.int64])
def test_many_short_sequences(cu):
    k = K()
    g = torch.Generator().manual_seed(71)
    lens = torch.randint(0, 4, (4500,), generator=g).tolist()
    lens[17], lens[4000] = 90, 41
    T, N = sum(lens), len(lens)
    c = scan_case(g, T, 1, 1, 64, 64, z=False, softplus=True, skip=True)
    s0 = rand(g, N, 1, 64, 64, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    a, kw = scan_args(on_gpu(c))
    for piece in (0, 64):
        out, fin = k.ssm_prefill(*a, **kw, cu_seqlens=offsets(lens, cu).cuda(), initial_state=s0.cuda(),
                                 piece_tokens=piece)
        R.assert_scan_out(out.cpu(), ref, mag)
        R.assert_state(fin.cpu(), final, smag)
    x, w, r0 = rand(g, T, 16), rand(g, 16, 4), rand(g, N, 3, 16)
    ref, final, mag = R.conv(x, w, None, "silu", r0, lens)
    out, fin = k.conv_prefill(x.cuda(), w.cuda(), cu_seqlens=offsets(lens, cu).cuda(), initial_state=r0.cuda())
    R.assert_conv(out.cpu(), ref, mag, "silu")
    assert torch.equal(fin.cpu().to(R.F64), final)


@pytest.mark.parametrize("dims", [(128, 128), (64, 64)], ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_automatic_pieces(dims, packed):
    P, N = dims
    lens, H = ([2100, 2100] if not packed else [3000, 0, 40, 1300]), 2
    g = torch.Generator().manual_seed(72)
    c = scan_case(g, sum(lens), H, 1, P, N, z=True, softplus=True, skip=True)
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    p = K().SsmProblem(len(lens), sum(lens), H, 1, P, N, 1, 0, 0, 0, int(packed), 0, 0, 0, 0, 0)
    assert K().ssm_plan(p) > 0
    d = on_gpu(c)
    if not packed:
        d = {k: v.unflatten(0, (2, 2100)) if k in ("x", "B", "C", "z", "dt") else v for k, v in d.items()}
    a, kw = scan_args(d)
    more = dict(cu_seqlens=offsets(lens).cuda()) if packed else {}
    out, fin = K().ssm_prefill(*a, **kw, **more, initial_state=s0.cuda())
    R.assert_scan_out(out.cpu().view(ref.shape), ref, mag)
    R.assert_state(fin.cpu(), final, smag)


def test_a_reset_among_slow_tokens():
    # tokens that keep nothing, between others that keep nearly all: the small
    # logarithms behind a huge one count
    H, P, N = 2, 64, 128
    g = torch.Generator().manual_seed(73)
    c = scan_case(g, 140, H, 1, P, N, z=False, softplus=False, skip=False)
    c["A"] = torch.full((H,), -1.0)
    for t in (5, 40, 41, 96, 127):
        c["dt"][t] = 1e7
        c["x"][t] *= 1e-6
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, [140])
    a, kw = scan_args(on_gpu(c))
    for piece in (0, 64):
        out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets([140]).cuda(), initial_state=s0.cuda(),
                                   piece_tokens=piece)
        R.assert_scan_out(out.cpu(), ref, mag)
        R.assert_state(fin.cpu(), final, smag)


def test_nothing_to_do():
    k = K()
    e = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")
    f32 = torch.float32
    s0 = torch.randn(2, 2, 64, 64, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, fin = k.ssm_prefill(e(0, 2, 64), e(0, 2, dtype=f32), e(2, dtype=f32), e(0, 1, 64), e(0, 1, 64),
                             cu_seqlens=cu, initial_state=s0)
    assert out.shape == (0, 2, 64) and torch.equal(fin, s0)
    r0 = torch.randn(2, 3, 16, device="cuda").to(BF)
    out, fin = k.conv_prefill(e(0, 16), e(16, 4), cu_seqlens=cu, initial_state=r0)
    assert out.shape == (0, 16) and torch.equal(fin, r0)
    assert k.add_rmsnorm(e(0, 64), e(64))[0].shape == (0, 64)
    pool = r0.clone()
    idx = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert k.conv_decode(e(0, 1, 16), e(16, 4), None, pool, idx).shape == (0, 1, 16)
    states = s0.clone()
    k.ssm_decode(e(0, 1, 2, 64), e(0, 1, 2, dtype=f32), e(2, dtype=f32), e(0, 1, 1, 64), e(0, 1, 1, 64), states, idx)
    torch.cuda.synchronize()
    assert torch.equal(pool, r0) and torch.equal(states, s0)


def test_rows_past_32_bit_offsets():
    # rows 2^23 - 8 elements apart: the last of 400 starts 6.7e9 bytes in
    k = K()
    stride, T, H, P, N = (1 << 23) - 8, 400, 2, 64, 64
    g = torch.Generator().manual_seed(74)
    c = scan_case(g, T, H, 1, P, N, z=False, softplus=True, skip=True)
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    big = torch.empty(T * stride, dtype=BF, device="cuda").view(T, stride)
    d = on_gpu(c)
    at = 0
    for name, width in (("x", H * P), ("B", N), ("C", N)):
        view = big[:, at:at + width].unflatten(-1, d[name].shape[1:])
        view.copy_(d[name])
        d[name], at = view, at + width
    a, kw = scan_args(d)
    ref, final, mag, smag = scan_ref(c, s0, [T])
    for piece in (0, 64):
        out, fin = k.ssm_prefill(*a, **kw, cu_seqlens=offsets([T]).cuda(), initial_state=s0.cuda(),
                                 piece_tokens=piece)
        R.assert_scan_out(out.cpu(), ref, mag)
        R.assert_state(fin.cpu(), final, smag)
    w = rand(g, at, 4)
    ref, _, mag = R.conv(big[:, :at].cpu(), w, None, "silu", torch.zeros(1, 3, at, dtype=BF), [T])
    wide = torch.empty_like(big)[:, 64:64 + at]
    out, _ = k.conv_prefill(big[:, :at], w.cuda(), out=wide)
    R.assert_conv(out.cpu(), ref, mag, "silu")
    nw = rand(g, at)
    out, _, _ = k.add_rmsnorm(big[:, :at], nw.cuda())
    R.assert_norm(out.cpu(), None, R.norm(big[:, :at].cpu(), None, nw, 1e-6)[0], 0)


def test_pool_entries_past_32_bit_offsets():
    k = K()
    H, P, N, size = 32, 128, 128, 8300  # 4.35e9 elements
    g = torch.Generator().manual_seed(75)
    pool = torch.empty(size, H, N, P, device="cuda")
    idx = torch.tensor([size - 1, 1], dtype=torch.int32)
    s0 = rand(g, 2, H, N, P, dtype=torch.float32)
    pool[idx.long().cuda()] = s0.cuda()
    c = scan_case(g, 2, H, 1, P, N, z=True, softplus=True, skip=True)
    ref, final, mag, smag = scan_ref(c, s0, [1, 1])
    d = {n: v.unflatten(0, (2, 1)) if n in ("x", "B", "C", "z", "dt") else v for n, v in on_gpu(c).items()}
    a, kw = scan_args(d)
    out = k.ssm_decode(*a, pool, idx.cuda(), **kw)
    R.assert_scan_out(out.cpu().flatten(0, 1), ref, mag)
    R.assert_state(pool[idx.long().cuda()].cpu(), final, smag)
    del pool
    dim, size = 8192, 90000  # 2.2e9 elements
    rows = torch.empty(size, 3, dim, dtype=BF, device="cuda")
    at = torch.tensor([size - 1, 0], dtype=torch.int32)
    r0, x, w = rand(g, 2, 3, dim), rand(g, 2, 1, dim), rand(g, dim, 4)
    rows[at.long().cuda()] = r0.cuda()
    out = k.conv_decode(x.cuda(), w.cuda(), None, rows, at.cuda())
    ref, final, mag = R.conv(x.flatten(0, 1), w, None, "silu", r0, [1, 1])
    R.assert_conv(out.cpu().flatten(0, 1), ref, mag, "silu")
    assert torch.equal(rows[at.long().cuda()].cpu().to(R.F64), final)


# ---------------------------------------------------------------------------
# refusals of the binding (nothing is enqueued)

def test_binding_refusals():
    k = K()
    g = torch.Generator().manual_seed(81)
    x, w = rand(g, 10, 64).cuda(), rand(g, 64, 4).cuda()
    d = on_gpu(scan_case(g, 10, 2, 1, 64, 64, z=True, softplus=True, skip=True))
    a, kw = scan_args(d)
    nw = rand(g, 64).cuda()
    idx = torch.zeros(1, dtype=torch.int32).cuda()
    pool = torch.zeros(2, 3, 64, dtype=BF).cuda()
    states = torch.zeros(2, 2, 64, 64).cuda()
    for call, err in [
            (lambda: k.conv_prefill(x.cpu(), w), ValueError),
            (lambda: k.conv_prefill(x, w.cpu()), ValueError),
            (lambda: k.conv_prefill(x.float(), w), TypeError),
            (lambda: k.conv_prefill(x, w.t().contiguous()), ValueError),
            (lambda: k.conv_prefill(x, w, out=x), k.KDAError),
            (lambda: k.conv_prefill(x.t(), w), ValueError),
            (lambda: k.conv_prefill(x, w, activation="relu"), ValueError),
            (lambda: k.conv_prefill(x[None], w, cu_seqlens=idx), ValueError),
            (lambda: k.conv_prefill(x, w, cu_seqlens=torch.zeros(2).cuda()), TypeError),
            (lambda: k.conv_prefill(x, w, initial_state=pool[:1].float()), TypeError),
            (lambda: k.conv_decode(x, w, None, pool, idx), ValueError),
            (lambda: k.conv_decode(x[None], w, None, pool, idx.long()), TypeError),
            (lambda: k.conv_decode(x[None], w, None, pool.transpose(1, 2), idx), ValueError),
            (lambda: k.ssm_prefill(a[0], a[1].to(BF), *a[2:], **kw), TypeError),
            (lambda: k.ssm_prefill(*a[:4], a[4][:, :, :32], **kw), ValueError),
            (lambda: k.ssm_prefill(a[0][..., :48].contiguous(), *a[1:], D=kw["D"]), k.KDAError),
            (lambda: k.ssm_prefill(*a, **kw, out=a[0]), k.KDAError),
            (lambda: k.ssm_prefill(*a, **kw, piece_tokens=48), k.KDAError),
            (lambda: k.ssm_prefill(*a, **kw, piece_tokens=-64), k.KDAError),
            (lambda: k.ssm_prefill(*a, **kw, initial_state=states[:1].half()), TypeError),
            (lambda: k.ssm_prefill(*a, **kw, initial_state=states), ValueError),
            (lambda: k.ssm_decode(*a, states, idx, **kw), ValueError),
            (lambda: k.add_rmsnorm(x, nw, residual_out=x), ValueError),
            (lambda: k.add_rmsnorm(x, nw, out_dtype=torch.float16), TypeError),
            (lambda: k.add_rmsnorm(x, nw, scale_group=128), ValueError),
            (lambda: k.add_rmsnorm(x, nw, out_dtype=E4M3, scale_group=64), k.KDAError),
            (lambda: k.add_rmsnorm(x[:, :60].contiguous(), nw[:60]), k.KDAError),
            (lambda: k.add_rmsnorm(x, nw, eps=-1.0), k.KDAError)]:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
    assert not pool.any() and not states.any()


@pytest.mark.parametrize("dims", [(128, 128), (64, 128), (128, 64), (64, 64)], ids=str)
@pytest.mark.parametrize("H,skip,z", [(1, False, False), (2, True, True)])
def test_single_tokens_are_rounded_once(dims, H, skip, z):
    # sequences of one token from a zero state: nothing evens a score's rounding
    # out, so what it loses has to be added back; the output's rounding is left
    P, N = dims
    lens = [1] * 50
    g = torch.Generator().manual_seed(91)
    c = scan_case(g, 50, H, 1, P, N, z=z, softplus=True, skip=skip)
    ref, _, mag, _ = scan_ref(c, torch.zeros(50, H, N, P), lens)
    a, kw = scan_args(on_gpu(c))
    out, _ = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda())
    err = (out.cpu().to(R.F64) - ref).abs()
    assert (err <= R.BF16 * ref.abs() + 2e-5 * mag).all(), (err - R.BF16 * ref.abs() - 2e-5 * mag).max()


@pytest.mark.parametrize("dims", [(128, 128), (64, 64)], ids=str)
@pytest.mark.parametrize("piece", [0, 64])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN, 3e38])
def test_special_inputs_reach_their_column_and_later_tokens_alone(dims, piece, value):
    # x feeds one column of one head's state: everything else, and that column
    # ahead of the token, is as if it were not there (a huge value is finite but
    # overflows what follows it)
    P, N = dims
    T, H = 200, 2
    g = torch.Generator().manual_seed(92)
    c = scan_case(g, T, H, 1, P, N, z=False, softplus=False, skip=True, slow=True)
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, [T])
    hit = [(70, 0, 5), (17, 1, P - 1), (95, 1, 33)]
    for t, h, p in hit:
        c["x"][t, h, p] = value
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets([T]).cuda(), initial_state=s0.cuda(), piece_tokens=piece)
    out, fin = out.cpu(), fin.cpu()
    clean, kept = torch.ones(T, H, P, dtype=torch.bool), torch.ones(H, N, P, dtype=torch.bool)
    for t, h, p in hit:
        clean[t:, h, p] = False
        kept[h, :, p] = False
        if value != 3e38:
            assert not torch.isfinite(out[t:, h, p].float()).any() and not torch.isfinite(fin[0, h, :, p]).any()
    R.assert_scan_out(out[clean], ref[clean], mag[clean])
    R.assert_state(fin[0][kept], final[0][kept], smag[0][kept])


@pytest.mark.parametrize("dims", [(128, 128), (64, 128)], ids=str)
@pytest.mark.parametrize("piece", [0, 64])
def test_a_bad_step_stays_in_its_head_and_a_bad_read_in_its_token(dims, piece):
    P, N = dims
    T, H = 150, 4
    g = torch.Generator().manual_seed(93)
    c = scan_case(g, T, H, 2, P, N, z=True, softplus=True, skip=True)
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, [T])
    c["dt"][70, 0] = NAN
    c["C"][33, 1, 3] = NAN
    c["z"][100, 1, 7] = NAN
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets([T]).cuda(), initial_state=s0.cuda(), piece_tokens=piece)
    out, fin = out.cpu(), fin.cpu()
    bad = torch.zeros(T, H, P, dtype=torch.bool)
    bad[70:, 0] = bad[33, 2:] = True
    bad[100, 1, 7] = True
    assert torch.isnan(out[bad].float()).all() and torch.isnan(fin[0, 0]).all()
    R.assert_scan_out(out[~bad], ref[~bad], mag[~bad])
    R.assert_state(fin[0, 1:], final[0, 1:], smag[0, 1:])


@pytest.mark.parametrize("piece", [0, 64])
def test_outputs_do_not_depend_on_the_final_state(piece):
    lens, H, P, N = [1, 130, 0, 64, 40], 2, 64, 128
    g = torch.Generator().manual_seed(94)
    a, kw = scan_args(on_gpu(scan_case(g, sum(lens), H, 1, P, N, z=False, softplus=True, skip=False)))
    kw |= dict(cu_seqlens=offsets(lens).cuda(), piece_tokens=piece)
    out, fin = K().ssm_prefill(*a, **kw)
    bare, none = K().ssm_prefill(*a, **kw, output_final_state=False)
    assert none is None and torch.equal(out, bare)
    half, fin16 = K().ssm_prefill(*a, **kw, state_dtype=BF)
    assert torch.equal(out, half) and torch.equal(fin.to(BF), fin16)
