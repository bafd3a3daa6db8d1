"""The layer operators at the edges of their ranges, against their formulas in
64 bits (tests/layer_reference.py, which states the error bounds)."""
import pytest
import torch

import layer_reference as R
from test_layer_gpu import BF, DIMS, K, offsets, on_gpu, rand, scan_args, scan_case, scan_ref

pytestmark = pytest.mark.gpu
INF = float("inf")
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---------------------------------------------------------------------------
# time steps: a logit of -inf or of the type's lowest value is no step at all,
# and the type's largest value keeps nothing of the state

def masked_steps(g, T, H, P, N):
    c = scan_case(g, T, H, 1, P, N, z=True, softplus=True, skip=True)
    c["dt"][3], c["dt"][17, 0], c["dt"][40:45] = -INF, LOWEST, -3e38
    c["dt"][70, 1], c["x"][70], c["B"][70] = -LOWEST, 0, c["B"][70] * 1e-3
    return c


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [0, 64])
def test_masked_time_steps_in_prompts(dims, piece):
    P, N = dims
    lens, H = [90, 1, 55], 2
    g = torch.Generator().manual_seed(101)
    c = masked_steps(g, sum(lens), H, P, N)
    c["dt"][90] = -INF  # a sequence that is masked throughout
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    assert torch.equal(final[1], s0[1].to(R.F64))
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=s0.cuda(), piece_tokens=piece)
    R.assert_scan_out(out.cpu(), ref, mag)
    R.assert_state(fin.cpu(), final, smag)


def test_a_bias_that_masks_a_head():
    T, H, P, N = 70, 2, 64, 64
    g = torch.Generator().manual_seed(102)
    c = scan_case(g, T, H, 1, P, N, z=False, softplus=True, skip=True)
    c["dt_bias"][1] = -INF
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, [T])
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, initial_state=s0.cuda(), cu_seqlens=offsets([T]).cuda())
    R.assert_scan_out(out.cpu(), ref, mag)
    R.assert_state(fin.cpu(), final, smag)


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_masked_time_steps_of_single_tokens(dims, dtype):
    P, N = dims
    H, reqs, T = 2, 16, 5
    g = torch.Generator().manual_seed(103)
    c = masked_steps(g, reqs * T, H, P, N)
    pool = rand(g, reqs, H, N, P, dtype=dtype)
    ref, final, mag, smag = scan_ref(c, pool, [T] * reqs)
    d = {k: v.unflatten(0, (reqs, T)) if k in ("x", "B", "C", "z", "dt") else v for k, v in on_gpu(c).items()}
    a, kw = scan_args(d)
    pd = pool.cuda()
    out = K().ssm_decode(*a, pd, torch.arange(reqs, dtype=torch.int32).cuda(), **kw)
    R.assert_scan_out(out.cpu().flatten(0, 1), ref, mag)
    R.assert_state(pd.cpu(), final, smag)


# ---------------------------------------------------------------------------
# calls on a given stream beside work that is still queued on the current one

def stream_calls(seed):
    """name -> call(stream, **inputs) -> outputs, with two sets of inputs."""
    k = K()
    g = torch.Generator().manual_seed(seed)
    w, rw = rand(g, 520, 4).cuda(), rand(g, 520).cuda()
    idx = torch.tensor([3, -1, 0], dtype=torch.int32).cuda()
    scan = on_gpu(scan_case(g, 2048, 2, 1, 128, 128, z=False, softplus=False, skip=False))
    step = on_gpu(scan_case(g, 6, 4, 1, 64, 128, z=True, softplus=True, skip=True))
    step = {n: v.unflatten(0, (3, 2)) if n in ("x", "B", "C", "z", "dt") else v for n, v in step.items()}
    s_a, s_kw = scan_args(scan)
    t_a, t_kw = scan_args(step)
    rows, states = rand(g, 5, 3, 520).cuda(), rand(g, 5, 4, 128, 64, dtype=torch.float32).cuda()
    cu = offsets([2048]).cuda()
    two = lambda *shape: [rand(g, *shape).cuda() for _ in range(2)]
    return {
        "conv": (two(2048, 520), lambda s, x: k.conv_prefill(x, w, stream=s)),
        "conv_step": (two(3, 2, 520), lambda s, x: [k.conv_decode(x, w, None, rows, idx, stream=s)]),
        "scan": (two(2048, 2, 128), lambda s, x: k.ssm_prefill(x, *s_a[1:], **s_kw, cu_seqlens=cu, stream=s)),
        "scan_step": (two(3, 2, 4, 64), lambda s, x: [k.ssm_decode(x, *t_a[1:], states, idx, **t_kw, stream=s)]),
        "norm": (two(2048, 520), lambda s, x: k.add_rmsnorm(x, rw, residual=x, out_dtype=torch.float8_e4m3fn,
                                                            scale_group=128, stream=s)),
    }, [rows, states]


def slow(n=24):
    a = torch.ones(8192, 8192, dtype=BF, device="cuda")
    for _ in range(n):
        a @ a


def as_bytes(outs):
    return [t.contiguous().view(torch.uint8) for t in outs]


@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "norm"])
def test_results_on_a_given_stream_are_not_memory_that_queued_work_still_writes(name):
    calls, pools = stream_calls(111)
    (x, _), call = calls[name]
    start = [p.clone() for p in pools]
    want = [t.clone() for t in as_bytes(call(None, x))]
    workspace = 2048 // 64 * 2 * (128 * 128 + 1) * 4
    side = torch.cuda.Stream()
    slow(2)
    for p, s in zip(pools, start):
        p.copy_(s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    slow()
    for size in [t.numel() for t in want] + [workspace // n for n in (1, 2, 4, 8, 16)]:
        # freed with the fill still queued
        junk = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
        for t in junk:
            t.fill_(0xff)
        del junk, t
    got = call(side, x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(as_bytes(got), want))


@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "norm"])
def test_results_of_a_given_stream_stay_while_the_current_one_reads_them(name):
    calls, pools = stream_calls(112)
    (x, other), call = calls[name]
    start = [p.clone() for p in pools]
    want = [t.clone() for t in as_bytes(call(None, x))]
    for p, s in zip(pools, start):
        p.copy_(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = as_bytes(call(side, x))
    torch.cuda.current_stream().wait_stream(side)
    slow()
    kept = [t.clone() for t in got]
    del got
    more = [call(side, other) for _ in range(3)]
    torch.cuda.synchronize()
    del more
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


# ---------------------------------------------------------------------------
# a head that keeps nothing

@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [0, 64])
def test_a_head_with_an_infinite_rate_keeps_its_last_token_alone(dims, piece):
    P, N = dims
    lens, H = [37, 1, 70, 0, 64, 130], 2
    g = torch.Generator().manual_seed(121)
    c = scan_case(g, sum(lens), H, 1, P, N, z=False, softplus=True, skip=True)
    c["A"][1] = -INF
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    assert torch.isfinite(ref).all() and torch.isfinite(final).all()
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=s0.cuda(), piece_tokens=piece)
    R.assert_scan_out(out.cpu(), ref, mag)
    R.assert_state(fin.cpu(), final, smag)


# ---------------------------------------------------------------------------
# the scan is linear in x and the initial state: their scale leaves the relative
# errors as they are, up to near the largest float

@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [0, 64])
@pytest.mark.parametrize("power", [112, -80])
def test_states_far_from_one(dims, piece, power):
    P, N = dims
    lens, H = [150, 33, 0, 90], 2
    g = torch.Generator().manual_seed(131)
    c = scan_case(g, sum(lens), H, 1, P, N, z=True, softplus=True, skip=True)
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    far = 2.0 ** power
    c["x"] = c["x"] * far
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=(s0 * far).cuda(),
                               piece_tokens=piece)
    R.assert_scan_out(out.cpu().to(R.F64) / far, ref, mag)
    R.assert_state(fin.cpu().to(R.F64) / far, final, smag)


# ---------------------------------------------------------------------------
# offsets that break the contract (their arithmetic is swept on the CPU by
# test_layer_spans.py)

def guarded(*shape, dtype=BF):
    """A tensor inside a larger one of sentinels, and a check that they are whole."""
    n, pad = torch.Size(shape).numel(), 1 << 14
    wide = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")

    def whole():
        return bool((wide[:pad] == 7.0).all()) and bool((wide[pad + n:] == 7.0).all())

    return wide[pad:pad + n].view(shape), whole


@pytest.mark.parametrize("bad", [[-5, 40, 20, 1000], [10, 5, 90, 91], [0, 1 << 30, 3, 90], [90, 90, 90, 90],
                                 [0, 90, 0, 90], [200, -200, 150, -1], [-(1 << 31), (1 << 31) - 1, 0, 64]], ids=str)
@pytest.mark.parametrize("cu", [torch.int32, torch.int64])
def test_bad_offsets_write_inside_the_buffers(bad, cu):
    k = K()
    H, G, P, N, T, D = 2, 1, 64, 64, 200, 64
    g = torch.Generator().manual_seed(141)
    c = scan_case(g, T, H, G, P, N, z=True, softplus=True, skip=True)
    a, kw = scan_args(on_gpu(c))
    off = torch.tensor(bad, dtype=cu).cuda()
    s0 = rand(g, 3, H, N, P, dtype=torch.float32).cuda()
    for piece in (0, 64, 128):
        out, out_whole = guarded(T, H, P)
        fin, fin_whole = guarded(3, H, N, P, dtype=torch.float32)
        ws, ws_whole = guarded(((T // 64 + 3) * H * (N * P + 1) + 3) // 4 * 4, dtype=torch.float32)
        k.ssm_prefill(*a, **kw, cu_seqlens=off, piece_tokens=piece, initial_state=s0, out=out, final_state=fin, workspace=ws)
        assert out_whole() and fin_whole() and ws_whole()
    x, w, r0 = rand(g, T, D).cuda(), rand(g, D, 4).cuda(), rand(g, 3, 3, D).cuda()
    out, out_whole = guarded(T, D)
    fin, fin_whole = guarded(3, 3, D)
    k.conv_prefill(x, w, cu_seqlens=off, initial_state=r0, out=out, final_state=fin)
    assert out_whole() and fin_whole()


# ---------------------------------------------------------------------------
# accuracy in the mean, and calls that the other files do not make

@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [0, 64, 256])
def test_outputs_are_two_roundings_off_in_the_mean(dims, piece):
    # an output's own rounding and one of each term (of a score or of the state):
    # independent, each uniform over half a step to either side, 2^-8 of the value
    # at most, so 2^-8 / sqrt(3) each in the mean square
    P, N = dims
    lens, H = [700, 64, 1, 300, 900], 2
    g = torch.Generator().manual_seed(151)
    c = scan_case(g, sum(lens), H, 1, P, N, z=True, softplus=True, skip=True)
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, *_ = scan_ref(c, s0, lens)
    a, kw = scan_args(on_gpu(c))
    out, _ = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=s0.cuda(), piece_tokens=piece)
    rel = ((out.cpu().to(R.F64) - ref).norm() / ref.norm()).item()
    assert rel <= 2.0 ** 0.5 * R.BF16 / 3.0 ** 0.5, rel


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [0, 64, 192])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_states_updated_in_place_with_rows_behind_the_last_sequence(dims, piece, dtype):
    P, N = dims
    lens, H, tail = [300, 0, 65, 64, 1], 4, 9
    g = torch.Generator().manual_seed(152)
    c = scan_case(g, sum(lens), H, 2, P, N, z=True, softplus=True, skip=False)
    s0 = rand(g, len(lens), H, N, P, dtype=dtype)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    for k in ("x", "B", "C", "z", "dt"):
        c[k] = torch.cat([c[k], torch.full((tail, *c[k].shape[1:]), float("nan"), dtype=c[k].dtype)])
    a, kw = scan_args(on_gpu(c, True))
    state = s0.cuda()
    out = torch.full((sum(lens) + tail, H, P), 7.0, dtype=BF, device="cuda")
    _, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=state, final_state=state, out=out,
                             piece_tokens=piece)
    assert fin is state and (out[sum(lens):] == 7.0).all()
    R.assert_scan_out(out[:sum(lens)].cpu(), ref, mag)
    R.assert_state(fin.cpu(), final, smag)
    assert torch.equal(fin[1].cpu(), s0[1])


@pytest.mark.parametrize("T", [1, 4, 7])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_ssm_decode_may_overwrite_its_input(T, dtype):
    k = K()
    H, P, N, reqs = 4, 128, 64, 3
    g = torch.Generator().manual_seed(153)
    c = on_gpu(scan_case(g, reqs * T, H, 2, P, N, z=True, softplus=True, skip=True))
    c = {n: v.unflatten(0, (reqs, T)) if n in ("x", "B", "C", "z", "dt") else v for n, v in c.items()}
    a, kw = scan_args(c)
    pool = rand(g, reqs, H, N, P, dtype=dtype)
    idx = torch.tensor([2, -1, 0], dtype=torch.int32).cuda()
    p1, p2 = pool.cuda(), pool.cuda()
    want = k.ssm_decode(*a, p1, idx, **kw)
    x = a[0].clone()
    got = k.ssm_decode(x, *a[1:], p2, idx, **kw, out=x)
    assert got is x and torch.equal(got, want) and torch.equal(p1, p2)
    wide = torch.zeros(reqs, T, H * P + 16, dtype=BF, device="cuda")
    x = wide[..., 8:8 + H * P].unflatten(-1, (H, P))  # rows of a wider buffer
    x.copy_(a[0])
    k.ssm_decode(x, *a[1:], pool.cuda(), idx, **kw, out=x)
    assert torch.equal(x, want) and not wide[..., :8].any() and not wide[..., -8:].any()


def test_empty_fixed_batches_and_single_rows():
    k = K()
    s0 = torch.randn(2, 2, 64, 64, device="cuda")
    e = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")
    out, fin = k.ssm_prefill(e(2, 0, 2, 64), e(2, 0, 2, dtype=torch.float32), e(2, dtype=torch.float32),
                             e(2, 0, 1, 64), e(2, 0, 1, 64), initial_state=s0)
    assert out.shape == (2, 0, 2, 64) and torch.equal(fin, s0)
    r0 = torch.randn(2, 3, 16, device="cuda").to(BF)
    out, fin = k.conv_prefill(e(2, 0, 16), e(16, 4), initial_state=r0)
    assert out.shape == (2, 0, 16) and torch.equal(fin, r0)
    g = torch.Generator().manual_seed(154)
    x, w = rand(g, 264), rand(g, 264)
    y, _, s = k.add_rmsnorm(x.cuda(), w.cuda(), out_dtype=torch.float8_e4m3fn, scale_group=128)
    assert y.shape == (264,) and s.shape == (3,)
    R.assert_norm(y.cpu()[None], s.cpu()[None], R.norm(x[None], None, w, 1e-6)[0], 128)


def test_q_k_and_v_from_columns_of_one_projection():
    # three convolutions of a row's columns give the packed tensors that the
    # recurrence takes, bit for bit those of one convolution over the whole row
    k = K()
    H, D, T = 2, 128, 150
    g = torch.Generator().manual_seed(155)
    u, w = rand(g, T, 3 * H * D + 8).cuda(), rand(g, 3 * H * D, 4, scale=0.4).cuda()
    whole, _ = k.conv_prefill(u[:, :3 * H * D], w)
    parts = []
    for i in range(3):
        cols = slice(i * H * D, (i + 1) * H * D)
        y, _ = k.conv_prefill(u[:, cols], w[cols])
        assert y.is_contiguous() and torch.equal(y, whole[:, cols])
        parts.append(y.unflatten(-1, (H, D)))
    decay, beta = torch.full((T, H, D), -0.1, device="cuda"), torch.full((T, H), 0.5, device="cuda")
    out, _ = k.prefill(*parts, decay, beta, qk_l2norm=True)
    assert out.shape == (T, H, D) and torch.isfinite(out).all()


@pytest.mark.parametrize("name", ["conv", "scan", "norm"])
def test_a_given_stream_inside_a_capture(name):
    # forked from the captured stream and joined to it again; results and
    # workspaces come out of the graph's pool
    calls, _ = stream_calls(113)
    (x, other), call = calls[name]
    want = {i: [t.clone() for t in as_bytes(call(None, v))] for i, v in enumerate((x, other))}
    graph, side, into = torch.cuda.CUDAGraph(), torch.cuda.Stream(), x.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side, into)
        torch.cuda.current_stream().wait_stream(side)
    for i in (1, 0, 1, 0):
        into.copy_((x, other)[i])
        for t in got:
            t.view(torch.uint8).fill_(0x55)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(as_bytes(got), want[i]))
