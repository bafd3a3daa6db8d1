"""The layer operators on the GPU -- short causal convolution, selective state
space scan, residual RMS norm -- against their formulas in 64 bits
(tests/layer_reference.py, which states the error bounds)."""
import pytest
import torch

import layer_reference as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def K():
    import kda_gated_delta_chunked_amd as k
    k.load_library()
    return k


def cuda(t):
    return None if t is None else t.cuda()


def rand(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def offsets(lens, dtype=torch.int32):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    return cu.to(dtype)


def padded_rows(t, extra):
    """The same rows inside wider ones, the rest NaN: [T, row] views of
    [T, row + 2 extra], `extra` columns in."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 2 * extra), NAN, dtype=t.dtype, device=t.device)
    view = wide[..., extra:extra + t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# convolution

LENS = [[1], [2], [7], [37], [64, 1], [5, 0, 1, 2, 130, 3], [0, 0], [700, 33, 300]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("width,dim,bias,act,init,strided,cu", [
    (4, 64, True, "silu", True, False, torch.int32), (4, 520, False, "none", False, True, torch.int64),
    (3, 1032, True, "silu", True, True, torch.int32), (2, 8, False, "silu", True, False, torch.int64)])
def test_conv_prefill(lens, width, dim, bias, act, init, strided, cu):
    g = torch.Generator().manual_seed(sum(lens) * 8 + width)
    T, N = sum(lens), len(lens)
    x, w = rand(g, T, dim), rand(g, dim, width, scale=0.5)
    b = rand(g, dim, scale=0.3) if bias else None
    s0 = rand(g, N, width - 1, dim) if init else torch.zeros(N, width - 1, dim, dtype=BF)
    ref, final, mag = R.conv(x, w, b, act, s0, lens)
    # rows behind the last sequence belong to nobody
    tail = torch.full((3, dim), NAN, dtype=BF)
    xd, out = torch.cat([x, tail]).cuda(), torch.full((T + 3, dim), 7.0, dtype=BF, device="cuda")
    if strided:
        xd, out = padded_rows(xd, 16), padded_rows(out, 8)
    got, fin = K().conv_prefill(xd, w.cuda(), cuda(b), cu_seqlens=offsets(lens, cu).cuda(),
                                initial_state=s0.cuda() if init else None, activation=act, out=out)
    torch.cuda.synchronize()
    assert got is out
    R.assert_conv(got[:T].cpu(), ref, mag, act, f"{lens}")
    assert (got[T:] == 7.0).all()
    assert torch.equal(fin.cpu().to(R.F64), final)


@pytest.mark.parametrize("T", [1, 3, 70])
def test_conv_prefill_fixed_layout_in_place_state(T):
    g = torch.Generator().manual_seed(T)
    x, w, s0 = rand(g, 3, T, 96), rand(g, 96, 4), rand(g, 3, 3, 96)
    ref, final, mag = R.conv(x.view(-1, 96), w, None, "silu", s0, [T] * 3)
    state = s0.cuda()
    out, fin = K().conv_prefill(x.cuda(), w.cuda(), initial_state=state, final_state=state)
    assert fin is state and out.shape == x.shape
    R.assert_conv(out.cpu().view(-1, 96), ref, mag, "silu")
    assert torch.equal(state.cpu().to(R.F64), final)


def test_conv_special_values_stay_in_their_sequence_and_channel():
    lens, dim = [40, 3, 90], 64
    g = torch.Generator().manual_seed(3)
    x, w = rand(g, sum(lens), dim), rand(g, dim, 4)
    x[39, 5], x[41, 6], x[60, 7] = NAN, float("inf"), -float("inf")
    ref, final, _ = R.conv(x, w, None, "none", torch.zeros(3, 3, dim, dtype=BF), lens)
    out, fin = K().conv_prefill(x.cuda(), w.cuda(), cu_seqlens=offsets(lens).cuda(), activation="none")
    out = out.cpu().to(R.F64)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(out), fine)
    assert torch.allclose(out[fine], ref[fine], rtol=2 * R.BF16, atol=1e-4)
    assert torch.equal(torch.isnan(fin.cpu()), torch.isnan(final))


@pytest.mark.parametrize("reqs,T,dim,width,strided", [(1, 1, 64, 4, False), (5, 1, 1032, 4, True), (7, 2, 520, 3, False),
                                                      (3, 6, 8, 2, True), (66, 1, 96, 4, False)])
def test_conv_decode(reqs, T, dim, width, strided):
    g = torch.Generator().manual_seed(reqs)
    P = reqs + 2
    pool, x = rand(g, P, width - 1, dim), rand(g, reqs, T, dim)
    w, b = rand(g, dim, width), rand(g, dim)
    idx = torch.randperm(P, generator=g)[:reqs].to(torch.int32)
    if reqs > 2:
        idx[1], idx[2] = -1, P + 4
    live = [n for n in range(reqs) if 0 <= idx[n] < P]
    want_pool = pool.clone()
    out_d = torch.full(x.shape, NAN, dtype=BF, device="cuda")
    xd, pd = x.cuda(), pool.cuda()
    if strided:
        xd, out_d = padded_rows(xd, 8), padded_rows(out_d, 24)
    out = K().conv_decode(xd, w.cuda(), b.cuda(), pd, idx.cuda(), out=out_d).cpu()
    for n in range(reqs):
        if n not in live:
            assert not out[n].any()
            continue
        ref, final, mag = R.conv(x[n], w, b, "silu", pool[idx[n]][None], [T])
        R.assert_conv(out[n], ref, mag, "silu", f"request {n}")
        want_pool[idx[n]] = final[0].to(BF)
    assert torch.equal(pd.cpu(), want_pool)


def test_conv_decode_may_overwrite_its_input():
    g = torch.Generator().manual_seed(8)
    pool, x, w = rand(g, 4, 3, 128), rand(g, 4, 3, 128), rand(g, 128, 4)
    idx = torch.arange(4, dtype=torch.int32).cuda()
    a = K().conv_decode(x.cuda(), w.cuda(), None, pool.cuda(), idx)
    xd = x.cuda()
    b = K().conv_decode(xd, w.cuda(), None, pool.cuda(), idx, out=xd)
    assert b is xd and torch.equal(a, b)


# ---------------------------------------------------------------------------
# scan

DIMS = [(128, 128), (64, 128), (128, 64), (64, 64)]  # (head_dim, d_state)


def scan_case(g, T, H, G, P, N, *, z, softplus, skip, slow=False):
    c = dict(x=rand(g, T, H, P, scale=0.7), B=rand(g, T, G, N, scale=0.7), C=rand(g, T, G, N, scale=0.7),
             z=rand(g, T, H, P) if z else None, A=-(torch.rand(H, generator=g) * 15 + 1) * (1e-3 if slow else 1.0),
             D=torch.rand(H, generator=g) if skip else None)
    if softplus:
        c |= dict(dt=torch.randn(T, H, generator=g), dt_bias=torch.randn(H, generator=g) - 3, dt_softplus=True)
    else:
        c |= dict(dt=torch.rand(T, H, generator=g) * 0.1, dt_bias=None, dt_softplus=False)
    return c


def scan_ref(c, states, lens):
    step = R.steps(c["dt"], c["dt_bias"], c["dt_softplus"])
    return R.scan(c["x"], step, c["A"], c["B"], c["C"], c["D"], c["z"], states, lens)


def on_gpu(c, strided=False):
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}
    if strided:
        for k in ("x", "B", "C", "z"):
            if d[k] is not None:
                d[k] = padded_rows(d[k].flatten(-2), 8).unflatten(-1, d[k].shape[-2:])
    return d


def scan_args(d):
    return [d[k] for k in ("x", "dt", "A", "B", "C")], {k: d[k] for k in ("D", "z", "dt_bias", "dt_softplus")}


SCAN_LENS = [[1], [2], [63], [64], [65], [37, 0, 1, 130], [0, 0], [200, 5, 128, 0, 300], [1] * 70]


@pytest.mark.parametrize("lens", SCAN_LENS, ids=str)
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("H,G,z,softplus,skip,init,strided,slow", [
    (3, 1, True, True, True, True, False, False), (4, 2, False, False, False, False, True, False),
    (2, 2, True, False, True, True, True, True)])
def test_ssm_prefill(lens, dims, H, G, z, softplus, skip, init, strided, slow):
    P, N = dims
    T = sum(lens)
    g = torch.Generator().manual_seed(T * 4 + H)
    c = scan_case(g, T, H, G, P, N, z=z, softplus=softplus, skip=skip, slow=slow)
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    states = s0 if init else torch.zeros_like(s0)
    ref, final, mag, smag = scan_ref(c, states, lens)
    # rows behind the last sequence: NaN going in, left alone coming out
    for k in ("x", "B", "C", "z", "dt"):
        if c[k] is not None:
            c[k] = torch.cat([c[k], torch.full((5, *c[k].shape[1:]), NAN, dtype=c[k].dtype)])
    d = on_gpu(c, strided)
    out = torch.full((T + 5, H, P), 7.0, dtype=BF, device="cuda")
    a, kw = scan_args(d)
    got, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=s0.cuda() if init else None,
                               out=out)
    torch.cuda.synchronize()
    assert (got[T:] == 7.0).all()
    R.assert_scan_out(got[:T].cpu(), ref, mag, f"{lens}")
    R.assert_state(fin.cpu(), final, smag, f"{lens}")


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("piece", [64, 128, 192, 256])
def test_ssm_prefill_in_pieces(dims, piece):
    P, N = dims
    lens, H, G = [piece * 3 + 7, 0, piece, 1, piece + 1, piece * 4], 2, 1
    g = torch.Generator().manual_seed(piece)
    c = scan_case(g, sum(lens), H, G, P, N, z=True, softplus=True, skip=True)
    s0 = rand(g, len(lens), H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    a, kw = scan_args(on_gpu(c))
    state = s0.cuda()  # in place: later pieces must not see the final state
    got, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda(), initial_state=state, final_state=state,
                               piece_tokens=piece)
    R.assert_scan_out(got.cpu(), ref, mag, f"{piece}")
    R.assert_state(fin.cpu(), final, smag, f"{piece}")


def test_ssm_prefill_fixed_layout_bf16_state_int64_offsets():
    g = torch.Generator().manual_seed(5)
    N_seq, T, H, G, P, N = 3, 100, 2, 1, 128, 128
    c = scan_case(g, N_seq * T, H, G, P, N, z=False, softplus=True, skip=True)
    s0 = rand(g, N_seq, H, N, P)
    ref, final, mag, smag = scan_ref(c, s0, [T] * N_seq)
    d = on_gpu(c)
    a, kw = scan_args(d)
    packed, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets([T] * N_seq, torch.int64).cuda(),
                                  initial_state=s0.cuda())
    assert fin.dtype == BF
    R.assert_scan_out(packed.cpu(), ref, mag)
    R.assert_state(fin.cpu(), final, smag)
    f = {k: v.unflatten(0, (N_seq, T)) if torch.is_tensor(v) and v.dim() > 1 else v for k, v in d.items()}
    a, kw = scan_args(f)
    out, fin2 = K().ssm_prefill(*a, **kw, initial_state=s0.cuda())
    assert torch.equal(out.flatten(0, 1), packed) and torch.equal(fin2, fin)


def test_ssm_special_values_stay_in_their_sequence():
    # a NaN and infinities in one sequence leave the neighbours' results alone,
    # also where one chunk's rows are followed by them
    lens, H, G, P, N = [30, 50, 70], 2, 1, 64, 64
    g = torch.Generator().manual_seed(6)
    c = scan_case(g, sum(lens), H, G, P, N, z=False, softplus=False, skip=False)
    clean = scan_ref(c, torch.zeros(3, H, N, P), lens)
    c["x"][40], c["B"][33], c["dt"][35] = float("inf"), NAN, NAN
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, cu_seqlens=offsets(lens).cuda())
    out, fin = out.cpu(), fin.cpu()
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[30:80] = False
    R.assert_scan_out(out[keep], clean[0][keep], clean[2][keep])
    R.assert_state(fin[[0, 2]], clean[1][[0, 2]], clean[3][[0, 2]])
    assert torch.isnan(out[40:80].float()).all() and torch.isnan(fin[1]).all()
    R.assert_scan_out(out[30:33], clean[0][30:33], clean[2][30:33])


@pytest.mark.parametrize("rate", [0.0, 30.0, 1e4])
def test_ssm_extreme_decays(rate):
    # no decay at all, a chunk's product below the smallest float, and nothing kept
    lens, H, G, P, N = [150], 2, 1, 128, 64
    g = torch.Generator().manual_seed(7)
    c = scan_case(g, 150, H, G, P, N, z=False, softplus=False, skip=True)
    c["A"] = torch.full((H,), -rate)
    s0 = rand(g, 1, H, N, P, dtype=torch.float32)
    ref, final, mag, smag = scan_ref(c, s0, lens)
    a, kw = scan_args(on_gpu(c))
    out, fin = K().ssm_prefill(*a, **kw, initial_state=s0.cuda())
    R.assert_scan_out(out.cpu(), ref, mag, f"{rate}")
    R.assert_state(fin.cpu(), final, smag, f"{rate}")


def test_ssm_bad_offsets_stay_inside_the_buffers():
    # offsets past the batch, negative and decreasing ones: clamped on the device
    H, G, P, N, T = 2, 1, 64, 64, 90
    g = torch.Generator().manual_seed(9)
    c = scan_case(g, T, H, G, P, N, z=True, softplus=True, skip=True)
    a, kw = scan_args(on_gpu(c))
    x = rand(g, T, 64).cuda()
    w = rand(g, 64, 4).cuda()
    for bad in ([-5, 40, 20, 1000], [10, 5, 90, 91], [0, 1 << 30, 3, 90], [90, 90, 90, 90]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        K().ssm_prefill(*a, **kw, cu_seqlens=cu)
        K().ssm_prefill(*a, **kw, cu_seqlens=cu, piece_tokens=64)
        K().conv_prefill(x, w, cu_seqlens=cu)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("reqs,T,H,G,z,softplus,skip,strided,dtype", [
    (1, 1, 1, 1, True, True, True, False, torch.float32), (5, 1, 3, 1, False, False, False, True, BF),
    (9, 4, 4, 2, True, True, True, True, torch.float32), (67, 1, 2, 2, True, True, True, False, BF)])
def test_ssm_decode(dims, reqs, T, H, G, z, softplus, skip, strided, dtype):
    P, N = dims
    g = torch.Generator().manual_seed(reqs + T)
    size = reqs + 2
    c = scan_case(g, reqs * T, H, G, P, N, z=z, softplus=softplus, skip=skip)
    pool = rand(g, size, H, N, P, dtype=dtype)
    idx = torch.randperm(size, generator=g)[:reqs].to(torch.int32)
    if reqs > 2:
        idx[1], idx[2] = -3, size
    live = torch.tensor([n for n in range(reqs) if 0 <= idx[n] < size])
    ref, final, mag, smag = scan_ref(c, pool[idx.clamp(0, size - 1).long()], [T] * reqs)
    d = on_gpu(c, strided)
    d = {k: v.unflatten(0, (reqs, T)) if k in ("x", "B", "C", "z", "dt") and v is not None else v
         for k, v in d.items()}
    a, kw = scan_args(d)
    pd = pool.cuda()
    out = torch.full((reqs, T, H, P), NAN, dtype=BF, device="cuda")
    got = K().ssm_decode(*a, pd, idx.cuda(), **kw, out=out).cpu()
    rows = ref.unflatten(0, (reqs, T))
    R.assert_scan_out(got[live], rows[live], mag.unflatten(0, (reqs, T))[live])
    gone = [n for n in range(reqs) if n not in live.tolist()]
    assert not got[gone].any()
    at = idx[live].long()
    R.assert_state(pd.cpu()[at], final[live], smag[live])
    rest = [i for i in range(size) if i not in at.tolist()]
    assert torch.equal(pd.cpu()[rest], pool[rest])


# ---------------------------------------------------------------------------
# norm

@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 128), (5, 136), (2, 1536), (70, 520), (9, 2048), (4, 2056), (3, 4096),
                                      (2, 8200), (2, 16384), (1000, 128)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out,group", [(BF, 0), (torch.float8_e4m3fn, 0), (torch.float8_e4m3fn, 128)])
def test_add_rmsnorm(rows, dim, residual, out, group):
    g = torch.Generator().manual_seed(rows + dim)
    x, w = rand(g, rows, dim, scale=3.0), rand(g, dim, scale=0.2) + 1
    res = rand(g, rows, dim) if residual else None
    if rows > 2:
        x[1] = 0
        if res is not None:
            res[1] = 0
    ref, s = R.norm(x, res, w, 1e-5)
    y, r_out, scales = K().add_rmsnorm(padded_rows(x.cuda(), 8), w.cuda(), residual=cuda(res), eps=1e-5,
                                       out_dtype=out, scale_group=group)
    R.assert_norm(y.cpu(), cuda(scales) if scales is None else scales.cpu(), ref, group, f"{rows}x{dim}")
    if residual:
        assert torch.equal(r_out.cpu(), (x.float() + res.float()).to(BF))
    else:
        assert r_out is None


def test_add_rmsnorm_in_place_and_without_residual_out():
    g = torch.Generator().manual_seed(1)
    x, res, w = rand(g, 6, 256), rand(g, 6, 256), rand(g, 256)
    y, r, _ = K().add_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda())
    xd, rd = x.cuda(), res.cuda()
    y2, r2, _ = K().add_rmsnorm(xd, w.cuda(), residual=rd, residual_out=rd, out=xd)
    assert y2 is xd and r2 is rd and torch.equal(y, y2) and torch.equal(r, r2)
    y3, r3, _ = K().add_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), residual_out=False)
    assert r3 is None and torch.equal(y, y3)


@pytest.mark.parametrize("dim", [128, 1536, 4096])
@pytest.mark.parametrize("out,group", [(BF, 0), (torch.float8_e4m3fn, 0), (torch.float8_e4m3fn, 128)])
def test_add_rmsnorm_special_rows(dim, out, group):
    # NaN, infinity, tiny and huge rows do what fp32 arithmetic does, row by row
    g = torch.Generator().manual_seed(2)
    x, w = rand(g, 6, dim), rand(g, dim)
    x[0, 7], x[1, 3], x[2] = NAN, float("inf"), 1e-38
    x[3], x[4] = 3e38, 0
    xf = x.float()
    y = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    got, _, scales = K().add_rmsnorm(x.cuda(), w.cuda(), out_dtype=out, scale_group=group)
    got = got.cpu()
    assert torch.isnan(got[0].float()).all() and torch.isnan(got[1, 3].float())
    if scales is None:
        assert not got[1, 4:].float().any() and not got[3].float().any()
    else:
        s = scales.cpu()
        assert torch.isnan(s[0]).all() and torch.isnan(s[1, 0])
        if s.shape[1] > 1:
            assert (s[1, 1:] == 2.0 ** -126).all() and not got[1, 128:].float().any()
        assert (s[3] == 2.0 ** -126).all() and not got[3].float().any()
    fine = [2, 4, 5]
    ref, _ = R.norm(x[fine], None, w, 1e-6)
    R.assert_norm(got[fine], None if scales is None else scales.cpu()[fine], ref, group)
