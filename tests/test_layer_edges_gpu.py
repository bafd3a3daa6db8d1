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
