"""Offsets that are no offsets (decreasing, negative, past the tokens) reach nothing outside of the tensors: they are
taken between 0 and the token count, and a sequence that would end ahead of its start is empty."""
import pytest
import torch

from test_attn_gpu import BF, attn, rand

pytestmark = pytest.mark.gpu
SENTINEL = 12345.0
BAD = [[0, 150, 20, 100], [0, 10 ** 6, 5], [-7, 60, 60, 199], [50, 40, 30, 20, 10], [0, 2 ** 31 - 1, -2 ** 31, 200], [300, 400]]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("cu", BAD, ids=str)
def test_prompts(cu, dtype, many):
    T, H, D, pad = 200, 2, 64, 64
    if many:  # (more sequences than lanes)
        cu = cu[:-1] + [cu[-1]] * 70 + cu[::-1] + cu
    g = torch.Generator().manual_seed(len(cu))
    wide = rand(g, T + 2 * pad, 3 * H * D)
    wide[:pad] = wide[-pad:] = float("nan")
    rows = wide.cuda()[pad:-pad]
    q, k, v = (rows[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    outer = torch.full((T + 2 * pad, H, D), SENTINEL, dtype=BF, device="cuda")
    lses = torch.full((T + 2 * pad, H), SENTINEL, device="cuda")
    attn().prefill(q, k, v, cu_seqlens=torch.tensor(cu, dtype=dtype).cuda(), out=outer[pad:-pad], lse=lses[pad:-pad])
    assert (outer[:pad] == SENTINEL).all() and (outer[-pad:] == SENTINEL).all()
    assert (lses[:pad] == SENTINEL).all() and (lses[-pad:] == SENTINEL).all()
    assert torch.isfinite(outer).all() and torch.isfinite(lses).all()


@pytest.mark.parametrize("cu", BAD, ids=str)
def test_pages(cu):
    T, size, W, F, pad = 200, 16, 8, 40, 64
    N = len(cu) - 1
    lens = torch.tensor([0, 5, 2 ** 31 - 1, 17][:N], dtype=torch.int32).cuda()
    table = torch.full((N + 2 * pad, W), 77, dtype=torch.int32).cuda()
    slots = torch.full((T + 2 * pad,), 777, dtype=torch.int64).cuda()
    free = torch.arange(F, dtype=torch.int32).cuda()
    for head in (0, 3, -5, 2 ** 31 - 1):
        _, lens_out, head_out = attn().assign_pages(lens, table[pad:-pad], free, torch.tensor([head], dtype=torch.int32).cuda(),
                                                    page_size=size, cu_seqlens=torch.tensor(cu, dtype=torch.int64).cuda(),
                                                    slots=slots[pad:-pad])
        assert (table[:pad] == 77).all() and (table[-pad:] == 77).all()
        assert (slots[:pad] == 777).all() and (slots[-pad:] == 777).all()
        got = slots[pad:-pad]
        assert ((got == -1) | ((got >= 0) & (got < 78 * size))).all()
        inner = table[pad:-pad]
        assert ((inner == -1) | (inner == 77) | ((inner >= 0) & (inner < F))).all()
        assert (lens_out >= lens).all() and int(head_out) >= head
