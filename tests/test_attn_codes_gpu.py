"""The codes that the store of keys and values writes are those of the fp32 quotient x / scale, in
every bit: all finite bf16 numbers, zeros' signs included, over scales of many significands."""
import pytest
import torch

from test_attn_gpu import BF, E4M3, attn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def numbers():
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    return x[torch.isfinite(x.float())]


def scales(kind):
    g = torch.Generator().manual_seed(len(kind))
    if kind == "ordinary":
        s = torch.rand(512, generator=g) * 0.05 + 1e-4
        s[:8] = torch.tensor([1.0, 2.0, 0.5, 2.0 ** -20, 1.0 / 3, 0.1, 448.0, 7.0 / 448])
        return s
    if kind == "far":  # past what the corrected reciprocal takes, and close to it
        return torch.tensor([2.0 ** -60, 2.0 ** 60, 2.0 ** -61, 2.0 ** 61, 2.0 ** -126, 2.0 ** 126, 1e-30, 1e30])
    return ((torch.randint(0, 1 << 23, (1024,), generator=g) | 1).double() * 2.0 ** -23 + 1).float()  # significands


@pytest.mark.parametrize("kind", ["ordinary", "far", "significands"])
def test_codes_of_all_numbers(kind):
    x, s = numbers(), scales(kind)
    KV, D, size = len(s), 64, 16
    T = -(-len(x) // D)
    rows = torch.zeros(T * D, dtype=BF)
    rows[:len(x)] = x
    rows = rows.view(T, 1, D)
    want = (rows.float() / s[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
    pages = -(-T // size)
    kc, vc = (torch.zeros(pages, size, KV, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    k = rows.cuda().expand(T, KV, D).contiguous()
    sd = s.cuda()
    attn().store(k, -k, kc, vc, torch.arange(T, device="cuda"), k_scale=sd, v_scale=sd)
    got = kc.view(torch.uint8).flatten(0, 1)[:T].cpu()
    assert torch.equal(got, want), int((got != want).sum())
    got = vc.view(torch.uint8).flatten(0, 1)[:T].cpu()
    assert torch.equal(got, want ^ 0x80), int((got != want ^ 0x80).sum())
