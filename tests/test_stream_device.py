"""A stream belongs to the device of the tensors: every entry point with
``stream=`` refuses another device's before it allocates or enqueues anything."""
import inspect
from types import SimpleNamespace

import pytest
import torch

import kda_gated_delta_chunked_amd as K
from kda_gated_delta_chunked_amd import ops

BF = torch.bfloat16
ELSEWHERE = SimpleNamespace(device=torch.device("cuda", 1))  # (no handle: nothing may be enqueued on it)


def test_streams_are_compared_by_device():
    here = torch.device("cuda", 0)
    ops._check_stream(None, here)
    ops._check_stream(SimpleNamespace(device=here), here)
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        ops._check_stream(ELSEWHERE, here)


def calls():
    """entry point -> a call on small zeros"""
    e = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda:0")
    f32, i32 = torch.float32, torch.int32
    qkv = [e(1, 2, 1, 128) for _ in range(3)] + [e(1, 2, 1, 128, dtype=f32), e(1, 2, 1, dtype=f32)]
    pool, idx = e(1, 1, 128, 128, dtype=f32), e(1, dtype=i32)
    trace, accepted = e(1, 2, 1, 128, 128, dtype=f32), e(1, dtype=i32)
    x, w, rows, states = e(1, 4, 64), e(64, 4), e(1, 3, 64), e(1, 1, 64, 64, dtype=f32)
    scale = e(64)
    scan = [e(1, 4, 1, 64), e(1, 4, 1, dtype=f32), e(1, dtype=f32), e(1, 4, 1, 64), e(1, 4, 1, 64)]
    return {
        "prefill": lambda s: K.prefill(*qkv, stream=s),
        "decode": lambda s: K.decode(*qkv, pool, idx, stream=s),
        "decode_verify": lambda s: K.decode_verify(*qkv, pool, idx, stream=s),
        "decode_advance": lambda s: K.decode_advance(*qkv, pool, idx, accepted, stream=s),
        "decode_commit": lambda s: K.decode_commit(pool, idx, trace, accepted, stream=s),
        "conv_prefill": lambda s: K.conv_prefill(x, w, stream=s),
        "conv_decode": lambda s: K.conv_decode(x, w, None, rows, idx, stream=s),
        "ssm_prefill": lambda s: K.ssm_prefill(*scan, stream=s),
        "ssm_decode": lambda s: K.ssm_decode(*scan, states, idx, stream=s),
        "add_rmsnorm": lambda s: K.add_rmsnorm(x, scale, stream=s),
    }


NAMES = ["prefill", "decode", "decode_verify", "decode_advance", "decode_commit", "conv_prefill", "conv_decode",
         "ssm_prefill", "ssm_decode", "add_rmsnorm"]


def test_every_entry_point_is_covered():
    with_stream = {n for n in K.__all__ if inspect.isfunction(getattr(K, n)) and not n.endswith("_raw")
                   and "stream" in inspect.signature(getattr(K, n)).parameters}
    assert with_stream == set(NAMES)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_another_devices_stream_is_refused(name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    call = calls()[name]  # (it holds its tensors)
    side = torch.cuda.Stream(torch.device("cuda", 0))
    torch.cuda.synchronize()
    call(side)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(ELSEWHERE)
    torch.cuda.synchronize()
