"""The delta-rule entry points on a given stream beside work that is still
queued on the current one: what a call allocates is not memory that this work
still writes, and stays while the current stream reads it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, D = 2, 128


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(seed, *lead):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(*lead, H, D, generator=g) for _ in range(3))
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    decay = -torch.rand(*lead, H, D, generator=g) * 0.2
    beta = torch.rand(*lead, H, generator=g)
    return [t.cuda() for t in (q.to(BF), k.to(BF), v.to(BF), decay, beta)]


def calls():
    """name -> call(stream, seed) -> outputs, on inputs that are made before"""
    import kda_gated_delta_chunked_amd as K
    K.load_library()
    prompt = {s: inputs(s, 1, 2048) for s in (1, 2)}
    step = {s: inputs(s, 5, 3) for s in (1, 2)}
    g = torch.Generator().manual_seed(3)
    pool = torch.randn(6, H, D, D, generator=g).cuda()
    idx = torch.tensor([4, 0, -1, 2, 5], dtype=torch.int32).cuda()

    def decode(stream, seed):
        states = pools.pop()
        return [K.decode(*step[seed], states, idx, stream=stream)]

    pools = [pool.clone() for _ in range(8)]
    return {
        "prefill": lambda stream, seed: K.prefill(*prompt[seed], stream=stream),
        "prefill_one_launch": lambda stream, seed: K.prefill(*prompt[seed], variant="fused", stream=stream),
        "decode": decode,
        "decode_verify": lambda stream, seed: K.decode_verify(*step[seed], pool, idx, stream=stream),
    }, K


NAMES = ["prefill", "prefill_one_launch", "decode", "decode_verify"]


def slow(n=24):
    a = torch.ones(8192, 8192, dtype=BF, device="cuda")
    for _ in range(n):
        a @ a


def as_bytes(outs):
    return [t.contiguous().view(torch.uint8) for t in outs]


def assert_same(name, got, want):
    for a, b in zip(got, want):
        if name.startswith("decode"):  # the trace of an empty slot is left as it was
            a, b = a[[0, 1, 3, 4]], b[[0, 1, 3, 4]]
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_results_are_not_memory_that_queued_work_still_writes(name):
    table, K = calls()
    call = table[name]
    want = [t.clone() for t in as_bytes(call(None, 1))]
    sizes = [t.numel() for t in want]
    if name == "prefill":
        sizes.append(K.workspace_size(K.make_problem(1, 2048, H, scale=D ** -0.5)))
    side = torch.cuda.Stream()
    slow(2)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    slow()
    for size in sizes:
        # freed with the fill still queued
        junk = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
        for t in junk:
            t.fill_(0xff)
        del junk, t
    got = call(side, 1)
    torch.cuda.synchronize()
    assert_same(name, as_bytes(got), want)


@pytest.mark.parametrize("name", NAMES)
def test_results_stay_while_the_current_stream_reads_them(name):
    table, _ = calls()
    call = table[name]
    want = [t.clone() for t in as_bytes(call(None, 1))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = as_bytes(call(side, 1))
    torch.cuda.current_stream().wait_stream(side)
    slow()
    kept = [t.clone() for t in got]
    del got
    more = [call(side, 2) for _ in range(3)]
    torch.cuda.synchronize()
    del more
    assert_same(name, kept, want)
