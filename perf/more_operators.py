"""Cases of the operators of softmax attention beside the recurrent layers: causal
attention over prompts, attention of drafted tokens over a paged cache, the
cache's block tables and slots, and the store of keys and values into it.

``run`` computes a case with elementary torch operations where ``own`` is
false, and through the package's entry points where it is true.  ``exact``
gives the same results in 64 bits, one request after the other, from the
definition.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROWS = 1024       # query rows of the plain forms' blocks
GATHER = 1 << 29  # elements of a gathered block of keys


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a short prompt: latency
        dict(name="prompt_b1_t37_h4", op="prompt", lens="37", heads=4, kv=2, dim=64, sliced=False, lse=True),
        # six ragged prompts, 12 heads, out of one projection's rows
        dict(name="prompt_mixed6_h12", op="prompt", lens="1300,547,2048,963,271,3063", heads=12, kv=4, dim=128,
             sliced=True, lse=False),
        # 32 ragged prompts of 24 heads of 64 on two shared ones
        dict(name="prompt_ragged32_h24", op="prompt", count=32, lo=1, hi=4096, lens_seed=2003, heads=24, kv=2,
             dim=64, sliced=True, lse=False),
        # a prefill batch that fills the device
        dict(name="prompt_b8_t8192_h32", op="prompt", count=8, lo=8192, hi=8192, lens_seed=0, heads=32, kv=8,
             dim=128, sliced=False, lse=False),
        # four drafts in a row for each of nine requests on short pages: latency
        dict(name="drafts_n9_t4_h12", op="tokens", reqs=9, tokens=4, tree=False, lo=1, hi=600, lens_seed=7, heads=12,
             kv=2, dim=64, page=16, cache="bf16", empty=0, lse=True),
        # a decode step of 256 requests of all lengths
        dict(name="step_n256_h32", op="tokens", reqs=256, tokens=1, tree=False, lo=1, hi=8192, lens_seed=11, heads=32,
             kv=8, dim=128, page=64, cache="bf16", empty=4, lse=False),
        # the next token behind one long context
        dict(name="step_n1_c131072_h32", op="tokens", reqs=1, tokens=1, tree=False, lo=131072, hi=131072, lens_seed=0,
             heads=32, kv=8, dim=128, page=256, cache="bf16", empty=0, lse=False),
        # trees of 32 drafts over an 8-bit cache
        dict(name="tree_n32_t32_e4m3", op="tokens", reqs=32, tokens=32, tree=True, lo=1, hi=16384, lens_seed=13,
             heads=32, kv=4, dim=128, page=64, cache="e4m3", empty=1, lse=False),
        # keys and values of a decode step of 1024 requests
        dict(name="store_n1024", op="store", tokens=1024, kv=8, dim=128, page=64, cache="bf16", sliced=True, skip=16),
        # keys and values of a prefill batch, to 8 bits
        dict(name="store_65536_e4m3", op="store", tokens=65536, kv=8, dim=128, page=64, cache="e4m3", sliced=True,
             skip=0),
        # one more token for each of 1024 requests
        dict(name="pages_n1024", op="pages", count=1024, lo=1, hi=1, lens_seed=0, old=8192, page=64, empty=16),
        # pages and slots of 64 ragged prompts, some behind earlier ones
        dict(name="pages_ragged64", op="pages", count=64, lo=1, hi=8192, lens_seed=17, old=4096, page=16, empty=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _yes(rng):
    return rng.random() < 0.5


def _draw_lens(rng, most):
    """One to 64 sequences: equal lengths, or ragged ones from a single token up."""
    count = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, most)
    return dict(count=count, lo=hi if _yes(rng) else 1, hi=hi, lens_seed=rng.randrange(1 << 20))


def _draw_heads(rng):
    kv = _log_int(rng, 1, 16)
    return dict(heads=kv * _log_int(rng, 1, 16), kv=kv, dim=rng.choice([64, 128]))


def _draw_one(rng):
    op = rng.choice(["prompt", "prompt", "tokens", "tokens", "store", "pages"])
    if op == "prompt":
        return dict(op=op, **_draw_lens(rng, 16384), **_draw_heads(rng), sliced=_yes(rng), lse=_yes(rng))
    if op == "tokens":
        reqs, hi = _log_int(rng, 1, 1024), _log_int(rng, 1, 131072)
        tree = _yes(rng)
        empty = rng.randint(0, reqs // 3)
        return dict(op=op, reqs=reqs, tokens=rng.randint(2, 64) if tree else rng.choice([1, 1, 2, 3, 4, 5]), tree=tree,
                    lo=hi if _yes(rng) else 1, hi=hi, lens_seed=rng.randrange(1 << 20), **_draw_heads(rng),
                    page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["bf16", "e4m3"]), empty=empty,
                    lse=empty == 0)
    if op == "store":
        tokens = _log_int(rng, 1, 65536)
        return dict(op=op, tokens=tokens, kv=_log_int(rng, 1, 16), dim=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["bf16", "e4m3"]), sliced=_yes(rng),
                    skip=rng.randint(0, tokens // 3))
    lens = _draw_lens(rng, 8192) if _yes(rng) else dict(count=_log_int(rng, 1, 4096), lo=1, hi=rng.choice([1, 1, 4]),
                                                        lens_seed=rng.randrange(1 << 20))
    return dict(op=op, **lens, old=_log_int(rng, 1, 16384), page=rng.choice([16, 32, 64, 128, 256]),
                empty=rng.randint(0, lens["count"] // 3))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        case = _draw_one(rng)
        if case["op"] == "prompt" and sum(_lens(case)) > 65536:
            continue
        # (requests of one page share no cache line: the pool has a page each at least)
        if case["op"] == "tokens" and case["reqs"] * case["page"] * case["kv"] * case["dim"] > 1 << 30:
            continue
        if _cost(case) <= most[case["op"]]:
            return case


def _lens(case):
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case.get("count") or case["reqs"])]


def _live(case):
    """The requests that are not empty slots of their batch."""
    n = case.get("count") or case["reqs"]
    gone = set(random.Random(case["lens_seed"] + 1).sample(range(n), case["empty"]))
    return [i for i in range(n) if i not in gone]


def _olds(case):
    """Tokens that requests have in the cache already: a third of them none."""
    r = random.Random(case["lens_seed"] + 2)
    return [0 if r.random() < 1 / 3 else r.randint(1, case["old"]) for _ in range(case["count"])]


def work(case):
    op = case["op"]
    if op == "prompt":
        lens, D, H = _lens(case), case["dim"], case["heads"]
        T = sum(lens)
        return {"bytes": T * (4 * H * D + 4 * case["kv"] * D + (4 * H if case["lse"] else 0)),
                "flops": 2 * D * H * sum(n * (n + 1) for n in lens)}
    if op == "tokens":
        lens, D, H, T, ps = _lens(case), case["dim"], case["heads"], case["tokens"], case["page"]
        live = _live(case)
        held = sum(lens[i] + T for i in live)
        size = 2 if case["cache"] == "bf16" else 1
        return {"bytes": 2 * held * case["kv"] * D * size + case["reqs"] * (4 * T * H * D + 8) + 4 * (held // ps)
                + (8 * T * case["reqs"] if case["tree"] else 0) + (4 * T * H * case["reqs"] if case["lse"] else 0),
                "flops": 4 * D * H * T * sum(lens[i] + (T + 1) / 2 for i in live)}
    if op == "store":
        n = 2 * case["kv"] * case["dim"] * (case["tokens"] - case["skip"])
        return {"bytes": n * (4 if case["cache"] == "bf16" else 3) + 8 * case["tokens"], "flops": n}
    lens = _lens(case)
    return {"bytes": 8 * sum(lens) + sum(4 + 4 * -(-n // case["page"]) * 2 for n in lens) + 12 * len(lens),
            "flops": 4 * sum(lens)}


# ---------------------------------------------------------------------------
# inputs

class State(dict):
    __getattr__ = dict.__getitem__


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    if dtype != torch.float32 and math.prod(shape) > 1 << 28:  # (a large one in parts)
        return torch.cat([_normal(g, n, *shape[1:], scale=scale, dtype=dtype)
                          for n in (len(p) for p in torch.arange(shape[0]).chunk(16))])
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _packed(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    return cu.to(torch.int32).to(DEV)


def _qkv(g, T, H, kv, D, sliced):
    """Queries, keys and values of T tokens, columns of one projection's rows
    where the case says sliced.  Scores spread by about two."""
    if sliced:
        rows = _normal(g, T, (H + 2 * kv) * D, scale=1.4)
        q, k, v = torch.split(rows, [H * D, kv * D, kv * D], dim=1)
        return q.unflatten(1, (H, D)), k.unflatten(1, (kv, D)), v.unflatten(1, (kv, D))
    return _normal(g, T, H, D, scale=1.4), _normal(g, T, kv, D, scale=1.4), _normal(g, T, kv, D)


def _prepare_prompt(case, g):
    lens = _lens(case)
    q, k, v = _qkv(g, sum(lens), case["heads"], case["kv"], case["dim"], case["sliced"])
    return State(op="prompt", q=q, k=k, v=v, cu=_packed(lens), lens=lens, lse=case["lse"])


def _scales(g, kv):
    return torch.rand(kv, generator=g, device=DEV) * 0.02 + 0.01


def _pool(case, g, pages):
    """Keys and values in pages, and their scales where they are 8 bits wide."""
    shape = (pages, case["page"], case["kv"], case["dim"])
    if case["cache"] == "bf16":
        return dict(kc=_normal(g, *shape, scale=1.4), vc=_normal(g, *shape), ks=None, vs=None)
    ks, vs = _scales(g, case["kv"]), _scales(g, case["kv"])
    kc, vc = ((_normal(g, *shape) * 50).to(torch.float8_e4m3fn) for _ in range(2))
    return dict(kc=kc, vc=vc, ks=ks, vs=vs)


def _trees(r, T):
    """Ancestors (itself among them) of T drafts, as bits: the first draft is a
    root, the others' parents are drafts ahead of them or none."""
    up = []
    for i in range(T):
        parent = r.randint(-1, i - 1) if i else -1
        up.append((up[parent] if parent >= 0 else 0) | 1 << i)
    return [u - (1 << 64) if u >> 63 else u for u in up]


def _table(g, lens, page, live, width):
    """A table of pages for more requests than the batch has, the batch's rows in
    it (-1 in its empty slots), and the count of pages handed out, from the
    front of a shuffled list of them."""
    n = len(lens)
    rows = torch.randperm(n + 3, generator=g, device=DEV)[:n].to(torch.int32)
    counts = torch.tensor([-(-x // page) for x in lens])
    keep = torch.zeros(n, dtype=torch.bool)
    keep[live] = True
    counts = torch.where(keep, counts, 0)
    used = int(counts.sum())
    first = torch.cumsum(counts, 0) - counts
    free = torch.randperm(used + 5, generator=g, device=DEV).to(torch.int32)
    at = first[:, None] + torch.arange(width)
    at = torch.where(torch.arange(width) < counts[:, None], at, -1).to(DEV)
    table = torch.full((n + 3, width), -1, dtype=torch.int32, device=DEV)
    table[rows.long()] = torch.where(at >= 0, free[at.clamp(min=0)], -1)
    rows = torch.where(keep.to(DEV), rows, -1)
    return table, rows, free, used


def _prepare_tokens(case, g):
    n, T, H, D, page = case["reqs"], case["tokens"], case["heads"], case["dim"], case["page"]
    lens, live = _lens(case), _live(case)
    width = -(-(max(lens) + T) // page)
    table, rows, free, _ = _table(g, [x + T for x in lens], page, live, width)
    tree = None
    if case["tree"]:
        r = random.Random(case["lens_seed"] + 3)
        tree = torch.tensor([_trees(r, T) for _ in range(n)], dtype=torch.int64, device=DEV)
    return State(op="tokens", q=_normal(g, n, T, H, D, scale=1.4), **_pool(case, g, len(free)), table=table, rows=rows,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), tree=tree, host_lens=lens, live=live,
                 lse=case["lse"])


def _prepare_store(case, g):
    T, kv, D, page = case["tokens"], case["kv"], case["dim"], case["page"]
    _, k, v = _qkv(g, T, 1, kv, D, case["sliced"])
    pages = -(-T // page) + 2
    pool = _pool(case, g, pages)
    if case["tokens"] < 4096:  # (a token each of many requests)
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    else:                      # (prompts fill pages in order)
        t = torch.arange(T, device=DEV)
        slots = torch.randperm(pages, generator=g, device=DEV)[t // page] * page + t % page
    slots[torch.randperm(T, generator=g, device=DEV)[:case["skip"]]] = -1
    return State(op="store", k=k, v=v, **pool, slots=slots)


def _prepare_pages(case, g):
    lens, olds, live = _lens(case), _olds(case), _live(case)
    page = case["page"]
    width = -(-(case["old"] + case["hi"]) // page)
    table, rows, free, used = _table(g, olds, page, live, width)
    more = sum(-(-(olds[i] + lens[i]) // page) + 1 for i in live)
    rest = torch.arange(len(free), len(free) + more, dtype=torch.int32, device=DEV)
    return State(op="pages", lens=torch.tensor(olds, dtype=torch.int32, device=DEV), table=table, rows=rows,
                 free=torch.cat([free, rest[torch.randperm(more, generator=g, device=DEV)]]),
                 head=torch.tensor([used], dtype=torch.int32, device=DEV), cu=_packed(lens), total=sum(lens),
                 page=page)


def prepare(case, seed):
    make = {"prompt": _prepare_prompt, "tokens": _prepare_tokens, "store": _prepare_store, "pages": _prepare_pages}
    return make[case["op"]](case, _gen(seed))


# ---------------------------------------------------------------------------
# plain forms

def _attend(q, k, v, seen, scale):
    """Rows q [..., r, D] over keys and values [..., L, D] where `seen` holds;
    a row that sees nothing is zero, with a logarithm of minus infinity."""
    s = torch.where(seen, (q @ k.transpose(-1, -2).contiguous()) * scale, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (torch.log(total) + top).squeeze(-1)


def _prompt(s):
    T, H, D = s.q.shape
    kv = s.k.shape[1]
    G = H // kv
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, H, dtype=torch.float32, device=DEV) if s.lse else None
    begin = 0
    for n in s.lens:
        k, v = (x[begin:begin + n].float().transpose(0, 1).contiguous() for x in (s.k, s.v))
        for a in range(0, n, ROWS):
            b = min(n, a + ROWS)
            q = s.q[begin + a:begin + b].float().unflatten(1, (kv, G)).permute(1, 2, 0, 3).flatten(1, 2)
            seen = torch.arange(b, device=DEV) <= torch.arange(a, b, device=DEV)[:, None]
            o, l = _attend(q, k[:, :b], v[:, :b], seen.repeat(G, 1), D ** -0.5)
            out[begin + a:begin + b] = o.unflatten(1, (G, b - a)).permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
            if s.lse:
                lse[begin + a:begin + b] = l.unflatten(1, (G, b - a)).permute(2, 0, 1).flatten(1)
        begin += n
    return {"out": out, "lse": lse} if s.lse else {"out": out}


def _widen(x, scale):
    x = x.float()
    return x if scale is None else x * scale[:, None]


def _tokens(s):
    N, T, H, D = s.q.shape
    page, kv = s.kc.shape[1], s.kc.shape[2]
    G = H // kv
    out = torch.zeros(N, T, H, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(N, T, H, dtype=torch.float32, device=DEV) if s.lse else None
    order = sorted(s.live, key=lambda i: s.host_lens[i])
    while order:
        # the longest that are left, as many as a gathered block holds
        longest = s.host_lens[order[-1]] + T
        take = max(1, GATHER // (longest * kv * D))
        who, order = torch.tensor(order[-take:], device=DEV), order[:-take]
        pos = torch.arange(longest, device=DEV)
        at = s.table[s.rows[who].long()][:, pos // page].long() * page + pos % page
        at = at.clamp(min=0)
        k, v = (_widen(x.flatten(0, 1)[at], sc).transpose(1, 2) for x, sc in ((s.kc, s.ks), (s.vc, s.vs)))
        draft = pos - s.lens[who, None]  # [n, L]
        if s.tree is None:
            seen = draft[:, None] <= torch.arange(T, device=DEV)[:, None]
        else:
            bits = s.tree[who][..., None] >> draft[:, None].clamp(0, 63) & 1
            seen = (draft[:, None] < 0) | ((draft[:, None] < T) & (bits == 1))
        q = s.q[who].float().unflatten(2, (kv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, kv, T G, D]
        o, l = _attend(q, k, v, seen.repeat_interleave(G, 1)[:, None], D ** -0.5)
        out[who] = o.unflatten(2, (T, G)).transpose(1, 2).flatten(2, 3).to(torch.bfloat16)
        if s.lse:
            lse[who] = l.unflatten(2, (T, G)).transpose(1, 2).flatten(2)
    return {"out": out, "lse": lse} if s.lse else {"out": out}


def _store(s):
    put = s.slots >= 0
    at = s.slots[put]
    for x, cache, scale in ((s.k, s.kc, s.ks), (s.v, s.vc, s.vs)):
        x = x[put]
        if scale is not None:
            x = (x.float() / scale[:, None]).clamp(-448.0, 448.0).to(cache.dtype)
        # (the framework's index assignment does not take 8-bit floats: through bytes)
        flat = cache.flatten(0, 1)
        if scale is None:
            flat[at] = x
        else:
            flat.view(torch.uint8)[at] = x.view(torch.uint8)
    return {"k": s.kc, "v": s.vc}


def _pages(s):
    width, page = s.table.shape[1], s.page
    live = s.rows >= 0
    new = (s.cu[1:] - s.cu[:-1]).long()
    old = s.lens.long()
    have = ((old + page - 1) // page).clamp(max=width)
    need = torch.where(live, ((old + new + page - 1) // page).clamp(max=width) - have, 0)
    start = s.head.long() + torch.cumsum(need, 0) - need
    t = torch.arange(s.total, device=DEV)
    seq = torch.searchsorted(s.cu.long(), t, right=True) - 1
    pos = old[seq] + t - s.cu[seq]
    block = pos // page
    fresh = start[seq] + block - have[seq]
    fits = live[seq] & (block < width)
    opened = fits & (block >= have[seq])
    known = s.table[s.rows[seq].clamp(min=0).long(), block.clamp(max=width - 1)].long()
    got = torch.where(fresh < len(s.free), s.free[fresh.clamp(0, len(s.free) - 1)].long(), -1)
    at = torch.where(opened, got, known)
    slots = torch.where(fits & (at >= 0), at * page + pos % page, -1)
    first = opened & (pos % page == 0)
    s.table[s.rows[seq[first]].long(), block[first]] = got[first].to(torch.int32)
    return {"slots": slots, "lens": torch.where(live, old + new, old).to(torch.int32),
            "head": (s.head + need.sum()).to(torch.int32), "table": s.table}


# ---------------------------------------------------------------------------
# the package's entry points

def _own(s):
    from kda_gated_delta_chunked_amd import attn

    if s.op == "prompt":
        out, lse = attn.prefill(s.q, s.k, s.v, cu_seqlens=s.cu, return_lse=s.lse)
        return {"out": out, "lse": lse} if s.lse else {"out": out}
    if s.op == "tokens":
        out, lse = attn.decode(s.q, s.kc, s.vc, s.table, s.lens, rows=s.rows, tree=s.tree, k_scale=s.ks, v_scale=s.vs,
                               return_lse=s.lse)
        return {"out": out, "lse": lse} if s.lse else {"out": out}
    if s.op == "store":
        attn.store(s.k, s.v, s.kc, s.vc, s.slots, k_scale=s.ks, v_scale=s.vs)
        return {"k": s.kc, "v": s.vc}
    slots, lens, head = attn.assign_pages(s.lens, s.table, s.free, s.head, page_size=s.page, rows=s.rows,
                                          cu_seqlens=s.cu, total_tokens=s.total)
    return {"slots": slots, "lens": lens, "head": head, "table": s.table}


def run(state):
    if own:
        return _own(state)
    return {"prompt": _prompt, "tokens": _tokens, "store": _store, "pages": _pages}[state.op](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(q, k, v, seen):
    """q [r, D] over k, v [L, D], seen [r, L], all in 64 bits."""
    s = q @ k.t() / math.sqrt(q.shape[1])
    s.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]) @ v, lse


def _exact_prompt(s):
    out, lse = (torch.empty(n, dtype=torch.float64, device=DEV) for n in (s.q.shape, s.q.shape[:2]))
    share = s.q.shape[1] // s.k.shape[1]
    cu = s.cu.tolist()
    for b, e in zip(cu, cu[1:]):
        for h in range(s.q.shape[1]):
            k, v = (x[b:e, h // share].to(torch.float64) for x in (s.k, s.v))
            for a in range(b, e, 4096):
                z = min(e, a + 4096)
                seen = torch.ones(z - a, z - b, dtype=torch.bool, device=DEV).tril(a - b)
                out[a:z, h], lse[a:z, h] = _exact_rows(s.q[a:z, h].to(torch.float64), k[:z - b], v[:z - b], seen)
    return {"out": out, "lse": lse} if s.lse else {"out": out}


def _exact_tokens(s):
    N, T, H, D = s.q.shape
    page, kv = s.kc.shape[1], s.kc.shape[2]
    out = torch.zeros(s.q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((N, T, H), -math.inf, dtype=torch.float64, device=DEV)
    for n, (row, c) in enumerate(zip(s.rows.tolist(), s.lens.tolist())):
        if row < 0:
            continue
        pages = s.table[row, :-(-(c + T) // page)].long()
        k, v = (x[pages].to(torch.float64).flatten(0, 1)[:c + T] for x in (s.kc, s.vc))
        if s.ks is not None:
            k, v = k * s.ks.to(torch.float64)[:, None], v * s.vs.to(torch.float64)[:, None]
        seen = torch.ones(T, c + T, dtype=torch.bool, device=DEV)
        if s.tree is None:
            seen[:, c:] = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
        else:
            seen[:, c:] = torch.tensor([[bool(m >> j & 1) for j in range(T)] for m in s.tree[n].tolist()], device=DEV)
        for h in range(kv):
            G = H // kv
            q = s.q[n, :, h * G:(h + 1) * G].to(torch.float64).reshape(T * G, D)
            o, l = _exact_rows(q, k[:, h], v[:, h], seen.repeat_interleave(G, 0))
            out[n, :, h * G:(h + 1) * G], lse[n, :, h * G:(h + 1) * G] = o.view(T, G, D), l.view(T, G)
    return {"out": out, "lse": lse} if s.lse else {"out": out}


def _exact_store(s):
    res = {}
    for name, x, cache, scale in (("k", s.k, s.kc, s.ks), ("v", s.v, s.vc, s.vs)):
        flat = cache.to(torch.float64).flatten(0, 1)
        x = x.to(torch.float64)
        if scale is not None:
            x = torch.clamp(x / scale.to(torch.float64)[:, None], -448, 448)
        put = torch.nonzero(s.slots != -1).flatten()
        flat.index_copy_(0, s.slots[put], x[put])
        res[name] = flat.view(cache.shape)
    return res


def _exact_pages(s):
    table, free, page = s.table.tolist(), s.free.tolist(), s.page
    cu, lens, head = s.cu.tolist(), s.lens.tolist(), int(s.head)
    slots = []
    for n, row in enumerate(s.rows.tolist()):
        for _ in range(cu[n], cu[n + 1]):
            if row < 0:
                slots.append(-1)
                continue
            block, off = divmod(lens[n], page)
            if off == 0:
                table[row][block] = free[head]
                head += 1
            slots.append(table[row][block] * page + off)
            lens[n] += 1
    res = (slots, lens, [head], table)
    return {name: torch.tensor(x, dtype=torch.int64 if name == "slots" else torch.int32, device=DEV)
            for name, x in zip(("slots", "lens", "head", "table"), res)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "tokens": _exact_tokens, "store": _exact_store, "pages": _exact_pages}[s.op](s)
