"""Softmax attention, the paged cache and its tables in plain torch, in 64 bits, on the
CPU, and the error bounds that the tests hold the kernels to.

Written from the definitions in include/kda_attn.h, without the library.

Bounds.  A weight is rounded to bf16 (2^-8 of it at most) and an output once more
(2^-8 of it): an output is off by 2^-8 (mag + |out|) at most, mag the weighted
mean of the values' magnitudes, and in the mean square, with rounding errors
spread evenly, by sqrt(2 / 3) 2^-8 = 0.0032 of mag at most.  fp32 (scores as sums of D
products, exponentials, sums) adds less than 2^-15 of mag for the scores here:
an exponent's error is (D + 8) 2^-24 of the score's terms' magnitude."""
import math

import torch

F64 = torch.float64
STEP = 2.0 ** -8


def attend(q, k, v, seen, scale):
    """q [r, D] over k, v [L, D] where seen [r, L]: outputs, logarithms, the
    weighted mean of |v|, and the scores' largest magnitude of terms."""
    q, k, v = (x.to(F64) for x in (q, k, v))
    r, D = q.shape
    out, mag = torch.zeros(r, v.shape[1], dtype=F64), torch.zeros(r, v.shape[1], dtype=F64)
    lse, terms = torch.full((r,), -math.inf, dtype=F64), torch.zeros(r, dtype=F64)
    for i in range(r):
        at = torch.nonzero(seen[i]).flatten()
        if len(at) == 0:
            continue
        s = scale * (k[at] @ q[i])
        terms[i] = (scale * (k[at].abs() @ q[i].abs())).max()
        lse[i] = torch.logsumexp(s, 0)
        p = torch.softmax(s, 0)  # (exp(s - lse) would lose the sum where |s| is past 2^53)
        out[i], mag[i] = p @ v[at], p @ v[at].abs()
    return out, lse, mag, terms


def prefill(q, k, v, lens, scale=None):
    """q [T, H, D], k, v [T, KV, D] of packed sequences."""
    T, H, D = q.shape
    G = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, mag = torch.zeros(T, H, D, dtype=F64), torch.zeros(T, H, D, dtype=F64)
    lse, terms = torch.zeros(T, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    b = 0
    for n in lens:
        seen = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(H):
            s = slice(b, b + n)
            out[s, h], lse[s, h], mag[s, h], terms[s, h] = attend(q[s, h], k[s, h // G], v[s, h // G], seen, scale)
        b += n
    return out, lse, mag, terms


def decode(q, k_cache, v_cache, table, lens, rows=None, tree=None, scale=None, k_scale=None, v_scale=None):
    """As ``attn.decode``; absent pages and empty slots included."""
    N, T, H, D = q.shape
    P, size, KV, _ = k_cache.shape
    G, W = H // KV, table.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, mag = torch.zeros(N, T, H, D, dtype=F64), torch.zeros(N, T, H, D, dtype=F64)
    lse, terms = torch.full((N, T, H), -math.inf, dtype=F64), torch.zeros(N, T, H, dtype=F64)
    for n in range(N):
        row = n if rows is None else int(rows[n])
        if not 0 <= row < table.shape[0]:
            continue
        before = max(0, int(lens[n]))
        pos = [(x, int(table[row, x // size])) for x in range(min(before + T, W * size))]
        pos = [(x, p) for x, p in pos if 0 <= p < P]
        if not pos:
            continue
        x, p = (torch.tensor(list(t)) for t in zip(*pos))
        k, v = (c[p, x % size].to(F64) for c in (k_cache, v_cache))
        if k_scale is not None:
            k, v = k * k_scale.to(F64)[:, None], v * v_scale.to(F64)[:, None]
        for t in range(T):
            word = (1 << (t + 1)) - 1 if tree is None else int(tree[t] if tree.dim() == 1 else tree[n, t])
            own = x - before
            seen = (own < 0) | torch.tensor([o >= 0 and bool(word >> o & 1) for o in own.tolist()])
            for h in range(H):
                r = attend(q[n, t, h][None], k[:, h // G], v[:, h // G], seen[None], scale)
                out[n, t, h], lse[n, t, h], mag[n, t, h], terms[n, t, h] = (y[0] for y in r)
    return out, lse, mag, terms


def assert_out(out, ref, mag):
    out = out.to(F64)
    assert torch.isfinite(out).all()
    off = (out - ref).abs()
    assert (off <= STEP * (mag + ref.abs()) * (1 + 2 ** -6) + 1e-30).all(), float((off / (STEP * (mag + ref.abs()) + 1e-30)).max())
    assert off.square().mean().sqrt() <= 0.0033 * mag.square().mean().sqrt()


def assert_lse(lse, ref, terms, D):
    lse = lse.to(F64)
    empty = ref == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    off = (lse - ref)[~empty].abs()
    # the largest score's error, the sum's and the logarithm's, and the result's rounding
    bound = (D + 8) * 2.0 ** -24 * terms[~empty] + 2.0 ** -20 + 2.0 ** -22 * ref[~empty].abs()
    assert (off <= bound).all(), float((off / bound).max())


def assign(lens, rows, cu, table, free, head, size):
    """Token by token; returns slots, lens, head, table."""
    table, lens = table.clone(), [max(0, int(x)) for x in lens]
    R, W = table.shape
    kept = list(lens)
    slots = []
    for n in range(len(lens)):
        row = n if rows is None else int(rows[n])
        for _ in range(int(cu[n]), int(cu[n + 1])):
            slot = -1
            if 0 <= row < R:
                block, at = divmod(lens[n], size)
                if block < W:
                    if at == 0:
                        table[row, block] = max(-1, int(free[head])) if 0 <= head < len(free) else -1
                        head += 1
                    page = int(table[row, block])
                    slot = page * size + at if page >= 0 else -1
            slots.append(slot)
            lens[n] += 1
        if not 0 <= row < R:
            lens[n] = kept[n]
    return slots, lens, head, table
