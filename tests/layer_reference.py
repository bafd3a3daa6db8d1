"""The layer operators' formulas in 64 bits on the CPU, token by token, with
the magnitudes (the same sums over absolute values) that error bounds use.
Written from the definitions in include/kda_ssm.h, without the library."""
from __future__ import annotations

import torch

F64 = torch.float64


def silu(v):
    return v / (1 + torch.exp(-v))


def conv(x, weight, bias, act, states, lens):
    """x [T, D]; states [N, W - 1, D].  Returns out, final states and the sum
    of absolute terms, all fp64."""
    W = weight.shape[1]
    w = weight.to(F64)
    outs, mags, finals, at = [], [], [], 0
    for n, L in enumerate(lens):
        rows = torch.cat([states[n].to(F64), x[at:at + L].to(F64)])
        y = torch.zeros(L, x.shape[1], dtype=F64)
        m = torch.zeros_like(y)
        for t in range(L):
            for j in range(W):
                term = w[:, j] * rows[t + j]
                y[t] += term
                m[t] += term.abs()
        if bias is not None:
            y += bias.to(F64)
            m += bias.to(F64).abs()
        outs.append(silu(y) if act == "silu" else y)
        mags.append(m)
        finals.append(rows[L:])
        at += L
    return torch.cat(outs), torch.stack(finals), torch.cat(mags)


def steps(dt, bias, softplus):
    dt = dt.to(F64)
    if bias is not None:
        dt = dt + bias.to(F64)
    return torch.logaddexp(dt, torch.zeros_like(dt)) if softplus else dt


def scan(x, step, A, B, C, D, z, states, lens):
    """x [T, H, P], step [T, H], B and C [T, G, N], states [N_seqs, H, N, P].
    Returns out, final states, the magnitude of out's sum and of the states."""
    H = x.shape[1]
    rep = H // B.shape[1]
    x, A = x.to(F64), A.to(F64)
    B, C = (v.to(F64).repeat_interleave(rep, 1) for v in (B, C))
    outs, mags = torch.zeros(x.shape, dtype=F64), torch.zeros(x.shape, dtype=F64)
    S = states.to(F64).clone()
    M = S.abs()
    at = 0
    for n, L in enumerate(lens):
        for t in range(at, at + L):
            d = torch.exp(step[t] * A)[:, None, None]
            add = (step[t][:, None] * B[t])[:, :, None] * x[t][:, None, :]
            S[n] = d * S[n] + add
            M[n] = d * M[n] + add.abs()
            outs[t] = (C[t][:, :, None] * S[n]).sum(1)
            mags[t] = (C[t].abs()[:, :, None] * M[n]).sum(1)
        at += L
    if D is not None:
        outs = outs + D.to(F64)[:, None] * x
        mags = mags + (D.to(F64)[:, None] * x).abs()
    if z is not None:
        gate = silu(z.to(F64))
        outs, mags = outs * gate, mags * gate.abs()
    return outs, S, mags, M


def norm(x, residual, weight, eps):
    """y in fp64 over the last dimension, and x + residual."""
    s = x.to(F64)
    if residual is not None:
        s = s + residual.to(F64)
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * weight.to(F64), s


# Error bounds.  A bf16 rounding is off by at most half a step, 2^-8 of the
# value; fp32 sums of a few hundred terms by less than 1e-5 of their magnitude.
BF16 = 2.0 ** -8
FP32 = 1e-5


def assert_conv(out, ref, mag, act, what=""):
    """out is rounded once; its fp32 sum is off by at most 6 roundings of 2^-24
    of the magnitude, and silu's slope is below 1.1."""
    err = (out.to(F64) - ref).abs()
    bound = BF16 * ref.abs() + 1.1 * FP32 * mag + FP32 * ref.abs()
    assert (err <= bound).all(), f"{what}: {(err - bound).max()}"


def assert_scan_out(out, ref, mag, what=""):
    """Besides out's own rounding, every term passes through at most one bf16
    rounding inside (of a score, or of the state it is read from): half a step
    of the term, and of the magnitude in sum."""
    err = (out.to(F64) - ref).abs()
    bound = BF16 * ref.abs() + (BF16 * (1 + BF16) + 2 * FP32) * mag + 1e-30
    assert (err <= bound).all(), f"{what}: {(err - bound).max()}"
    if ref.numel() and ref.norm() > 0:
        # the two roundings are independent: 2^-8 / sqrt(3) at most each in the mean
        rel = ((out.to(F64) - ref).norm() / ref.norm()).item()
        assert rel <= 5e-3, f"{what}: {rel}"


def assert_state(state, ref, mag, what=""):
    """fp32 states: decays (argument and exponential), steps and sums are fp32,
    below 2e-5 of the magnitude together; bf16 states are rounded once more."""
    err = (state.to(F64) - ref).abs()
    bound = 2e-5 * mag + (BF16 * ref.abs() if state.dtype == torch.bfloat16 else 0) + 1e-30
    assert (err <= bound).all(), f"{what}: {(err - bound).max()}"


def assert_norm(out, scales, ref, group, what=""):
    """bf16: one rounding, of half a step: 2^-8 of the value, or 2^-134 below
    2^-126, where bf16's steps are 2^-133 whatever the value.  e4m3: a code is off by half a step, 2^-4 of its
    value or 2^-10 (the subnormals' half step), both in scales of fp32
    accuracy."""
    out = out.to(F64) if scales is None else out.float().to(F64)
    if scales is None:
        err, bound = (out - ref).abs(), (BF16 + FP32) * ref.abs() + 2.0 ** -134
    else:
        D = ref.shape[-1]
        n = -(-D // group) if group else 1
        width = group or D
        pad = torch.nn.functional.pad(ref, (0, n * width - D)).unflatten(-1, (n, width))
        want = (pad.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
        assert ((scales.to(F64) - want).abs() <= FP32 * want).all(), what
        each = scales.to(F64).repeat_interleave(width, -1)[..., :D]
        err = (out * each - ref).abs()
        bound = (2.0 ** -4 + FP32) * ref.abs() + 2.0 ** -10 * each * (1 + FP32)
    assert (err <= bound).all(), f"{what}: {(err - bound).max()}"
