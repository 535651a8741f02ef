"""Plain 64-bit forms of linear attention and rotary positions for the tests, and how
far the kernels may be from them.

``attn`` and ``attn_grads`` are the recurrences themselves, token by token, on CPU
tensors.  ``tolerance`` bounds the rounding of an fp32 evaluation to first order: an
output that is a sum of products is off by at most 2^-24 of the sum of their
magnitudes A for each operation that a term goes through.  A comes from the same
recurrence on the magnitudes of the inputs (every weight is a power of lambda, so
>= 0).  The longest way of a term: a score (d products), a sum over a chunk (32
tokens), the state's product (d), one decay and one addition per chunk, the scale, and
the powers of lambda, whose exponents n log(lambda) are off by 2^-24 relatively, so
that a power lambda^n = e^-x is off by x 2^-24 of itself plus two units of expf; terms
with x > 64 are below 2^-92 of the sum's largest weight.  Where a bf16 kernel splits
operands of an output in two parts, 2^-16 of A comes on top for each of the at most
two split operands of a term (scores and states).  A rounding of the output itself is
half a step of its type: eps / 2.
"""
from __future__ import annotations

import math

import torch


def attn(q, k, v, log_decay, w0=None, scale=1.0, lens=None):
    """z [B, H, T, d] and W_final [B, H, d, d] in float64."""
    q, k, v, g = (x.double() for x in (q, k, v, log_decay))
    B, H, T, d = q.shape
    share = torch.arange(H) // (H // k.shape[1])
    k, v = k[:, share], v[:, share]
    lam = torch.exp(g)[:, None, None]
    W = torch.zeros(B, H, d, d, dtype=torch.float64) + (0 if w0 is None else w0.double())
    z = torch.zeros(B, H, T, d, dtype=torch.float64)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        for t in range(n):
            W[b] = lam * W[b] + v[b, :, t, :, None] * k[b, :, t, None, :]
            z[b, :, t] = scale * (W[b] * q[b, :, t, None, :]).sum(-1)
    return z, W


def attn_grads(q, k, v, log_decay, dz, w0=None, dw_final=None, scale=1.0, lens=None, magnitudes=False):
    """(dq, dk, dv, dlog_decay [B, H], dw0 [B, H, d, d]) in float64; with magnitudes, the sums of the
    magnitudes of their terms."""
    args = [q, k, v, dz, w0, dw_final]
    q, k, v, dz, w0, dw_final = (None if x is None else (x.double().abs() if magnitudes else x.double()) for x in args)
    if magnitudes:
        scale = abs(scale)
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    share = torch.arange(H) // (H // Hkv)
    kk, vv = k[:, share], v[:, share]
    lam = torch.exp(log_decay.double())[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(kk), torch.zeros_like(vv)
    dg = torch.zeros(B, H, dtype=torch.float64)
    dw0 = torch.zeros(B, H, d, d, dtype=torch.float64)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        W = torch.zeros(H, d, d, dtype=torch.float64)
        if w0 is not None:
            W = W + (w0[b] if w0.dim() == 4 else w0)
        before = []
        for t in range(n):
            before.append(W)
            W = lam * W + vv[b, :, t, :, None] * kk[b, :, t, None, :]
            dq[b, :, t] = scale * (W * dz[b, :, t, :, None]).sum(-2)
        G = torch.zeros(H, d, d, dtype=torch.float64) if dw_final is None else dw_final[b].clone()
        for t in reversed(range(n)):
            G = G + scale * dz[b, :, t, :, None] * q[b, :, t, None, :]
            dk[b, :, t] = (G * vv[b, :, t, :, None]).sum(-2)
            dv[b, :, t] = (G * kk[b, :, t, None, :]).sum(-1)
            G = lam * G
            dg[b] += (G * before[t]).sum((-1, -2))
        dw0[b] = G
    fold = lambda x: x.view(B, Hkv, H // Hkv, T, d).sum(2)  # noqa: E731
    return dq, fold(dk), fold(dv), dg, dw0


def tolerance(ref, magnitude, d, T, out=torch.float64, split=False, group=1):
    steps = 4 * d + 2 * 32 + 4 * math.ceil(T / 32) + 64 + 8 + group
    part = steps * 2.0 ** -24 + (2 * 2.0 ** -16 if split else 0.0)
    return torch.finfo(out).eps / 2 * ref.abs() * (out != torch.float32) + part * magnitude + 1e-30


def check(what, got, ref, tol):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - ref).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    print(f"{what}: largest error {off.max().item() if off.numel() else 0:.2e}, {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst} times the bound"


def turn(x, pos, freqs, layout="half", scale=1.0, inverse=False):
    """Rotary positions in float64: x [B, H, T, d], pos [B, T] int64 -> each pair times scale e^(i pos f)."""
    x = x.double()
    n = freqs.shape[0]
    angle = pos.double()[:, None, :, None] * freqs
    if inverse:
        angle = -angle
    first, second = ((slice(0, n), slice(n, 2 * n)) if layout == "half" else
                     (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = scale * (a * torch.cos(angle) - b * torch.sin(angle))
    y[..., second] = scale * (a * torch.sin(angle) + b * torch.cos(angle))
    return y
