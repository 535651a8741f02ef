"""Plain 64-bit forms of the short convolution, the selective scan and the block norm for the tests, and how far the
kernels may be from them.

Each form is the operator's definition on CPU tensors, token by token where it is a recurrence.  With ``magnitudes`` it
adds up the magnitudes of the terms instead (decays are positive and stay what they are), which is what an fp32
evaluation's rounding is measured in: a result is off by at most u = 2^-24 of its magnitude for each rounding that a term
goes through, to first order.  Those numbers of roundings, by way of a term:

- a sigmoid, or a softplus and its slope: at most 16 and |x|: exp2 and 1/x are good to 1 ulp = 2 u, the exponent x log2(e)
  is rounded twice (2 |x| e^-|x| <= 1 of the result for the softplus' tail, |x| of it where the result is the tail itself),
  eight steps of a series whose terms fall by 9 each time.  STEP counts them for |x| <= 16.
- a state: each token's decay 2 u of exp2, and one u for the sum; the exponents of the decays that a term goes through add
  up to x, are off by (STEP + 3) u x in all, and terms with x > 32 are below 2^-46 of the largest: 4 T + 32 (STEP + 3).
- sums over channels, states, taps or a row: at most one u each.
A rounding of the output itself is half a step of its type: eps / 2.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
STEP = 40


def silu(x):
    return x * torch.sigmoid(x)


def live_rows(lens, B, T):
    if lens is None:
        return torch.ones(B, T, 1, dtype=torch.float64)
    n = lens.clamp(0, T)
    return (torch.arange(T)[None, :, None] < n[:, None, None]).double()


def masked(x, live):
    return None if x is None else torch.where(live > 0, x.double(), torch.zeros((), dtype=torch.float64))


# ------------------------------------------------------------ convolution --

def conv(x, w, bias=None, state=None, act=False, lens=None, magnitudes=False):
    """(y, state_final, the sum before the activation)"""
    B, T, D = x.shape
    K = w.shape[1]
    live = live_rows(lens, B, T)
    f = (lambda t: t.double().abs()) if magnitudes else (lambda t: t.double())
    x = f(masked(x, live))
    first = torch.zeros(B, K - 1, D, dtype=torch.float64) if state is None else f(state)
    rows = torch.cat([first, x], 1)
    pre = torch.zeros(B, T, D, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            pre[:, t] += f(w[:, j]) * rows[:, t + j]
    if bias is not None:
        pre = pre + f(bias)
    n = torch.full((B,), T) if lens is None else lens.long().clamp(0, T)
    last = torch.stack([rows[b, int(n[b]):int(n[b]) + K - 1] for b in range(B)])
    return (silu(pre) if act else pre) * live, last, pre


def conv_grads(x, w, dy, bias=None, state=None, act=False, lens=None, dstate_final=None):
    """((dx, dw, dbias, dstate), their magnitudes, in 64 bits)"""
    B, T, D = x.shape
    K = w.shape[1]
    live = live_rows(lens, B, T)
    pre = conv(x, w, bias, state, act, lens)[2]
    size = conv(x, w, bias, state, act, lens, magnitudes=True)[2]
    xs = masked(x, live)
    first = torch.zeros(B, K - 1, D, dtype=torch.float64) if state is None else state.double()
    rows = torch.cat([first, xs], 1)
    g = masked(dy, live)
    mag = g.abs()
    if act:
        s = torch.sigmoid(pre)
        g = g * (s + pre * s * (1 - s))
        mag = mag * (1.1 + 0.5 * size)  # |silu'| <= 1.1, |silu''| <= 0.5
    n = torch.full((B,), T) if lens is None else lens.long().clamp(0, T)
    out = []
    for g, rows, w, df in ((g, rows, w.double(), dstate_final), (mag, rows.abs(), w.double().abs(), dstate_final)):
        dw = torch.stack([(g * rows[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
        drows = torch.zeros_like(rows)
        for j in range(K):
            drows[:, j:j + T] += w[:, j] * g
        if df is not None:
            for b in range(B):
                i = int(n[b])
                drows[b, i:i + K - 1] += df[b].double().abs() if out else df[b].double()
        out.append((drows[:, K - 1:] * live, dw, g.sum((0, 1)), drows[:, :K - 1]))
    return out


# ------------------------------------------------------------------- scan --

def scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, softplus=False, lens=None, magnitudes=False, dy=None,
         dh_final=None):
    """(y, h_final), or with dy the gradients (du, ddt, dA, dBm, dCm, dD, dz, ddt_bias, dh0)."""
    B, T, C = u.shape
    G, N = Bm.shape[1], Bm.shape[3]
    each = C // G
    live = live_rows(lens, B, T)
    m = (lambda t: None if t is None else t.abs()) if magnitudes else (lambda t: t)
    u, raw = m(masked(u, live)), masked(dt, live)
    if dt_bias is not None:
        raw = raw + dt_bias.double()
    slope = torch.ones_like(raw)
    if softplus:
        step, slope = torch.logaddexp(raw, torch.zeros_like(raw)), torch.sigmoid(raw)
    else:
        step = raw
    step = step * live
    A = A.double()
    at = m(A)
    gate, dgate = None, None
    if z is not None:
        z = masked(z, live)
        s = torch.sigmoid(z)
        gate, dgate = m(z * s), (s + m(z * s) * (1 - s) if magnitudes else s + z * s * (1 - s))
    Bx, Cx = (m(masked(x, live[:, None])).repeat_interleave(each, 1) for x in (Bm, Cm))  # [B, C, T, N]
    h = torch.zeros(B, C, N, dtype=torch.float64) if h0 is None else m(h0.double())
    ms = m(step)
    hs, ys = [h], []
    for t in range(T):
        a = torch.exp(torch.nan_to_num(step[:, t, :, None] * A, nan=0.0, neginf=-float("inf")))
        on = live[:, t, :, None] > 0
        h = torch.where(on, a * h + (ms[:, t] * u[:, t])[..., None] * Bx[:, :, t], h)
        hs.append(h)
        ys.append((h * Cx[:, :, t]).sum(-1))
    y = torch.stack(ys, 1) if ys else torch.zeros(B, 0, C, dtype=torch.float64)
    if D is not None:
        y = y + m(D.double()) * u
    if dy is None:
        return (y if gate is None else y * gate) * live, h
    up = m(masked(dy, live))
    dz = None
    if gate is not None:
        dz = up * y * dgate
        up = up * gate
    skip = torch.zeros(C, dtype=torch.float64) if D is None else m(D.double())
    du, ddt = up * skip, torch.zeros(B, T, C, dtype=torch.float64)
    dA = torch.zeros(C, N, dtype=torch.float64)
    dB, dC = (torch.zeros(B, G, T, N, dtype=torch.float64) for _ in range(2))
    g = torch.zeros(B, C, N, dtype=torch.float64) if dh_final is None else m(dh_final.double())
    fold = lambda x: x.view(B, G, each, N).sum(2)  # noqa: E731
    safe = torch.nan_to_num(at, neginf=0.0, posinf=0.0)  # (a decay that keeps nothing has no gradient)
    for t in reversed(range(T)):
        on = live[:, t, :, None]
        a = torch.exp(torch.nan_to_num(step[:, t, :, None] * A, nan=0.0, neginf=-float("inf")))
        g = g + up[:, t, :, None] * Cx[:, :, t]
        dC[:, :, t] = fold(up[:, t, :, None] * hs[t + 1])
        dB[:, :, t] = fold(g * (ms[:, t] * u[:, t])[..., None])
        gB = (g * Bx[:, :, t]).sum(-1)
        q = g * a * hs[t] * on
        du[:, t] += gB * ms[:, t]
        ddt[:, t] = (q * safe).sum(-1) + gB * u[:, t]
        dA += (q * ms[:, t, :, None]).sum(0)
        g = torch.where(on > 0, g * a, g)
    ddt = ddt * slope * live
    return du * live, ddt, dA, dB, dC, (up * u).sum((0, 1)), dz, ddt.sum((0, 1)), g


def scan_roundings(T, N, C):
    """(forward, backward): how many u of its magnitude a result may be off."""
    chain = 4 * T + 32 * (STEP + 3)
    return chain + N + 3 * STEP, 2 * chain + 2 * N + C + T + 4 * STEP + 64


# ------------------------------------------------------------------- norm --

def norm(x, res=None, z=None, alpha=None, gamma_post=None, beta_post=None, gamma_pre=None, beta_pre=None, kind="rms",
         eps=1e-6, gate_first=False):
    """(s, y) in 64 bits, differentiable."""
    def normed(v, g, b):
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * g
        return v if b is None else v + b

    v = x
    gate = None if z is None else silu(z)
    if gate is not None and gate_first:
        v = v * gate
    if gamma_post is not None:
        v = normed(v, gamma_post, beta_post)
    if gate is not None and not gate_first:
        v = v * gate
    if alpha is not None:
        v = v * alpha
    s = v if res is None else res + v
    return s, None if gamma_pre is None else normed(s, gamma_pre, beta_pre)


# ------------------------------------------------------------- comparison --

def check(what, got, ref, size, roundings, out=None):
    """got within half a step of its type and ``roundings`` u of ``size``."""
    out = out or got.dtype
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = (torch.finfo(out).eps / 2 * ref.abs() if out != torch.float32 else 0.0) + (roundings + 1) * U * size + 1e-35
    off = (got - ref).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    print(f"{what}: largest error {off.max().item() if off.numel() else 0:.2e}, {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst} times the bound"


class Rounded:
    """A value in 64 bits with a bound on how far an fp32 evaluation of the same steps may be from it, to first order."""

    def __init__(self, v, e=None):
        self.v = v.double()
        self.e = torch.zeros_like(self.v) if e is None else e

    def __add__(self, o):
        v = self.v + o.v
        return Rounded(v, self.e + o.e + U * v.abs())

    def __sub__(self, o):
        v = self.v - o.v
        return Rounded(v, self.e + o.e + U * v.abs())

    def __mul__(self, o):
        v = self.v * o.v
        return Rounded(v, self.v.abs() * o.e + o.v.abs() * self.e + U * v.abs())

    def mean(self):
        """Over a row: 8 elements a thread, 6 steps in a wave, at most 16 waves, the division."""
        n = self.v.shape[-1]
        v = self.v.mean(-1, keepdim=True)
        return Rounded(v, self.e.mean(-1, keepdim=True) + 31 * U * self.v.abs().sum(-1, keepdim=True) / n)

    def column_sums(self):
        rows = self.v.shape[0] * self.v.shape[1]
        return Rounded(self.v.sum((0, 1)), self.e.sum((0, 1)) + rows * U * self.v.abs().sum((0, 1)))

    def inverse_root(self, eps):
        v = (self.v + eps) ** -0.5
        return Rounded(v, 0.5 * v ** 3 * (self.e + U * (self.v + eps)) + 3 * U * v)

    def gate(self):
        """silu and its slope."""
        s = torch.sigmoid(self.v)
        v, d = self.v * s, s + self.v * s * (1 - s)
        own = (16 + self.v.abs()) * U
        return Rounded(v, 1.1 * self.e + own * v.abs()), Rounded(d, 0.5 * self.e + own * (s + v.abs()))


def norm_rounded(x, res, z, alpha, gp, bp, gn, bn, kind, eps, first, ds=None, dy=None, live=None):
    """The block norm and its gradients with their error bounds: (s, y) or (dx, dz, dres, dalpha, dgamma_post, dbeta_post,
    dgamma_pre, dbeta_pre)."""
    R = lambda t: None if t is None else Rounded(t)  # noqa: E731
    row = lambda t: R(t) if live is None or t is None else Rounded(masked(t, live))  # noqa: E731
    x, res, z, ds, dy = (row(t) for t in (x, res, z, ds, dy))
    alpha, gp, bp, gn, bn = (R(t) for t in (alpha, gp, bp, gn, bn))

    def unit(v):
        if kind == "layer":
            v = v - v.mean()
        inv = (v * v).mean().inverse_root(eps)
        return v * inv, inv

    def back(h, un, inv):
        d = h - un * (h * un).mean()
        if kind == "layer":
            d = d - h.mean()
        return d * inv

    gate = slope = None
    if z is not None:
        gate, slope = z.gate()
    o = x * gate if gate is not None and first else x
    u1 = inv1 = None
    n1 = o
    if gp is not None:
        u1, inv1 = unit(o)
        n1 = u1 * gp
        if bp is not None:
            n1 = n1 + bp
    v = n1 * gate if gate is not None and not first else n1
    s = v if alpha is None else v * alpha
    if res is not None:
        s = s + res
    y = u2 = None
    if gn is not None:
        u2, inv2 = unit(s)
        y = u2 * gn
        if bn is not None:
            y = y + bn
    if ds is None and dy is None:
        return s, y
    d = ds
    if dy is not None:
        b = back(dy * gn, u2, inv2)
        d = b if d is None else d + b
    if live is not None:
        d = Rounded(d.v * live, d.e * live)
    dv = d if alpha is None else d * alpha
    dz = None
    dn = dv
    if gate is not None and not first:
        dz, dn = dv * n1 * slope, dv * gate
    dx = dn if gp is None else back(dn * gp, u1, inv1)
    if gate is not None and first:
        dz, dx = dx * x * slope, dx * gate
    cols = lambda on, t: t.column_sums() if on is not None else None  # noqa: E731
    return (dx, dz, None if res is None else d, cols(alpha, d * v), None if gp is None else (dn * u1).column_sums(),
            cols(bp, dn), None if dy is None or gn is None else (dy * u2).column_sums(), None if bn is None or dy is None else dy.column_sums())


def check_rounded(what, got, ref, live=None):
    keep = 1.0 if live is None else live
    check(what, got, ref.v * keep, ref.e * keep / U, 1.02)
