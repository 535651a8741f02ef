"""Powers of a slow decay over long sequences: no rounding of lambda that repeats chunk after chunk or
segment after segment.

With k, v, q and dz zero the operators leave W_final = lambda^T W0, dW0 = lambda^T dW_final and
dlog_decay = T lambda^T <dW_final, W0>.  Each of N = d^2 values of a state is rounded by itself, by at most
2^-24 of it each time and as often up as down, so the mean of their relative errors shows what all of them
share: the decay.  Over n multiplications the mean of N values' roundings has a deviation of at most
2^-24 sqrt(n / (3 N)): 0.1 x 2^-24 for 128 of them and 4096 values, of which five are allowed.  Chunk factors
that alternate between the two fp32 values around lambda^32 are off by one step (2^-24 below 1) in any number
of chunks, and segments' factors in two parts by nothing that shows.  One rounded factor is off by up to half
a step each time."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
BF16 = torch.bfloat16
DEV = "cuda:0"
STEP = 2.0 ** -24
BOUND = (1 + 5 * 0.1) * STEP


def decays(n):
    """Four log decays whose lambda^n lies well between two fp32 values, two above and two below the nearer one."""
    got, g = {True: [], False: []}, np.float32(-3e-5)
    while min(map(len, got.values())) < 2:
        g = np.float32(g * np.float32(1.001))
        p = math.exp(float(g) * n)
        off = (p - float(np.float32(p))) / 2 ** -24
        if 0.42 < abs(off) < 0.48 and len(got[off > 0]) < 2:
            got[off > 0].append(float(g))
    return got[True] + got[False]


def _mean_error(got, start, power):
    return ((got.astype(np.float64) / (start.astype(np.float64) * power)) - 1).mean()


@pytest.mark.parametrize("seglen,segments", [(512, 64), (32 * 128, 1)])
def test_the_bound_sees_a_repeated_rounding(seglen, segments):
    """The sequences of factors in fp32 on the CPU: with the alternating factor and the two parts within the bound,
    with one rounded factor in the place of either beyond it."""
    start = np.random.default_rng(5).standard_normal(4096).astype(np.float32)
    f = np.float32
    n = 32 if segments == 1 else seglen
    for g in decays(n):
        p32, ps = math.exp(g * 32), math.exp(g * seglen)
        lo = f(p32) if float(f(p32)) <= p32 else np.nextafter(f(p32), f(0))
        frac = (p32 - float(lo)) / float(np.nextafter(lo, f(2)) - lo)
        hi_part = f(ps)
        lo_part = f(ps - float(hi_part))
        power = math.exp(g * seglen * segments)
        for chunk_parts, segment_parts in ((True, True), (segments > 1, False)):
            s, total = start.copy(), 0.5
            for _ in range(seglen // 32):
                total += frac
                up = total >= 1
                total -= up
                s = s * ((np.nextafter(lo, f(2)) if up else lo) if chunk_parts else f(p32))
            for _ in range(segments - 1):
                exact = s.astype(np.float64) * float(hi_part)
                if segment_parts:
                    exact = exact + (s * lo_part).astype(np.float64)
                s = exact.astype(np.float32)
            off = abs(_mean_error(s, start, power))
            assert (off <= BOUND) == (chunk_parts and segment_parts), (g, off / STEP)


# tokens; heads; head size; tokens that a factor stands for: 64 segments carried on by a launch of their own, 10 (6 in the
# backward) by each workgroup itself, and one walk of 128 chunks (more than 256 chains of d = 64, or 128 of d = 128)
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,d,n", [(32768, 4, 64, [512]), (8192, 48, 64, [832, 1376]), (4096, 520, 64, [32]),
                                     (4096, 260, 128, [32])])
def test_slow_decays_do_not_drift(T, H, d, n):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as ttt
    gen = torch.Generator().manual_seed(6)
    g = torch.tensor([x for m in n for x in decays(m)], dtype=torch.float32)
    g = g.repeat(-(-H // len(g)))[:H]
    none = torch.zeros(1, 1, 1, d, dtype=BF16, device=DEV).expand(1, H, T, d)
    w0, dw = torch.randn(1, H, d, d, generator=gen), torch.randn(1, H, d, d, generator=gen)
    power = torch.exp(g.double() * T)
    _, w = ttt.linear_attn_fwd(none, none, none, g.to(DEV), w0=w0.to(DEV), out_dtype=BF16)
    _, _, _, dg, dw0 = ttt.linear_attn_bwd(none, none, none, g.to(DEV), none, w0=w0.to(DEV), dw_final=dw.to(DEV))
    _, _, _, dg1, _ = ttt.linear_attn_bwd(none, none, none, g.to(DEV), none, w0=w0.to(DEV), dw_final=w0.to(DEV))
    for name, got, start in (("W_final", w, w0), ("dW0", dw0, dw)):
        off = (got.cpu().double() / (start.double() * power[:, None, None]) - 1).mean((0, 2, 3)).abs().max().item()
        print(f"{name}: {off / STEP:.2f} steps", flush=True)
        assert off <= BOUND, name
    # dW_final = W0: a sum of positive terms, rounded to fp32 at the end
    want = T * power * (w0.double() ** 2).sum((0, 2, 3))
    off = (dg1[0].cpu().double() / want - 1).abs().max().item()
    print(f"dlog_decay: {off / STEP:.2f} steps", flush=True)
    assert off <= BOUND + STEP
