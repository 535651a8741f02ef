"""How many bits linear attention keeps on the GPU, by inputs on which lost bits show: sums whose
terms cancel, and sums whose terms all lose on the same side."""
import itertools

import pytest

from attn_testutil import attn, attn_grads

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as m
    m.lib()
    return m


# Three pieces of one fp32 value that no two bf16 values hold: 1 + 2^-9 + 2^-18
ONE, MID, LOW = 1.0, 2.0 ** -9, 2.0 ** -18
TYPES = list(itertools.product([16, 32, 64, 128], [BF16, F32], [BF16, F32]))


@pytest.mark.parametrize("d,dtype,out", TYPES)
def test_scores_that_cancel(ttt, d, dtype, out):
    """Token 0 scores 1 + 2^-9 + 2^-18 and token 1 minus 1 + 2^-9, both with the same v: what is left, 2^-18, is a
    value of every type, and so is every partial sum: the result is exact.  dK and dV are such sums too."""
    x, y, v = (torch.zeros(1, 1, 3, d, dtype=dtype) for _ in range(3))
    x[0, 0, 2, :3] = torch.tensor([ONE, MID, LOW])
    y[0, 0, 0, :3] = 1
    y[0, 0, 1, :2] = -1
    v[0, 0, :2] = 1
    v[0, 0, 0, 1] = v[0, 0, 1, 1] = -2
    zero = torch.zeros(1, device=DEV)
    z, _ = ttt.linear_attn_fwd(x.to(DEV), y.to(DEV), v.to(DEV), zero, out_dtype=out)
    want = LOW * v[0, 0, 0].float()
    assert torch.equal(z[0, 0, 2].float().cpu(), want)
    # dK_j = sum_{i >= j} (dz_i.v_j) q_i: two later tokens that cancel, and the same for dV
    turn = lambda t: t.flip(2).contiguous()  # noqa: E731
    if out == dtype:
        a, b, c = (turn(t).to(DEV) for t in (x, y, v))
        dk = ttt.linear_attn_bwd(c, torch.zeros_like(c), a, zero, b)[1]      # v = a, dz = b, q = c
        dv = ttt.linear_attn_bwd(b, a, torch.zeros_like(c), zero, c)[2]      # k = a, q = b, dz = c
        assert torch.equal(dk[0, 0, 0].float().cpu(), want) and torch.equal(dv[0, 0, 0].float().cpu(), want)
        dq = ttt.linear_attn_bwd(torch.zeros_like(a), v.to(DEV), y.to(DEV), zero, x.to(DEV))[0]
        assert torch.equal(dq[0, 0, 2].float().cpu(), want)


@pytest.mark.parametrize("d,dtype,out", TYPES)
def test_states_that_cancel(ttt, d, dtype, out):
    """W0 holds 1 + 2^-9 + 2^-18 beside 1 + 2^-9, and q takes their difference; the same of W0^T, dW_final and its
    transpose for dQ, dK and dV."""
    T = 40  # (a second chunk)
    w = torch.zeros(1, 1, d, d)
    w[0, 0, :, 0] = ONE + MID + LOW
    w[0, 0, :, 1] = ONE + MID
    x = torch.zeros(1, 1, T, d, dtype=dtype)
    x[..., 0], x[..., 1] = 1, -1
    none, g = torch.zeros_like(x).to(DEV), torch.zeros(1, device=DEV)
    want = torch.full((T, d), LOW)
    z, _ = ttt.linear_attn_fwd(x.to(DEV), none, none, g, w0=w.to(DEV), out_dtype=out)
    assert torch.equal(z[0, 0].float().cpu(), want)
    wt = w.transpose(2, 3).contiguous().to(DEV)
    dq = ttt.linear_attn_bwd(none, none, none, g, x.to(out).to(DEV), w0=wt)[0]
    dk = ttt.linear_attn_bwd(none, none, x.to(DEV), g, none.to(out), dw_final=wt)[1]
    dv = ttt.linear_attn_bwd(none, x.to(DEV), none, g, none.to(out), dw_final=w.to(DEV))[2]
    for name, y in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(y[0, 0].float().cpu(), want), name


@pytest.mark.parametrize("d,dtype,out", TYPES)
def test_decay_gradient_of_states_that_cancel(ttt, d, dtype, out):
    """Without K and V: dlog_decay = sum_t (t + 1) q_t^T W0 dz_t (lambda = 1), here 2^-18 times the sum of t + 1, of
    differences between 1 + 2^-9 + 2^-18 and 1 + 2^-9.  Exact in fp32, through both chunks and in segments."""
    w = torch.zeros(1, 1, d, d)
    w[0, 0, 0, :] = ONE + MID + LOW
    w[0, 0, 1, :] = ONE + MID
    for T in (40, 700):
        x, q = torch.zeros(1, 1, T, d, dtype=out), torch.zeros(1, 1, T, d, dtype=dtype)
        x[..., 0], x[..., 1] = 1, -1
        q[..., 3] = 1
        none = torch.zeros_like(q).to(DEV)
        got = ttt.linear_attn_bwd(q.to(DEV), none, none, torch.zeros(1, device=DEV), x.to(DEV), w0=w.to(DEV))
        assert got[3].item() == LOW * T * (T + 1) / 2


# ---- sums that all lose on the same side --------------------------------------
#
# A = 1 + (2^-8 - 2^-15) + (2^-17 - 2^-23), its three bf16 parts, times powers of two: with two parts a value loses
# 2^-17 of itself, a product of two such values 2^-15 (both losses and the product of the second parts), always
# downwards; with three parts a product loses less than 2^-24.  A sum of positive terms goes through n additions
# of part products, each rounded by at most 2^-24 of the whole sum and as often up as down: beyond
# 2^-24 sqrt(2 n ln(2 / p)) with probability p (Hoeffding's bound); p = 10^-13 is taken.

A = 1 + (2.0 ** -8 - 2.0 ** -15) + (2.0 ** -17 - 2.0 ** -23)


def coherent(gen, *shape):
    return A * torch.exp2(torch.randint(-1, 2, shape, generator=gen).float())


def bound(n):
    return 2.0 ** -24 * ((2 * n * 30.6) ** 0.5 + 8)


def additions(d, T):
    """of outputs, states and the decay's gradient: a score (d terms of six part products), a chunk's sum and the state's
    product (32 + d), states (32 a chunk), products of two scores and their sums"""
    chunks = -(-T // 32)
    out = 6 * d + 6 * (32 + d) + 6 * 32 * chunks + 2 * chunks
    return dict(z=out, dq=out, dk=out, dv=out, w=6 * 32 * chunks + 2 * chunks, dw0=6 * 32 * chunks + 2 * chunks,
                dg=out + 6 * d + 3 * T)


@pytest.mark.parametrize("d,T", [(16, 32), (16, 64), (32, 40), (64, 33), (64, 64), (128, 32), (128, 45)])
def test_fp32_products_keep_their_third_parts(ttt, d, T):
    gen = torch.Generator().manual_seed(d + T)
    q, k, v, dz = (coherent(gen, 2, 2, T, d) for _ in range(4))
    w0, dw = coherent(gen, 2, 2, d, d), coherent(gen, 2, 2, d, d)
    c = dict(q=q, k=k, v=v, log_decay=torch.zeros(2), w0=w0)
    g = {n: x.to(DEV) for n, x in c.items()}
    z, w = ttt.linear_attn_fwd(**g)
    got = dict(zip(("z", "w", "dq", "dk", "dv", "dg", "dw0"),
                   (z, w, *ttt.linear_attn_bwd(**g, dz=dz.to(DEV), dw_final=dw.to(DEV)))))
    ref = dict(zip(("z", "w", "dq", "dk", "dv", "dg", "dw0"),
                   (*attn(**c), *attn_grads(**c, dz=dz, dw_final=dw))))
    n = additions(d, T)
    for name, y in got.items():
        off = (y.cpu().double() / ref[name] - 1).abs().max().item()
        print(f"{name}: {off * 2 ** 24:.1f} steps of {bound(n[name]) * 2 ** 24:.0f}", flush=True)
        assert off <= bound(n[name]), name
