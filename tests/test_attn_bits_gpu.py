"""How many bits linear attention keeps on the GPU, by inputs on which lost bits show: sums whose
terms cancel, and sums whose terms all lose on the same side."""
import itertools

import pytest

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
