"""The plain 64-bit forms that the linear-attention and rotary tests compare with,
against closed forms and differences (CPU)."""
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from attn_testutil import attn, attn_grads, turn  # noqa: E402


def _case(B=2, H=4, Hkv=2, T=7, d=5, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    g = -torch.rand(H, generator=gen, dtype=torch.float64)
    return dict(q=r(B, H, T, d), k=r(B, Hkv, T, d), v=r(B, Hkv, T, d), log_decay=g, w0=r(B, H, d, d), scale=0.7)


def test_attn_is_the_weighted_sum():
    """z_t = scale (sum_{j <= t} lambda^(t-j) (k_j . q_t) v_j + lambda^(t+1) W0 q_t)"""
    c = _case()
    z, W = attn(**c)
    lam = torch.exp(c["log_decay"])
    b, h, hk, t = 1, 3, 1, 5
    s = sum(lam[h] ** (t - j) * (c["k"][b, hk, j] @ c["q"][b, h, t]) * c["v"][b, hk, j] for j in range(t + 1))
    s = c["scale"] * (s + lam[h] ** (t + 1) * c["w0"][b, h] @ c["q"][b, h, t])
    assert torch.allclose(z[b, h, t], s, rtol=1e-13, atol=1e-13)
    last = sum(lam[h] ** (6 - j) * torch.outer(c["v"][b, hk, j], c["k"][b, hk, j]) for j in range(7))
    assert torch.allclose(W[b, h], last + lam[h] ** 7 * c["w0"][b, h], rtol=1e-13, atol=1e-13)


def test_attn_without_decay_is_ttt_with_batch_gradient_descent():
    """03 §8: TTT-Linear with W0 = 0 and one mini-batch of all tokens, eta = 1/2, is linear attention
    without a decay: W_t = sum_{j <= t} v_j k_j^T.  Against the TTT oracle."""
    gen = torch.Generator().manual_seed(3)
    n, T, d = 3, 8, 16
    q, k, v = (torch.randn(n, T, d, generator=gen, dtype=torch.float32) for _ in range(3))
    import numpy as np
    zr, wr = oracle.linear_primal(q.numpy(), k.numpy(), v.numpy(), np.zeros((n, d, d), np.float32),
                                  np.full((n, T), 0.5, np.float32), T)
    z, W = attn(q[:, None], k[:, None], v[:, None], torch.zeros(1))
    assert np.allclose(z[:, 0].numpy(), zr, rtol=1e-12, atol=1e-12)
    assert np.allclose(W[:, 0].numpy(), wr, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("lens", [None, [0, 4]])
def test_attn_grads_are_the_differences(lens):
    c = _case(seed=5)
    gen = torch.Generator().manual_seed(6)
    lens = None if lens is None else torch.tensor(lens)
    z, W = attn(**c, lens=lens)
    dz, dw = torch.randn(z.shape, generator=gen, dtype=torch.float64), torch.randn(W.shape, generator=gen, dtype=torch.float64)
    got = attn_grads(**c, dz=dz, dw_final=dw, lens=lens)
    loss = lambda c: sum((x * y).sum() for x, y in zip(attn(**c, lens=lens), (dz, dw)))  # noqa: E731
    for name, grad in zip(("q", "k", "v", "log_decay", "w0"), got):
        way = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        up, down = (loss({**c, name: c[name] + s * e * way}) for s in (1, -1))
        if name == "log_decay":
            grad = grad.sum(0)
        assert abs((up - down) / (2 * e) - (grad * way).sum()) < 1e-8 * (1 + abs((grad * way).sum())), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_turn(layout):
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(2, 3, 4, 10, generator=gen, dtype=torch.float64)
    f = torch.tensor([1.0, 0.3, 0.01])
    pos = torch.tensor([[0, 1, 2, 3], [5, 9, 1, 1000]])
    y = turn(x, pos, f, layout, 1.5)
    assert torch.equal(y[..., 6:], x[..., 6:])                      # the rest of the head
    assert torch.allclose(y[0, :, 0, :6], 1.5 * x[0, :, 0, :6])     # position 0
    assert torch.allclose(turn(y, pos, f, layout, 1 / 1.5, inverse=True), x, rtol=1e-12, atol=1e-12)
    # the product of two turned rows depends on the distance of their positions alone
    a = turn(x, pos, f, layout)
    b = turn(x, pos + 17, f, layout)
    assert torch.allclose((a[..., :6] @ a[..., :6].transpose(-1, -2)), (b[..., :6] @ b[..., :6].transpose(-1, -2)))
