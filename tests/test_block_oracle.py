"""The 64-bit forms that the short convolution, selective scan and block norm are tested against: their gradients against
differentiation and differences, and small cases worked by hand."""
import pytest
import torch

import block_testutil as bt

F64 = torch.float64


def rnd(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * std


def test_conv_by_hand():
    x = torch.tensor([[[1.0], [2.0], [4.0]]])
    w = torch.tensor([[10.0, 1.0]])  # the token before, the token
    y, last, _ = bt.conv(x, w, bias=torch.tensor([0.5]), state=torch.tensor([[[3.0]]]))
    assert y.flatten().tolist() == [31.5, 12.5, 24.5] and last.flatten().tolist() == [4.0]
    y, last, _ = bt.conv(x, w, state=torch.tensor([[[3.0]]]), lens=torch.tensor([1]))
    assert y.flatten().tolist() == [31.0, 0.0, 0.0] and last.flatten().tolist() == [1.0]
    # fewer tokens than taps: the state moves up
    _, last, _ = bt.conv(x, torch.ones(1, 4), state=torch.tensor([[[7.0], [8.0], [9.0]]]), lens=torch.tensor([1]))
    assert last.flatten().tolist() == [8.0, 9.0, 1.0]


@pytest.mark.parametrize("act", [False, True])
def test_conv_gradients(act):
    x, w, b, s = rnd(2, 5, 3), rnd(3, 3, seed=1), rnd(3, seed=2), rnd(2, 2, 3, seed=3)
    lens = torch.tensor([4, 1])
    dy, df = rnd(2, 5, 3, seed=4), rnd(2, 2, 3, seed=5)
    got = bt.conv_grads(x, w, dy, b, s, act, lens, df)[0]

    def f(x, w, b, s):  # in torch's own convolution
        rows = torch.cat([s, x], 1)
        pre = torch.nn.functional.conv1d(rows.transpose(1, 2), w[:, None], b, groups=3).transpose(1, 2)
        y = (pre * torch.sigmoid(pre) if act else pre) * bt.live_rows(lens, 2, 5)
        last = torch.stack([rows[i, int(lens[i]):int(lens[i]) + 2] for i in range(2)])
        return (y * dy).sum() + (last * df).sum()

    leaves = [t.clone().requires_grad_() for t in (x, w, b, s)]
    for a, r in zip(got, torch.autograd.grad(f(*leaves), leaves)):
        assert torch.allclose(a, r, rtol=1e-12, atol=1e-12)
    assert torch.autograd.gradcheck(f, leaves)


def _scan_case(seed=0):
    B, T, C, N, G = 2, 5, 4, 3, 2
    return dict(u=rnd(B, T, C, seed=seed), dt=rnd(B, T, C, seed=seed + 1), A=-rnd(C, N, seed=seed + 2).abs(),
                Bm=rnd(B, G, T, N, seed=seed + 3), Cm=rnd(B, G, T, N, seed=seed + 4), D=rnd(C, seed=seed + 5),
                z=rnd(B, T, C, seed=seed + 6), dt_bias=rnd(C, seed=seed + 7), h0=rnd(B, C, N, seed=seed + 8))


def test_scan_by_hand():
    one = torch.ones(1, 2, 1)
    y, h = bt.scan(u=torch.tensor([[[1.0], [2.0]]]), dt=one, A=torch.tensor([[-0.5]]), Bm=torch.full((1, 1, 2, 1), 3.0),
                   Cm=torch.full((1, 1, 2, 1), 2.0), D=torch.tensor([10.0]), h0=torch.tensor([[[4.0]]]))
    d = torch.exp(torch.tensor(-0.5, dtype=F64))
    h1 = 4 * d + 3
    h2 = d * h1 + 6
    assert torch.allclose(y.flatten(), torch.stack([2 * h1 + 10, 2 * h2 + 20])) and torch.allclose(h.flatten(), h2)


def test_scan_gradients():
    c = _scan_case()
    lens = torch.tensor([5, 3])
    dy, dh = rnd(2, 5, 4, seed=20), rnd(2, 4, 3, seed=21)
    got = bt.scan(**c, softplus=True, lens=lens, dy=dy, dh_final=dh)
    names = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")

    def f(*args):
        a = dict(zip(names, args))
        live = bt.live_rows(lens, 2, 5)
        step = torch.nn.functional.softplus(a["dt"] + a["dt_bias"]) * live
        h, total = a["h0"], 0.0
        for t in range(5):
            Bt, Ct = (a[n][:, :, t].repeat_interleave(2, 1) for n in ("Bm", "Cm"))
            h = torch.exp(step[:, t, :, None] * a["A"]) * h + (step[:, t] * a["u"][:, t])[..., None] * Bt
            y = (h * Ct).sum(-1) + a["D"] * a["u"][:, t]
            total = total + (y * bt.silu(a["z"][:, t]) * live[:, t] * dy[:, t]).sum()
        return total + (h * dh).sum()

    leaves = [c[n].clone().requires_grad_() for n in names]
    want = torch.autograd.grad(f(*leaves), leaves)
    order = (got[0], got[1], got[2], got[3], got[4], got[5], got[6], got[7], got[8])
    for n, a, r in zip(names, order, want):
        assert torch.allclose(a, r, rtol=1e-10, atol=1e-12), n
    assert torch.autograd.gradcheck(f, leaves)
    # magnitudes bound the values
    size = bt.scan(**c, softplus=True, lens=lens, dy=dy, dh_final=dh, magnitudes=True)
    for a, s in zip(got, size):
        assert (a.abs() <= s * (1 + 1e-12) + 1e-300).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("first", [False, True])
def test_norm_against_torch_and_differences(kind, first):
    x, z, r, al, g1, b1, g2, b2 = (rnd(*s, seed=i) for i, s in enumerate(((2, 3, 6),) * 3 + ((6,),) * 5))
    s, y = bt.norm(x, r, z, al, g1, b1, g2, b2, kind, 1e-5, first)
    own = (lambda v, g, b: torch.nn.functional.layer_norm(v, (6,), g, b, 1e-5)) if kind == "layer" else (
        lambda v, g, b: torch.nn.functional.rms_norm(v, (6,), g, 1e-5) + b)
    gate = bt.silu(z)
    v = own(x * gate, g1, b1) if first else own(x, g1, b1) * gate
    assert torch.allclose(s, r + al * v) and torch.allclose(y, own(r + al * v, g2, b2))
    leaves = [t.requires_grad_() for t in (x, r, z, al, g1, b1, g2, b2)]
    assert torch.autograd.gradcheck(lambda *a: bt.norm(*a, kind, 1e-5, first), leaves)
