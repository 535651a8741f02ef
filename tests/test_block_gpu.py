"""The short convolution, the selective scan and the block norm on the GPU against their 64-bit forms, over types, sizes,
lengths, layouts and masks."""
import pytest

import block_testutil as bt

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as m
    m.lib()
    return m


class Maker:
    """Random CPU tensors from one seed; ``dev`` hands them to the GPU."""

    def __init__(self, seed):
        self.gen = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, std=1.0, mean=0.0, dtype=F32):
        return (torch.randn(*shape, generator=self.gen) * std + mean).to(dtype)


def dev(x, how="dense"):
    """x on the GPU: dense, as a slice of wider rows, or (odd) starting one element off any alignment."""
    if x is None or how == "dense":
        return None if x is None else x.cuda()
    wide = torch.full((*x.shape[:-1], 2 * x.shape[-1] + (1 if how == "odd" else 0)), float("nan"), dtype=x.dtype, device="cuda")
    at = 1 if how == "odd" else 0
    wide[..., at:at + x.shape[-1]] = x.cuda()
    return wide[..., at:at + x.shape[-1]]


def lens_of(kind, B, T):
    if kind is None:
        return None
    return torch.tensor([(0, T, T // 2, 1, T + 3, -2)[(i + (kind == "late")) % 6] for i in range(B)], dtype=torch.int32)


def spoil(x, lens):
    """NaN in the rows behind each sequence's end: nothing may come of them."""
    if lens is None or x is None:
        return x
    x = x.clone()
    t = torch.arange(x.shape[-2])
    for b in range(x.shape[0]):
        x[b][..., t >= max(int(lens[b]), 0), :] = float("nan")
    return x


def device_of(x):
    return None if x is None else x.cuda()


CONV = [  # B, T, D, K, in, out, silu, bias, state, lens, layout
    (1, 1, 1, 2, BF, BF, True, True, False, None, "dense"),
    (2, 67, 64, 4, BF, BF, True, True, True, None, "dense"),
    (6, 33, 24, 4, BF, F32, True, False, True, "early", "slice"),
    (6, 33, 24, 3, F32, F32, False, True, True, "late", "slice"),
    (2, 16, 130, 2, F32, BF, True, True, False, None, "dense"),
    (3, 17, 9, 4, BF, BF, True, True, True, "late", "odd"),
    (3, 2, 8, 4, F32, F32, True, True, True, "early", "dense"),
    (1, 300, 264, 4, BF, BF, False, False, False, None, "slice"),
    (1, 1030, 12, 3, F32, F32, True, True, True, None, "odd"),
]


def conv_case(B, T, D, K, ind, outd, silu, bias, state, lens, layout, seed=0):
    mk = Maker(seed)
    lens = lens_of(lens, B, T)
    x = mk(B, T, D, dtype=ind)
    c = dict(x=x, w=mk(D, K, std=0.5), bias=mk(D) if bias else None, state=mk(B, K - 1, D, dtype=ind) if state else None)
    g = dict(x=dev(spoil(x, lens), layout), w=c["w"].cuda(), bias=device_of(c["bias"]), state=device_of(c["state"]))
    return mk, lens, c, g


@pytest.mark.parametrize("case", CONV)
def test_conv_forward(ttt, case):
    B, T, D, K, ind, outd, silu, *_ = case
    _, lens, c, g = conv_case(*case)
    y, last = ttt.short_conv_fwd(**g, silu=silu, lens=device_of(lens), out_dtype=outd)
    ref, rlast, _ = bt.conv(**c, act=silu, lens=lens)
    size = bt.conv(**c, lens=lens, magnitudes=True)[0]
    # K products and the bias, 1.1 at most through silu, whose own steps are 16 + |x|
    bt.check("y", y, ref, size * 1.1, K + 1 + (16 + size.max().item() if silu else 0))
    assert torch.equal(last.cpu().double(), rlast)


@pytest.mark.parametrize("case", CONV)
def test_conv_backward(ttt, case):
    B, T, D, K, ind, outd, silu, *_ = case
    mk, lens, c, g = conv_case(*case, seed=1)
    dy = mk(B, T, D, dtype=outd)
    df = mk(B, K - 1, D, dtype=outd) if c["state"] is not None else None
    got = ttt.short_conv_bwd(g["x"], g["w"], dev(spoil(dy, lens), case[-1]), bias=g["bias"], state=g["state"], silu=silu,
                             lens=device_of(lens), dstate_final=device_of(df))
    ref, size = bt.conv_grads(c["x"], c["w"], dy, c["bias"], c["state"], silu, lens, df)
    deep = bt.conv(**c, lens=lens, magnitudes=True)[2].max().item()
    for n, a, r, s in zip(("dx", "dw", "dbias", "dstate"), got, ref, size):
        # the pre-activation's K + 1 roundings (half of each shows in silu'), its own 20 + |x|, K taps, the rows' sums
        bt.check(n, a, r, s, 2 * K + 8 + (20 + deep if silu else 0) + (B * T if n in ("dw", "dbias") else 0))


@pytest.mark.parametrize("case", [c for c in CONV if c[8]])
def test_conv_tokens_are_the_prompt(ttt, case):
    """A prompt in one call, and in pieces of 1, 2 and more tokens from the carried state, bit for bit."""
    B, T, D, K, ind, outd, silu, *_ = case
    _, _, c, g = conv_case(*case)
    x = c["x"].cuda()
    y, last = ttt.short_conv_fwd(x, g["w"], bias=g["bias"], state=g["state"], silu=silu, out_dtype=outd)
    state, at = g["state"].clone(), 0
    for n in (1, 2, 1, T):
        n = min(n, T - at)
        if n:
            z = ttt.short_conv_decode(x[:, at:at + n], g["w"], state, bias=g["bias"], silu=silu, out_dtype=outd)
            assert torch.equal(z, y[:, at:at + n])
            at += n
    assert torch.equal(state, last)
    # sequences without new tokens keep their state
    lens = torch.tensor([i % 2 for i in range(B)], dtype=torch.int32, device="cuda")
    before = state.clone()
    z = ttt.short_conv_decode(x[:, :1], g["w"], state, bias=g["bias"], silu=silu, out_dtype=outd, lens=lens)
    assert torch.equal(state[::2], before[::2]) and not z[::2].any()
    if K > 2:
        assert torch.equal(state[1::2, :-1], before[1::2, 1:])
    assert torch.equal(state[1::2, -1], x[1::2, 0])


SCAN = [  # B, T, D, N, G, in, out, softplus, gate, D skip, bias, h0, lens, layout
    (1, 1, 1, 1, 1, F32, F32, False, False, False, False, False, None, "dense"),
    (2, 67, 64, 16, 1, BF, BF, True, True, True, True, False, None, "dense"),
    (1, 33, 130, 16, 1, BF, F32, True, True, True, True, True, None, "slice"),
    (6, 40, 24, 16, 3, BF, BF, True, True, False, True, True, "early", "slice"),
    (6, 40, 22, 8, 2, F32, F32, True, False, True, False, True, "late", "odd"),
    (1, 64, 72, 5, 1, F32, BF, False, True, True, True, True, None, "dense"),
    (2, 65, 66, 3, 2, F32, F32, True, True, True, True, True, None, "odd"),
    (2, 100, 64, 32, 1, BF, BF, True, True, True, True, True, None, "dense"),
    (3, 31, 8, 17, 1, F32, F32, True, True, True, True, True, "late", "dense"),
    (1, 700, 64, 16, 1, F32, F32, True, True, True, True, True, None, "dense"),   # few channels: segments
    (3, 517, 40, 4, 1, BF, F32, True, True, True, True, True, "late", "slice"),   # and sequences that end in them
    (2, 389, 20, 20, 2, F32, F32, True, False, True, True, False, None, "dense"),
]


def scan_case(B, T, D, N, G, ind, outd, softplus, gate, skip, bias, h0, lens, layout, seed=0):
    mk = Maker(seed)
    lens = lens_of(lens, B, T)
    bc = mk(B, G, T, 2 * N, dtype=ind)
    c = dict(u=mk(B, T, D, dtype=ind),
             dt=mk(B, T, D, std=0.7, mean=-2.0, dtype=ind) if softplus else (mk(B, T, D).abs() * 0.1).to(ind),
             A=-(mk(D, N).abs() * 3 + 0.01), Bm=bc[..., :N], Cm=bc[..., N:], D=mk(D) if skip else None,
             z=mk(B, T, D, std=2.0, dtype=ind) if gate else None, dt_bias=(mk(D, std=0.3) if softplus else mk(D).abs() * 0.01)
             if bias else None, h0=mk(B, D, N) if h0 else None)
    bad = spoil(bc, lens).cuda()
    g = {k: device_of(v) for k, v in c.items()}
    for n in ("u", "dt", "z"):
        g[n] = dev(spoil(c[n], lens), layout)
    g["Bm"], g["Cm"] = bad[..., :N], bad[..., N:]
    return mk, lens, c, g


@pytest.mark.parametrize("case", SCAN)
def test_scan_forward(ttt, case):
    B, T, D, N, G, ind, outd, softplus, *_ = case
    _, lens, c, g = scan_case(*case)
    y, h = ttt.selective_scan_fwd(**g, softplus=softplus, lens=device_of(lens), out_dtype=outd)
    ry, rh = bt.scan(**c, softplus=softplus, lens=lens)
    my, mh = bt.scan(**c, softplus=softplus, lens=lens, magnitudes=True)
    k = bt.scan_roundings(T, N, D)[0]
    bt.check("y", y, ry, my, k)
    bt.check("h_final", h, rh, mh, k)
    # the state carried in place
    if g["h0"] is not None:
        state = g["h0"].clone()
        y2, h2 = ttt.selective_scan_fwd(**{**g, "h0": state}, softplus=softplus, lens=device_of(lens), out_dtype=outd,
                                        h_final=state)
        assert h2 is state and torch.equal(y2, y) and torch.equal(state, h)


NAMES = ("du", "ddt", "dA", "dBm", "dCm", "dD", "dz", "ddt_bias", "dh0")


@pytest.mark.parametrize("case", SCAN)
def test_scan_backward(ttt, case):
    B, T, D, N, G, ind, outd, softplus, gate, skip, bias, h0, *_ = case
    mk, lens, c, g = scan_case(*case, seed=2)
    dy, dh = mk(B, T, D, dtype=outd), mk(B, D, N) if h0 else None
    got = ttt.selective_scan_bwd(dy=dev(spoil(dy, lens), case[-1]), dh_final=device_of(dh), softplus=softplus,
                                 lens=device_of(lens), **g)
    ref = bt.scan(**c, softplus=softplus, lens=lens, dy=dy, dh_final=dh)
    size = bt.scan(**c, softplus=softplus, lens=lens, dy=dy, dh_final=dh, magnitudes=True)
    k = bt.scan_roundings(T, N, D // G)[1]
    for n, a, r, s in zip(NAMES, got, ref, size):
        assert (a is None) == (r is None), n
        if a is not None:
            bt.check(n, a, r, s, k + (B * T if n in ("dA", "dD", "ddt_bias") else 0))
    again = ttt.selective_scan_bwd(dy=dev(spoil(dy, lens), case[-1]), dh_final=device_of(dh), softplus=softplus,
                                   lens=device_of(lens), **g)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("case", [c for c in SCAN if c[1] <= 100])
def test_scan_tokens(ttt, case):
    B, T, D, N, G, ind, outd, softplus, *_ = case
    _, _, c, g = scan_case(*case[:12], None, case[13], seed=3)
    ref = bt.scan(**c, softplus=softplus)
    size = bt.scan(**c, softplus=softplus, magnitudes=True)
    h = torch.zeros(B, D, N, device="cuda") if g["h0"] is None else g["h0"].clone()
    more = {k: g[k] for k in ("A", "D", "dt_bias")}
    ys, at = [], 0
    for n in (1, 3, 1, T):
        n = min(n, T - at)
        if n:
            cut = slice(at, at + n)
            z = None if g["z"] is None else g["z"][:, cut]
            ys.append(ttt.selective_scan_decode(g["u"][:, cut], g["dt"][:, cut], Bm=g["Bm"][:, :, cut], Cm=g["Cm"][:, :, cut],
                                                h=h, z=z, softplus=softplus, out_dtype=outd, **more))
            at += n
    k = bt.scan_roundings(T, N, D)[0]
    bt.check("y", torch.cat(ys, 1), ref[0], size[0], k)
    bt.check("h", h, ref[1], size[1], k)
    lens = torch.tensor([i % 2 for i in range(B)], dtype=torch.int32, device="cuda")
    before = h.clone()
    y = ttt.selective_scan_decode(g["u"][:, :1], g["dt"][:, :1], Bm=g["Bm"][:, :, :1], Cm=g["Cm"][:, :, :1], h=h,
                                  softplus=softplus, lens=lens, **more)
    assert torch.equal(h[::2], before[::2]) and not y[::2].any()


NORM = [  # B, T, D, in, res dtype, kind, gate, gate first, post, post beta, alpha, pre, pre beta, res, lens, layout
    (1, 1, 1, F32, F32, "rms", False, False, True, False, True, True, False, True, None, "dense"),
    (2, 5, 64, BF, BF, "rms", True, False, True, False, True, True, False, True, None, "dense"),
    (6, 7, 768, BF, F32, "layer", True, False, True, True, True, True, True, True, "early", "slice"),
    (2, 9, 500, F32, F32, "layer", True, True, True, True, True, True, True, True, None, "odd"),
    (1, 33, 2048, BF, F32, "rms", True, True, True, False, False, True, False, True, None, "dense"),
    (6, 3, 99, BF, BF, "layer", False, False, False, False, True, True, True, True, "late", "odd"),
    (2, 4, 1000, F32, BF, "rms", False, False, False, False, False, True, False, False, None, "dense"),
    (1, 6, 4096, BF, BF, "layer", True, False, True, False, True, False, False, True, None, "dense"),
    (1, 3, 8192, F32, F32, "rms", True, False, True, True, True, True, True, True, None, "dense"),
    (1, 5, 4099, BF, BF, "layer", True, True, True, True, True, True, True, True, None, "odd"),
    (1, 2, 8191, F32, F32, "layer", True, False, True, True, True, True, True, True, None, "dense"),
    (2, 600, 136, BF, F32, "layer", True, False, True, True, True, True, True, True, None, "dense"),
]


def norm_case(B, T, D, ind, rt, kind, gate, first, post, post_b, alpha, pre, pre_b, res, lens, layout, seed=0):
    mk = Maker(seed)
    lens = lens_of(lens, B, T)
    p = lambda on, mean: mk(D, std=0.2, mean=mean) if on else None  # noqa: E731
    c = dict(x=mk(B, T, D, mean=0.3, dtype=ind), res=mk(B, T, D, std=2.0, dtype=rt) if res else None,
             z=mk(B, T, D, dtype=ind) if gate else None, alpha=p(alpha, 0.5), gamma_post=p(post, 1.0), beta_post=p(post_b, 0.0),
             gamma_pre=p(pre, 1.0), beta_pre=p(pre_b, 0.0))
    g = {k: device_of(v) for k, v in c.items()}
    for n in ("x", "res", "z"):
        g[n] = dev(spoil(c[n], lens), layout)
    live = None if lens is None else bt.live_rows(lens, B, T)
    return mk, lens, c, g, live


def order(c):
    return [c[n] for n in ("x", "res", "z", "alpha", "gamma_post", "beta_post", "gamma_pre", "beta_pre")]


@pytest.mark.parametrize("case", NORM)
def test_norm_forward(ttt, case):
    B, T, D, ind, rt, kind, gate, first, *_ = case
    _, lens, c, g, live = norm_case(*case)
    s, y = ttt.block_norm_fwd(**g, kind=kind, eps=1e-5, gate_first=first, lens=device_of(lens), res_dtype=rt)
    rs, ry = bt.norm_rounded(*order(c), kind, 1e-5, first, live=live)
    bt.check_rounded("s", s, rs, live)
    assert (y is None) == (ry is None)
    if y is not None:
        bt.check_rounded("y", y, ry, live)
        none, y2 = ttt.block_norm_fwd(**g, kind=kind, eps=1e-5, gate_first=first, lens=device_of(lens), res_dtype=rt, keep=False)
        assert none is None and torch.equal(y2, y)
    if g["res"] is not None:  # the residual stream in place
        res = g["res"].contiguous().clone()
        s2, _ = ttt.block_norm_fwd(**{**g, "res": res}, kind=kind, eps=1e-5, gate_first=first, lens=device_of(lens), s=res)
        assert s2 is res and torch.equal(res, s)


@pytest.mark.parametrize("case", NORM)
def test_norm_backward(ttt, case):
    B, T, D, ind, rt, kind, gate, first, *_ = case
    mk, lens, c, g, live = norm_case(*case, seed=4)
    ds, dy = mk(B, T, D, dtype=rt), mk(B, T, D, dtype=ind) if c["gamma_pre"] is not None else None
    names = ("dx", "dz", "dres", "dalpha", "dgamma_post", "dbeta_post", "dgamma_pre", "dbeta_pre")
    for ds, dy in ((ds, dy), (ds, None), (None, dy)):
        if ds is None and dy is None:
            continue
        if ds is None and c["res"] is None and rt != ind:
            continue  # (nothing then has res_dtype)
        got = ttt.block_norm_bwd(g["x"], dev(spoil(ds, lens), case[-1]), dev(spoil(dy, lens), case[-1]),
                                 **{k: v for k, v in g.items() if k != "x"}, kind=kind, eps=1e-5, gate_first=first,
                                 lens=device_of(lens))
        ref = bt.norm_rounded(*order(c), kind, 1e-5, first, ds=ds, dy=dy, live=live)
        for n, a, r in zip(names, got, ref):
            if r is None:
                assert a is None or not a.any(), n  # (dgamma_pre without dy)
            else:
                bt.check_rounded(n, a, r, live if a.dim() == 3 else None)
