"""How the short convolution, the selective scan and the block norm are called: streams, captured graphs, far offsets, empty
calls, special values, and the three together as one block of a network."""
import pytest

import block_testutil as bt
from test_block_gpu import NAMES, Maker, norm_case, scan_case

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


def calls(ttt, T=70, seed=0):
    """Each entry point once, on inputs of its own: functions of a stream that return the outputs."""
    mk = Maker(seed)
    x, w, b, st = mk(2, T, 72, dtype=BF).cuda(), mk(72, 4).cuda(), mk(72).cuda(), mk(2, 3, 72, dtype=BF).cuda()
    _, _, _, g = scan_case(2, T, 72, 16, 1, BF, BF, True, True, True, True, True, None, "dense", seed)
    dy, dh = mk(2, T, 72, dtype=BF).cuda(), mk(2, 72, 16).cuda()
    _, _, _, n, _ = norm_case(2, T, 72, BF, F32, "layer", True, False, True, True, True, True, True, True, None, "dense", seed)
    ds = mk(2, T, 72).cuda()
    one = {k: (v[:, :1] if k in ("u", "dt", "z") else v[:, :, :1] if k in ("Bm", "Cm") else v) for k, v in g.items() if k != "h0"}

    def conv_token(s):
        state = st.clone() if s is None else st * 1
        return ttt.short_conv_decode(x[:, :1], w, state, bias=b, silu=True, stream=s), state

    def scan_token(s):
        h = g["h0"] * 1
        return ttt.selective_scan_decode(**one, h=h, softplus=True, stream=s), h

    return [lambda s: ttt.short_conv_fwd(x, w, bias=b, state=st, silu=True, stream=s),
            lambda s: ttt.short_conv_bwd(x, w, dy, bias=b, state=st, silu=True, stream=s),
            conv_token,
            lambda s: ttt.selective_scan_fwd(**g, softplus=True, stream=s),
            lambda s: ttt.selective_scan_bwd(**g, dy=dy, dh_final=dh, softplus=True, stream=s),
            scan_token,
            lambda s: ttt.block_norm_fwd(**n, kind="layer", stream=s),
            lambda s: ttt.block_norm_bwd(ds=ds, dy=dy, **n, kind="layer", stream=s)]


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [70, 600])
def test_streams(ttt, T):
    """On torch's current stream, on a side stream behind inputs made there, and on a stream that is handed over."""
    for f in calls(ttt, T):
        ref = f(None)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = f(None)
        s.synchronize()
        assert same(ref, got)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            made = f(s)
        s.synchronize()
        assert same(ref, made)


def test_two_streams_at_once(ttt):
    """Calls of the same kind at the same time: each has a workspace of its own."""
    a, b = calls(ttt, 600, 1), calls(ttt, 600, 2)
    for fa, fb in zip(a, b):
        ra, rb = fa(None), fb(None)
        torch.cuda.synchronize()
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(3):
            with torch.cuda.stream(s):
                ga = fa(None)
            with torch.cuda.stream(t):
                gb = fb(None)
            torch.cuda.synchronize()
            assert same(ra, ga) and same(rb, gb)


@pytest.mark.parametrize("T", [70, 600])
def test_graphs(ttt, T):
    """Captured once, replayed with eager work in between; two graphs with a workspace each."""
    for f in calls(ttt, T):
        ref = [None if x is None else x.clone() for x in f(None)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f(None)
        torch.cuda.current_stream().wait_stream(s)
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = f(None)
            graphs.append((graph, out))
        for _ in range(3):
            for graph, out in graphs:
                for x in out:
                    if x is not None:
                        x.fill_(7)
                graph.replay()
                eager = f(None)
                torch.cuda.synchronize()
                assert same(ref, out) and same(ref, eager)


def test_empty(ttt):
    mk = Maker(5)
    p = {k: mk(8).cuda() for k in ("D", "dt_bias")}
    A, w = -mk(8, 4).abs().cuda(), mk(8, 3).cuda()
    for B, T in ((0, 5), (2, 0), (0, 0)):
        x, bc = torch.zeros(B, T, 8, device="cuda"), torch.zeros(B, 1, T, 4, device="cuda")
        h0, st = mk(B, 8, 4).cuda(), mk(B, 2, 8).cuda()
        y, h = ttt.selective_scan_fwd(x, x, A, bc, bc, z=x, h0=h0, **p)
        assert y.shape == x.shape and torch.equal(h, h0)
        got = ttt.selective_scan_bwd(x, x, A, bc, bc, x, z=x, h0=h0, dh_final=h0, **p)
        assert torch.equal(got[8], h0) and not got[2].any() and not got[5].any() and not got[7].any()
        y, last = ttt.short_conv_fwd(x, w, state=st)
        assert y.shape == x.shape and torch.equal(last, st)
        dx, dw, db, dst = ttt.short_conv_bwd(x, w, x, state=st, dstate_final=st)
        assert torch.equal(dst, st) and not dw.any() and not db.any()
        assert ttt.short_conv_decode(x, w, st).shape == x.shape
        assert ttt.selective_scan_decode(x, x, A, bc, bc, h0).shape == x.shape
        s, y = ttt.block_norm_fwd(x, gamma_pre=p["D"])
        assert s.shape == x.shape == y.shape
        assert not ttt.block_norm_bwd(x, x, x, gamma_pre=p["D"])[6].any()


def far(shape, dtype, step):
    """A [B, T, D] tensor whose sequences lie ``step`` elements apart."""
    B, T, D = shape
    buf = torch.empty((B - 1) * step + T * D, dtype=dtype, device="cuda")
    return buf.as_strided(shape, (step, D, 1))


def test_far_offsets(ttt):
    """Sequences more than 2^31 elements apart, inputs and outputs."""
    mk, B, T, D = Maker(6), 2, 40, 64
    step = (1 << 31) + 8 * 64
    x, y = far((B, T, D), BF, step), far((B, T, D), BF, step)
    x.copy_(mk(B, T, D, dtype=BF))
    near = x.contiguous()
    w = mk(D, 4).cuda()
    assert torch.equal(ttt.short_conv_fwd(x, w, silu=True, y=y)[0], ttt.short_conv_fwd(near, w, silu=True)[0])
    dx = ttt.short_conv_bwd(near, w, near, silu=True)
    got = ttt.short_conv_bwd(x, w, x, silu=True, out=(y, *(torch.empty_like(t) for t in dx[1:])))
    assert same(got, dx)
    _, _, _, g = scan_case(B, T, D, 16, 1, BF, BF, True, False, True, True, False, None, "dense", 6)
    ref = ttt.selective_scan_fwd(**{**g, "u": near}, softplus=True)
    assert same(ttt.selective_scan_fwd(**{**g, "u": x}, softplus=True, y=y), ref)
    ref = ttt.selective_scan_bwd(**{**g, "u": near}, dy=near, softplus=True)
    got = ttt.selective_scan_bwd(**{**g, "u": x}, dy=x, softplus=True,
                                 out=(y, *(None if t is None else torch.empty_like(t) for t in ref[1:])))
    assert same(got, ref)
    ga = mk(D).cuda()
    ref = ttt.block_norm_fwd(near, res=near, gamma_pre=ga)
    assert same(ttt.block_norm_fwd(x, res=x, gamma_pre=ga, s=y), ref)


def test_long_sequence(ttt):
    """Many tokens and few channels: the most segments, and sequences that end in any of them."""
    case = (3, 9000, 10, 6, 2, F32, F32, True, True, True, True, True, None, "dense")
    mk, _, c, g = scan_case(*case, seed=7)
    lens = torch.tensor([9000, 4111, 1], dtype=torch.int32)
    y, h = ttt.selective_scan_fwd(**g, softplus=True, lens=lens.cuda())
    ry, rh = bt.scan(**c, softplus=True, lens=lens)
    my, mh = bt.scan(**c, softplus=True, lens=lens, magnitudes=True)
    k = bt.scan_roundings(9000, 6, 10)[0]
    bt.check("y", y, ry, my, k)
    bt.check("h", h, rh, mh, k)
    # rounding does not add up: a plain fp32 evaluation is this good
    assert ((h.cpu().double() - rh).abs() / mh).max() < 200 * bt.U


def test_decays_at_the_ends(ttt):
    """A = -inf keeps nothing and A = 0 everything; steps from e^-60 to 60; padded rows in between."""
    mk, B, T, D, N = Maker(8), 2, 45, 16, 4
    lens = torch.tensor([45, 20], dtype=torch.int32)
    _, _, c, _ = scan_case(B, T, D, N, 1, F32, F32, True, False, True, False, True, None, "dense", 8)
    c["A"][:, 0], c["A"][:, 1] = -float("inf"), 0.0
    c["dt"] = mk(B, T, D) * 20
    g = {k: None if v is None else v.cuda() for k, v in c.items()}
    y, h = ttt.selective_scan_fwd(**g, softplus=True, lens=lens.cuda())
    ry, rh = bt.scan(**c, softplus=True, lens=lens)
    my, mh = bt.scan(**c, softplus=True, lens=lens, magnitudes=True)
    k = bt.scan_roundings(T, N, D)[0] + 64  # steps to 80: their exponents' rounding
    bt.check("y", y, ry, my, k)
    bt.check("h", h, rh, mh, k)
    dy = mk(B, T, D)
    got = ttt.selective_scan_bwd(**g, dy=dy.cuda(), softplus=True, lens=lens.cuda())
    ref = bt.scan(**c, softplus=True, lens=lens, dy=dy)
    size = bt.scan(**c, softplus=True, lens=lens, dy=dy, magnitudes=True)
    k = bt.scan_roundings(T, N, D)[1] + 128 + B * T
    for n, a, r, s in zip(NAMES, got, ref, size):
        if a is not None:
            bt.check(n, a, r, s, k)
    h2 = g["h0"].clone()
    z = ttt.selective_scan_decode(**{k: v for k, v in g.items() if k != "h0"}, h=h2, softplus=True, lens=lens.cuda())
    bt.check("tokens y", z, ry, my, bt.scan_roundings(T, N, D)[0] + 64)
    bt.check("tokens h", h2, rh, mh, bt.scan_roundings(T, N, D)[0] + 64)


def test_nan_stays_in_its_sequence_and_channel(ttt):
    """A NaN reaches its channel from its token on, and nothing else."""
    _, _, _, g = scan_case(2, 50, 70, 16, 1, F32, F32, True, True, True, True, True, None, "dense", 9)
    y0, h0 = ttt.selective_scan_fwd(**g, softplus=True)
    u = g["u"].clone()
    u[1, 20, 66] = float("nan")
    y, h = ttt.selective_scan_fwd(**{**g, "u": u}, softplus=True)
    assert torch.isnan(y[1, 20:, 66]).all() and torch.isnan(h[1, 66]).all()
    y[1, 20:, 66], h[1, 66] = y0[1, 20:, 66], h0[1, 66]
    assert torch.equal(y, y0) and torch.equal(h, h0)
    x, w = g["u"], torch.ones(70, 4, device="cuda")
    c0, _ = ttt.short_conv_fwd(x, w)
    c, _ = ttt.short_conv_fwd(u, w)
    assert torch.isnan(c[1, 20:24, 66]).all()
    c[1, 20:24, 66] = c0[1, 20:24, 66]
    assert torch.equal(c, c0)
    ga = torch.ones(70, device="cuda")
    n0, n = (ttt.block_norm_fwd(t, gamma_pre=ga)[1] for t in (x, u))
    assert torch.isnan(n[1, 20]).all()
    n[1, 20] = n0[1, 20]
    assert torch.equal(n, n0)


class Block:
    """res, x -> res, x: norm, projections, convolution, scan, gated join: what a network calls, forward and backward, from
    one set of functions for the kernels and for plain 64 bits."""

    def __init__(self, D=48, N=16, seed=10):
        mk = Maker(seed)
        E, R = 2 * D, 4
        self.N, self.R, self.E = N, R, E
        self.p = dict(gamma=mk(D, std=0.1, mean=1), win=mk(D, 2 * E, std=D ** -0.5), w=mk(E, 4, std=0.5), b=mk(E, std=0.1),
                      wx=mk(E, R + 2 * N, std=E ** -0.5), wdt=mk(R, E, std=R ** -0.5), dtb=mk(E, std=0.3, mean=-3), logA=mk(E, N, std=0.5),
                      D=mk(E, std=0.1, mean=1), post=mk(E, std=0.1, mean=1), wout=mk(E, D, std=E ** -0.5), alpha=mk(D, std=0.1, mean=0.5))

    def plain(self, x, p):
        """In the parameters' own type, differentiable."""
        E, N, R = self.E, self.N, self.R
        _, n = bt.norm(x, gamma_pre=p["gamma"])
        uz = n @ p["win"]
        u, z = uz[..., :E], uz[..., E:]
        rows = torch.cat([torch.zeros_like(u[:, :3]), u], 1)
        c = bt.silu(sum(p["w"][:, j] * rows[:, j:j + u.shape[1]] for j in range(4)) + p["b"])
        q = c @ p["wx"]
        step = torch.nn.functional.softplus(q[..., :R] @ p["wdt"] + p["dtb"])
        h, ys = torch.zeros(x.shape[0], E, N, dtype=x.dtype), []
        A = -torch.exp(p["logA"])
        for t in range(x.shape[1]):
            h = torch.exp(step[:, t, :, None] * A) * h + (step[:, t] * c[:, t])[..., None] * q[:, t, None, R:R + N]
            ys.append((h * q[:, t, None, R + N:]).sum(-1) + p["D"] * c[:, t])
        # the norm behind the scan and its gate, then the projection and the residual sum
        v, _ = bt.norm(torch.stack(ys, 1), z=z, gamma_post=p["post"])
        return bt.norm(v @ p["wout"], res=x, alpha=p["alpha"])[0]

    def forward(self, ttt, x, p):
        E, N, R = self.E, self.N, self.R
        k = {"x": x}
        _, k["n"] = ttt.block_norm_fwd(x, gamma_pre=p["gamma"], keep=False)
        uz = k["n"] @ p["win"]
        k["u"], k["z"] = uz[..., :E], uz[..., E:]
        k["c"], k["conv"] = ttt.short_conv_fwd(k["u"], p["w"], p["b"], silu=True)
        k["q"] = k["c"] @ p["wx"]
        k["dt"] = k["q"][..., :R] @ p["wdt"]
        bc = k["q"].unsqueeze(1)
        k["Bm"], k["Cm"] = bc[..., R:R + N], bc[..., R + N:]
        k["A"] = -torch.exp(p["logA"])
        k["y"], k["h"] = ttt.selective_scan_fwd(k["c"], k["dt"], k["A"], k["Bm"], k["Cm"], D=p["D"], dt_bias=p["dtb"], softplus=True)
        k["v"], _ = ttt.block_norm_fwd(k["y"], z=k["z"], gamma_post=p["post"])
        k["o"] = k["v"] @ p["wout"]
        s, _ = ttt.block_norm_fwd(k["o"], res=x, alpha=p["alpha"])
        return s, k

    def token(self, ttt, x, p, k):
        E, N, R = self.E, self.N, self.R
        _, n = ttt.block_norm_fwd(x, gamma_pre=p["gamma"], keep=False)
        uz = n @ p["win"]
        c = ttt.short_conv_decode(uz[..., :E], p["w"], k["conv"], p["b"], silu=True)
        q = c @ p["wx"]
        bc = q.unsqueeze(1)
        y = ttt.selective_scan_decode(c, q[..., :R] @ p["wdt"], k["A"], bc[..., R:R + N], bc[..., R + N:], k["h"], D=p["D"],
                                      dt_bias=p["dtb"], softplus=True)
        v, _ = ttt.block_norm_fwd(y, z=uz[..., E:], gamma_post=p["post"])
        return ttt.block_norm_fwd(v @ p["wout"], res=x, alpha=p["alpha"])[0]

    def backward(self, ttt, ds, p, k):
        g = {}
        flat = lambda a, b: a.flatten(0, 1).t() @ b.flatten(0, 1)  # noqa: E731
        do, _, dx, g["alpha"], *_ = ttt.block_norm_bwd(k["o"], ds, None, res=k["x"], alpha=p["alpha"])
        g["wout"] = flat(k["v"], do)
        dv = do @ p["wout"].t()
        dy, dz, _, _, g["post"], *_ = ttt.block_norm_bwd(k["y"], dv, None, z=k["z"], gamma_post=p["post"])
        dc, ddt, dA, dB, dC, g["D"], _, g["dtb"], _ = ttt.selective_scan_bwd(
            k["c"], k["dt"], k["A"], k["Bm"], k["Cm"], dy, D=p["D"], dt_bias=p["dtb"], softplus=True)
        g["logA"] = dA * k["A"]
        g["wdt"] = flat(k["q"][..., :self.R], ddt)
        dq = torch.cat([ddt @ p["wdt"].t(), dB[:, 0], dC[:, 0]], -1)
        g["wx"] = flat(k["c"], dq)
        dc = dc + dq @ p["wx"].t()
        du, g["w"], g["b"], _ = ttt.short_conv_bwd(k["u"], p["w"], dc, p["b"], silu=True)
        duz = torch.cat([du, dz], -1)
        g["win"] = flat(k["n"], duz)
        dn = duz @ p["win"].t()
        dx2, _, _, _, _, _, g["gamma"], _ = ttt.block_norm_bwd(k["x"], None, dn, gamma_pre=p["gamma"])
        return dx + dx2, g


@pytest.mark.parametrize("B,T", [(2, 37), (1, 500)])
def test_block(ttt, B, T):
    """One block of a network from the three operators, fp32: outputs and every gradient against 64 bits, no further off than
    a few times what plain fp32 on the CPU is (the same chain with as many roundings, in another order: a factor of 8 and 2^-22 of
    the largest value)."""
    block, mk = Block(), Maker(11)
    x, ds = mk(B, T, 48), mk(B, T, 48)
    p = {n: v.cuda() for n, v in block.p.items()}
    s, k = block.forward(ttt, x.cuda(), p)
    dx, g = block.backward(ttt, ds.cuda(), p, k)

    def reference(dtype):
        leaves = {n: v.to(dtype).requires_grad_() for n, v in block.p.items()}
        xs = x.to(dtype).requires_grad_()
        out = block.plain(xs, leaves)
        grads = torch.autograd.grad(out, [xs, *leaves.values()], ds.to(dtype))
        return [out.detach(), *grads]

    exact, plain = reference(torch.float64), reference(F32)
    for n, a, r, f in zip(["s", "dx", *block.p], [s, dx, *(g[m] for m in block.p)], exact, plain):
        off, own = (a.cpu().double() - r).abs().max().item(), (f.double() - r).abs().max().item()
        print(f"{n}: off {off:.2e}, plain fp32 {own:.2e}", flush=True)
        assert off <= 8 * own + 2.0 ** -22 * r.abs().max().item(), n


def test_block_token_by_token(ttt):
    """Generating behind a prompt gives what the whole sequence in one call gives."""
    block, mk, B, T = Block(seed=12), Maker(13), 3, 40
    x = mk(B, T, 48)
    p = {n: v.cuda() for n, v in block.p.items()}
    whole = block.plain(x.double(), {n: v.double() for n, v in block.p.items()})
    own = (block.plain(x, block.p).double() - whole).abs().max().item()
    _, k = block.forward(ttt, x[:, :20].cuda(), p)
    got = [block.token(ttt, x[:, t:t + 1].cuda(), p, k) for t in range(20, T)]
    off = (torch.cat(got, 1).cpu().double() - whole[:, 20:]).abs().max().item()
    print(f"tokens: off {off:.2e}, plain fp32 {own:.2e}", flush=True)
    assert off <= 8 * own + 2.0 ** -22 * whole.abs().max().item()
