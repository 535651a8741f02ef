"""Linear attention with a decay per head on the GPU: forward, backward and decode
against the recurrence in 64 bits (attn_testutil: the bounds count the roundings)."""
import itertools

import pytest

from attn_testutil import attn, attn_grads, check, tolerance, turn

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


def rows(gen, B, H, T, d, dtype, layout="bhtd", std=1.0):
    x = (torch.randn(B, H, T, d, generator=gen) * std).to(dtype)
    return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "bthd" else x


def case(B, H, Hkv, T, d, dtype, w0="each", layout="bhtd", lens=None, seed=0, scale=1.0, g=None):
    gen = torch.Generator().manual_seed(1000 + seed)
    c = dict(q=rows(gen, B, H, T, d, dtype, layout), k=rows(gen, B, Hkv, T, d, dtype, layout, d ** -0.5),
             v=rows(gen, B, Hkv, T, d, dtype, layout),
             log_decay=-torch.exp2(-10 * torch.rand(H, generator=gen)) if g is None else torch.tensor(g, dtype=F32),
             scale=scale)
    c["w0"] = {"none": None, "shared": torch.randn(H, d, d, generator=gen),
               "each": torch.randn(B, H, d, d, generator=gen)}[w0]
    c["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return c


def on_gpu(c):
    return {n: x.to(DEV) if torch.is_tensor(x) else x for n, x in c.items()}


def size_of(c):
    """the same call on magnitudes"""
    return {n: x.abs() if torch.is_tensor(x) and n not in ("log_decay", "lens") else abs(x) if n == "scale" else x
            for n, x in c.items()}


def check_fwd(ttt, c, out, **more):
    z, w = ttt.linear_attn_fwd(**on_gpu(c), out_dtype=out, **more)
    assert z.dtype == out and w.dtype == F32
    zr, wr = attn(**c)
    za, wa = attn(**size_of(c))
    d, T = c["q"].shape[3], c["q"].shape[2]
    split = c["q"].dtype == BF16 and out == BF16
    check("Z", z, zr, tolerance(zr, za, d, T, out, split))
    check("W_final", w, wr, tolerance(wr, wa, d, T, F32))
    return z, w


def check_bwd(ttt, c, out, dw=True, **more):
    B, H, T, d = c["q"].shape
    gen = torch.Generator().manual_seed(77)
    dz = rows(gen, B, H, T, d, out)
    dwf = torch.randn(B, H, d, d, generator=gen) if dw else None
    got = ttt.linear_attn_bwd(**on_gpu(c), dz=dz.to(DEV), dw_final=None if dwf is None else dwf.to(DEV), **more)
    ref = attn_grads(**c, dz=dz, dw_final=dwf)
    size = attn_grads(**c, dz=dz, dw_final=dwf, magnitudes=True)
    split = c["q"].dtype == BF16 and out == BF16
    group = H // c["k"].shape[1]
    for i, name in enumerate(("dq", "dk", "dv", "dlog_decay", "dw0")):
        to = out if i < 3 else F32
        assert got[i].dtype == to
        check(name, got[i], ref[i], tolerance(ref[i], size[i], d, T, to, split and i < 4, group))
    return got


# lengths around the block (16) and chunk (32), segments (from 353 tokens on with this few chains), odd ones
LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 300, 515]


@pytest.mark.parametrize("T", LENGTHS)
def test_forward_lengths(ttt, T):
    check_fwd(ttt, case(1, 2, 2, T, 64, BF16, seed=T), BF16)


@pytest.mark.parametrize("d,dtype,out", list(itertools.product([16, 32, 64, 128], [BF16, F32], [BF16, F32])))
def test_forward_types(ttt, d, dtype, out):
    check_fwd(ttt, case(2, 3, 3, 77, d, dtype, seed=d, w0="shared"), out)
    check_fwd(ttt, case(1, 2, 1, 290, d, dtype, seed=d + 1, w0="none", scale=-0.3), out)


@pytest.mark.parametrize("T", LENGTHS)
def test_backward_lengths(ttt, T):
    check_bwd(ttt, case(1, 2, 2, T, 64, BF16, seed=T), BF16)


@pytest.mark.parametrize("d,dtype,out", list(itertools.product([16, 32, 64, 128], [BF16, F32], [BF16, F32])))
def test_backward_types(ttt, d, dtype, out):
    check_bwd(ttt, case(2, 3, 3, 77, d, dtype, seed=d, w0="shared"), out)
    check_bwd(ttt, case(1, 4, 2, 290, d, dtype, seed=d + 1, w0="none", scale=-0.3), out, dw=False)


# segments of 3 or 4 chunks whose states the workgroups carry over themselves, then so many that a launch does
@pytest.mark.parametrize("d,dtype,T", [(32, F32, 200), (128, BF16, 330), (64, BF16, 384), (16, BF16, 1000),
                                       (128, BF16, 800), (64, F32, 1500), (64, BF16, 2081), (32, F32, 2300),
                                       (16, BF16, 3200)])
def test_segments(ttt, d, dtype, T):
    for lens in (None, [T * 2 // 3, T - 1]):
        c = case(2, 2, 1, T, d, dtype, seed=T, lens=lens)
        check_fwd(ttt, c, dtype)
        check_bwd(ttt, c, dtype)


DECAYS = [0.0, float("-inf"), -1e-7, -1e-3, -0.7, -30.0, -1e4, 1e-3]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decays(ttt, dtype):
    """from keeping everything to keeping nothing, and a growing state"""
    for T in (40, 300):
        c = case(1, len(DECAYS), 1, T, 32, dtype, g=DECAYS)
        check_fwd(ttt, c, F32)
        check_bwd(ttt, c, F32)


def test_slow_decays_keep_their_accuracy(ttt):
    """4096 tokens with lambda = 1 - 1e-5: the powers of lambda over the chunks do not drift."""
    check_fwd(ttt, case(1, 1, 1, 4096, 16, BF16, g=[-1e-5], seed=3), F32)


LENS = [0, 1, 16, 31, 33, 127, 128, 129, 300, -4, 1000]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [300, 40])
def test_padded_batches(ttt, dtype, T):
    """Rows behind a sequence's end hold NaN and infinities: not read, and zero in Z and the gradients."""
    B = len(LENS)
    c = case(B, 2, 1, T, 32, dtype, lens=LENS, seed=9)
    dirty = dict(c)
    for n in ("q", "k", "v"):
        dirty[n] = c[n].clone()
        for b, m in enumerate(LENS):
            dirty[n][b, :, max(m, 0):] = float("nan") if b % 2 else float("inf")
            c[n][b, :, max(m, 0):] = 0
    z, w = ttt.linear_attn_fwd(**on_gpu(dirty), out_dtype=dtype)
    zr, wr = attn(**c)
    za, wa = attn(**size_of(c))
    check("Z", z, zr, tolerance(zr, za, 32, T, dtype, dtype == BF16))
    check("W_final", w, wr, tolerance(wr, wa, 32, T, F32))
    for b, m in enumerate(LENS):
        assert (z[b, :, max(m, 0):] == 0).all()
    dz = torch.randn(c["q"].shape, generator=torch.Generator().manual_seed(1)).to(dtype)
    dwf = torch.randn(w.shape, generator=torch.Generator().manual_seed(2))
    dirty_dz = dz.clone()
    for b, m in enumerate(LENS):
        dirty_dz[b, :, max(m, 0):] = float("nan")
    got = ttt.linear_attn_bwd(**on_gpu(dirty), dz=dirty_dz.to(DEV), dw_final=dwf.to(DEV))
    ref, size = (attn_grads(**c, dz=dz, dw_final=dwf, magnitudes=m) for m in (False, True))
    for i, name in enumerate(("dq", "dk", "dv", "dlog_decay", "dw0")):
        to = dtype if i < 3 else F32
        check(name, got[i], ref[i], tolerance(ref[i], size[i], 32, T, to, dtype == BF16 and i < 4, 2))
    for b, m in enumerate(LENS):
        assert all((x[b, :, max(m, 0):] == 0).all() for x in got[:3])


@pytest.mark.parametrize("H,Hkv", [(4, 4), (4, 2), (6, 1), (5, 5)])
def test_shared_heads(ttt, H, Hkv):
    for T in (45, 260):
        c = case(2, H, Hkv, T, 32, BF16, seed=H)
        check_fwd(ttt, c, BF16)
        check_bwd(ttt, c, BF16)


def test_no_tokens(ttt):
    c = on_gpu(case(2, 4, 2, 0, 32, BF16))
    z, w = ttt.linear_attn_fwd(**c)
    assert z.shape == (2, 4, 0, 32) and torch.equal(w, c["w0"])
    z, w = ttt.linear_attn_fwd(**{**c, "w0": None})
    assert (w == 0).all()
    dwf = torch.randn(2, 4, 32, 32, device=DEV)
    dq, dk, dv, dg, dw0 = ttt.linear_attn_bwd(**c, dz=c["q"], dw_final=dwf)
    assert torch.equal(dw0, dwf) and (dg == 0).all() and dk.shape == (2, 2, 0, 32)
    w = c["w0"].clone()
    assert ttt.linear_attn_decode(c["q"], c["k"], c["v"], c["log_decay"], w).shape == (2, 4, 0, 32)
    assert torch.equal(w, c["w0"])
    none = {n: c[n][:0] for n in ("q", "k", "v")}
    z, w = ttt.linear_attn_fwd(**none, log_decay=c["log_decay"])
    assert z.shape == (0, 4, 0, 32) and w.shape == (0, 4, 32, 32)


@pytest.mark.parametrize("T", [50, 300])
def test_layouts(ttt, T):
    """[B, T, H, d] views, slices of one projection, a repeated k, and outputs in such places"""
    c = case(2, 4, 4, T, 32, BF16, seed=4)
    ref = check_fwd(ttt, c, BF16)
    gref = check_bwd(ttt, c, BF16)
    g = on_gpu(c)
    t = {**g, **{n: g[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"}}
    z, w = ttt.linear_attn_fwd(**t, out_dtype=BF16)
    assert torch.equal(z, ref[0]) and torch.equal(w, ref[1]) and z.stride() == t["q"].stride()
    packed = torch.stack([g[n].transpose(1, 2) for n in "qkv"], 2)  # [B, T, 3, H, d]
    p = {**g, **{n: packed[:, :, i].transpose(1, 2) for i, n in enumerate("qkv")}}
    out = torch.full((2, T, 4, 64), float("nan"), device=DEV, dtype=BF16)
    z, w = ttt.linear_attn_fwd(**p, z=out[..., 32:].transpose(1, 2))
    assert torch.equal(z, ref[0]) and torch.equal(w, ref[1]) and out[..., :32].isnan().all()
    grads = torch.empty_like(packed)
    gen = torch.Generator().manual_seed(77)
    dz = rows(gen, 2, 4, T, 32, BF16).to(DEV)
    dwf = torch.randn(2, 4, 32, 32, generator=gen).to(DEV)
    places = tuple(grads[:, :, i].transpose(1, 2) for i in range(3))
    got = ttt.linear_attn_bwd(**p, dz=dz, dw_final=dwf, out=(*places, torch.empty_like(gref[3]), torch.empty_like(gref[4])))
    assert all(torch.equal(x, y) for x, y in zip(got, gref))
    one = {**c, "k": c["k"][:1].expand(2, 4, T, 32), "v": c["v"][:, :, :1].expand(2, 4, T, 32)}
    check_fwd(ttt, one, BF16)
    check_bwd(ttt, one, BF16)


def test_state_in_place_and_continued(ttt):
    """W_final over W0, with segments running at the same time; a prompt in two calls"""
    c = on_gpu(case(1, 2, 2, 700, 64, BF16, seed=8))
    z, w = ttt.linear_attn_fwd(**c)
    state = c["w0"].clone()
    z2, w2 = ttt.linear_attn_fwd(**{**c, "w0": state}, w_final=state)
    assert w2 is state and torch.equal(z, z2) and torch.equal(w, state)
    state = c["w0"].clone()
    parts = []
    for t in (slice(0, 411), slice(411, 700)):
        part = {**c, "w0": state, **{n: c[n][:, :, t].contiguous() for n in "qkv"}}
        parts.append(ttt.linear_attn_fwd(**part, w_final=state)[0])
    cc = {n: x.cpu() if torch.is_tensor(x) else x for n, x in c.items()}
    (zr, wr), (za, wa) = attn(**cc), attn(**size_of(cc))
    check("Z", torch.cat(parts, 2), zr, tolerance(zr, za, 64, 700, F32))
    check("W", state, wr, tolerance(wr, wa, 64, 700, F32))


# ---- decode ------------------------------------------------------------------

@pytest.mark.parametrize("d,dtype,out", list(itertools.product([16, 32, 64, 128], [BF16, F32], [BF16, F32])))
def test_decode_types(ttt, d, dtype, out):
    for T in (1, 3, 8, 19):
        c = case(3, 4, 2, T, d, dtype, lens=[T, 0, (T + 1) // 2], seed=d, scale=0.5)
        g = on_gpu(c)
        w = g.pop("w0").clone()
        z = ttt.linear_attn_decode(**g, w=w, out_dtype=out)
        (zr, wr), (za, wa) = attn(**c), attn(**size_of(c))
        check("Z", z, zr, tolerance(zr, za, d, T, out))
        check("W", w, wr, tolerance(wr, wa, d, T, F32))
        assert torch.equal(w[1].cpu(), c["w0"][1]) and (z[1] == 0).all()


def test_decode_unaligned(ttt):
    """rows at any address: columns of a wider tensor"""
    c = case(2, 2, 2, 5, 16, BF16)
    g = on_gpu(c)
    w = g.pop("w0").clone()
    z = ttt.linear_attn_decode(**g, w=w)
    wide = {n: torch.cat([g[n][..., :3], g[n], g[n][..., :2]], -1)[..., 3:19] for n in "qkv"}
    w2 = c["w0"].to(DEV)
    z2 = ttt.linear_attn_decode(**{**g, **wide}, w=w2)
    assert torch.equal(z, z2) and torch.equal(w, w2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_with_positions(ttt, layout, dtype):
    B, H, T, d, rot = 3, 4, 3, 32, 24
    c = case(B, H, 2, T, d, dtype, seed=2)
    freqs, scale = ttt.rotary_freqs(rot, scaling="yarn", factor=4.0)
    pos = torch.tensor([0, 1000003, 77])
    each = pos[:, None] + torch.arange(T)
    turned = dict(c)
    for n in "qk":
        turned[n] = turn(c[n], each, freqs, layout, scale)
    (zr, wr), (za, wa) = attn(**turned), attn(**size_of({n: x for n, x in turned.items()}))
    # a turned value is at most sqrt(2) scale times its pair and carries at most 8 roundings of that size
    size = {**size_of(c), "q": c["q"].abs().amax(-1, keepdim=True).expand_as(c["q"]) * 2 * scale,
            "k": c["k"].abs().amax(-1, keepdim=True).expand_as(c["k"]) * 2 * scale}
    za, wa = attn(**size)
    for p in (pos.to(DEV), each.to(DEV)):
        g = on_gpu(c)
        w = g.pop("w0").clone()
        z = ttt.linear_attn_decode(**g, w=w, rope=(p, freqs.to(DEV), layout, scale))
        check("Z", z, zr, tolerance(zr, za, d, T, F32))
        check("W", w, wr, tolerance(wr, wa, d, T, F32))
    # one start for all
    g = on_gpu(c)
    w, w2 = g["w0"].clone(), g.pop("w0").clone()
    z = ttt.linear_attn_decode(**g, w=w, rope=(5, freqs.to(DEV), layout, scale))
    z2 = ttt.linear_attn_decode(**g, w=w2, rope=(torch.full((B,), 5, device=DEV), freqs.to(DEV), layout, scale))
    assert torch.equal(z, z2) and torch.equal(w, w2)


def test_prompt_then_tokens(ttt):
    """The operators as a model runs them: the prompt's q and k turned, the chunked forward, then single
    tokens turned in the decode call, against one recurrence over all tokens."""
    B, H, Hkv, T, d, P = 2, 4, 2, 150, 64, 141
    c = case(B, H, Hkv, T, d, F32, w0="none", seed=12)
    freqs, scale = ttt.rotary_freqs(d, scaling="ntk", factor=2.0)
    at = torch.arange(T).expand(B, T)
    t = {**c, **{n: turn(c[n], at, freqs, "half", scale) for n in "qk"}}
    (zr, wr) = attn(**t)
    size = {**size_of(c), "q": c["q"].abs().amax(-1, keepdim=True).expand_as(c["q"]) * 2,
            "k": c["k"].abs().amax(-1, keepdim=True).expand_as(c["k"]) * 2}
    za, wa = attn(**size)
    g, f = on_gpu(c), freqs.to(DEV)
    q, k = ttt.rotary(g["q"][:, :, :P], g["k"][:, :, :P], 0, f, scale=scale)
    z, w = ttt.linear_attn_fwd(q, k, g["v"][:, :, :P], g["log_decay"])
    zs = [z]
    for p in range(P, T):
        zs.append(ttt.linear_attn_decode(*(g[n][:, :, p:p + 1] for n in "qkv"), g["log_decay"], w, rope=(p, f, "half", scale)))
    check("Z", torch.cat(zs, 2), zr, tolerance(zr, za, d, T, F32))
    check("W", w, wr, tolerance(wr, wa, d, T, F32))


def test_training_step(ttt):
    """A chain of the operators trained through: L = <dz, attn(rotary(q), rotary(k), v)>, its gradients against
    differences of the GPU forward.  L is linear in each of q, k, v and w0, so a central difference of any
    length is the derivative up to rounding."""
    B, H, Hkv, T, d = 1, 4, 2, 90, 32
    c = on_gpu(case(B, H, Hkv, T, d, F32, seed=14))
    f, s = ttt.rotary_freqs(16, device=DEV)
    gen = torch.Generator().manual_seed(15)
    dz = torch.randn(B, H, T, d, generator=gen).to(DEV)
    dwf = torch.randn(B, H, d, d, generator=gen).to(DEV)

    def loss(c):
        q, k = ttt.rotary(c["q"], c["k"], 3, f, scale=s)
        z, w = ttt.linear_attn_fwd(**{**c, "q": q, "k": k})
        return (z.double() * dz.double()).sum().item() + (w.double() * dwf.double()).sum().item()

    q, k = ttt.rotary(c["q"], c["k"], 3, f, scale=s)
    dq, dk, dv, dg, dw0 = ttt.linear_attn_bwd(**{**c, "q": q, "k": k}, dz=dz, dw_final=dwf)
    dq, dk = ttt.rotary_bwd(dq, dk, 3, f, scale=s)
    cc = {n: x.cpu() if torch.is_tensor(x) else x for n, x in c.items()}
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("w0", dw0)):
        way = torch.randn(c[name].shape, generator=gen).to(DEV)
        up, down = (loss({**c, name: c[name] + e * way}) for e in (1.0, -1.0))
        # both losses are sums over z and w, each term within its bound; pairs under sqrt(2) of a turned value
        size = size_of({**cc, name: cc[name].abs() + way.cpu().abs()})
        za, wa = attn(**size)
        tol = 2 * sum((tolerance(torch.zeros_like(x), x, d, T, F32) * y.cpu().abs()).sum().item()
                      for x, y in ((za, dz), (wa, dwf)))
        want = (grad.double() * way.double()).sum().item()
        print(f"{name}: difference {(up - down) / 2:.8g}, gradient {want:.8g}, bound {tol:.2g}", flush=True)
        assert abs((up - down) / 2 - want) <= tol


# ---- streams, graphs, determinism ----------------------------------------------

def test_same_bits_every_time(ttt):
    c = on_gpu(case(2, 4, 2, 600, 64, BF16, seed=20))
    dz = torch.randn(2, 4, 600, 64, device=DEV).to(BF16)
    a = [*ttt.linear_attn_fwd(**c), *ttt.linear_attn_bwd(**c, dz=dz)]
    torch.empty(1 << 26, device=DEV).fill_(float("nan"))  # the next workspaces hold something else
    b = [*ttt.linear_attn_fwd(**c), *ttt.linear_attn_bwd(**c, dz=dz)]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_side_stream(ttt):
    c = on_gpu(case(2, 4, 2, 600, 64, BF16, seed=21))
    dz = torch.randn(2, 4, 600, 64, device=DEV).to(BF16)
    ref = [*ttt.linear_attn_fwd(**c), *ttt.linear_attn_bwd(**c, dz=dz)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cc = {**c, "q": c["q"].clone()}
        got = [*ttt.linear_attn_fwd(**cc), *ttt.linear_attn_bwd(**cc, dz=dz)]
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    with torch.cuda.stream(s):
        v = c["v"].clone()
    cc = {**c, "v": v}
    got = [*ttt.linear_attn_fwd(**cc, stream=s), *ttt.linear_attn_bwd(**cc, dz=dz, stream=s)]
    other = torch.full((1 << 24,), float("nan"), device=DEV)  # the current stream goes on
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got)) and other.isnan().all()


def test_graphs(ttt):
    """Two captured calls, each with its own workspace, replayed in turn with eager work between"""
    cases = [on_gpu(case(1, 2, 1, 700, 64, BF16, seed=s)) for s in (30, 31)]
    dzs = [torch.randn(1, 2, 700, 64, device=DEV).to(BF16) for _ in cases]

    def step(c, dz):
        return [*ttt.linear_attn_fwd(**c), *ttt.linear_attn_bwd(**c, dz=dz)]

    refs = [step(c, dz) for c, dz in zip(cases, dzs)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, dz in zip(cases, dzs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c, dz))
        graphs.append(g)
    for i in range(3):
        for o in outs:
            for x in o:
                x.fill_(float("nan"))
        eager = step(cases[0], dzs[0])
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert all(torch.equal(x, y) for x, y in zip(o, r)), f"replay {i}"
        assert all(torch.equal(x, y) for x, y in zip(eager, refs[0]))


def test_decode_graph(ttt):
    """A captured token: the state and the positions move on with each replay."""
    B, H, d = 3, 2, 64
    c = on_gpu(case(B, H, H, 8, d, BF16, seed=33))
    f, s = ttt.rotary_freqs(d, device=DEV)
    w, w2 = c["w0"].clone(), c["w0"].clone()
    pos = torch.tensor([4, 0, 9], device=DEV)
    q, k, v = (torch.empty_like(c[n][:, :, :1]) for n in "qkv")
    z = torch.empty(B, H, 1, d, device=DEV)

    def token():
        ttt.linear_attn_decode(q, k, v, c["log_decay"], w, rope=(pos, f, "half", s), z=z)
        pos.add_(1)

    for x in (q, k, v):
        x.zero_()
    state = w.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        token()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        token()
    w.copy_(state)
    pos.copy_(torch.tensor([4, 0, 9]))
    for t in range(8):
        for x, n in ((q, "q"), (k, "k"), (v, "v")):
            x.copy_(c[n][:, :, t:t + 1])
        g.replay()
        ref = ttt.linear_attn_decode(*(c[n][:, :, t:t + 1] for n in "qkv"), c["log_decay"], w2,
                                     rope=(torch.tensor([4 + t, t, 9 + t], device=DEV), f, "half", s))
        torch.cuda.synchronize()
        assert torch.equal(z, ref) and torch.equal(w, w2), f"token {t}"


def test_offsets_past_32_bits(ttt):
    """Rows 2^17 elements apart, 20000 tokens: offsets beyond 2^31 elements, in q, k, v and z"""
    T, d = 20000, 16
    wide = torch.zeros(T, 1 << 17, device=DEV, dtype=BF16)
    gen = torch.Generator(device=DEV).manual_seed(3)
    views = {n: wide[:, 64 * i:64 * i + d][None, None] for i, n in enumerate("qkv")}
    for x in views.values():
        x.copy_(torch.randn(1, 1, T, d, generator=gen, device=DEV).to(BF16))
    g = torch.tensor([-0.01], device=DEV)
    z, w = ttt.linear_attn_fwd(**{n: x.contiguous() for n, x in views.items()}, log_decay=g, out_dtype=BF16)
    out = wide[:, 1024:1024 + d][None, None]
    z2, w2 = ttt.linear_attn_fwd(**views, log_decay=g, z=out)
    assert torch.equal(z, z2) and torch.equal(w, w2)
    grads = tuple(wide[:, 2048 + 64 * i:2048 + 64 * i + d][None, None] for i in range(3))
    a = ttt.linear_attn_bwd(**{n: x.contiguous() for n, x in views.items()}, log_decay=g, dz=z)
    b = ttt.linear_attn_bwd(**views, log_decay=g, dz=out, out=(*grads, torch.empty_like(a[3]), torch.empty_like(a[4])))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_on_the_gpu(ttt):
    c = on_gpu(case(1, 2, 2, 32, 64, BF16))
    with pytest.raises(ValueError, match="contiguous"):
        ttt.linear_attn_fwd(**{**c, "q": c["q"].transpose(2, 3).contiguous().transpose(2, 3)})
    with pytest.raises(ttt.TTTError) as e:
        ttt.linear_attn_fwd(**{**c, **{n: c[n][..., :48] for n in "qkv"}, "w0": None})
    assert e.value.status == 4
    with pytest.raises(ttt.TTTError) as e:
        ttt.linear_attn_fwd(**c, z=c["q"])
    assert e.value.status == 5
    wide = torch.zeros(1, 2, 32, 65, device=DEV, dtype=BF16)
    with pytest.raises(ttt.TTTError) as e:
        ttt.linear_attn_fwd(**{**c, "q": wide[..., 1:]})
    assert e.value.status == 6
    with pytest.raises(ttt.TTTError) as e:
        ttt.linear_attn_fwd(**on_gpu(case(1, 1, 1, 4096, 16, BF16)), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 11
    with pytest.raises(ValueError, match="one GPU"):
        ttt.linear_attn_fwd(**{**c, "log_decay": c["log_decay"].cpu()})


def test_decode_zero_rows_past_32_bits(ttt):
    # 2^24 + 8 rows of 128 elements, of which one sequence has a token: the rows behind it are zero to the last
    T, d = (1 << 24) + 8, 128
    gen = torch.Generator().manual_seed(5)
    row = torch.randn(3, 1, 1, 1, d, generator=gen).to(BF16).cuda()
    q, k, v = (x.expand(1, 1, T, d) for x in row)
    w = torch.zeros(1, 1, d, d, device="cuda")
    z = torch.full((1, 1, T, d), 7.0, dtype=BF16, device="cuda")
    ttt.linear_attn_decode(q, k, v, torch.zeros(1, device="cuda"), w, lens=torch.tensor([1], dtype=torch.int32).cuda(), z=z)
    assert torch.equal(w[0, 0], row[2].float().reshape(d, 1) * row[1].float().reshape(1, d))
    assert z[0, 0, 0].abs().max() > 0
    for part in z[0, 0, 1:].split(1 << 20):
        assert int(torch.count_nonzero(part)) == 0


def test_output_of_another_type_is_refused(ttt):
    c = on_gpu(case(1, 1, 1, 5, 16, BF16, w0="none"))
    z = torch.empty_like(c["q"], dtype=F32)
    with pytest.raises(ValueError, match="out_dtype"):
        ttt.linear_attn_fwd(**c, z=z, out_dtype=BF16)
    with pytest.raises(ValueError, match="out_dtype"):
        ttt.linear_attn_decode(c["q"], c["k"], c["v"], c["log_decay"], torch.zeros(1, 1, 16, 16, device=DEV), z=z,
                               out_dtype=BF16)
    assert ttt.linear_attn_fwd(**c, z=z)[0] is z and ttt.linear_attn_fwd(**c, z=z, out_dtype=F32)[0] is z
