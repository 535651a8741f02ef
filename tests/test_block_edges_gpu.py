"""The short convolution, the selective scan and the block norm where a value, a length or a walk is at an end of its range."""
import pytest

import block_testutil as bt
import test_block_gpu as small

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as m
    m.lib()
    return m


def random(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std + mean).to(dtype).cuda()


# the mean of a row with an infinity is infinite and its variance inf - inf: no element of such a row is a number.  Mean squares
# are: finite / inf = 0, and the infinity itself inf / inf.  768 and 766 channels: in pieces and element by element
@pytest.mark.parametrize("D", [768, 766])
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
def test_norm_of_a_row_with_an_infinity(ttt, D, value):
    x, ga, be = random((2, 5, D), F32, 1), random((D,), F32, 2, 0.1, 1.0), random((D,), F32, 3)
    bad = x.clone()
    bad[1, 3, 17] = value
    for kind in ("layer", "rms"):
        for where in (dict(gamma_post=ga, beta_post=be), dict(gamma_pre=ga, beta_pre=be)):
            at = 0 if "gamma_post" in where else 1
            want, got = (ttt.block_norm_fwd(t, kind=kind, **where)[at] for t in (x, bad))
            row = got[1, 3].clone()
            got[1, 3] = want[1, 3]
            assert torch.equal(got, want)
            if kind == "layer" or value != value:
                assert torch.isnan(row).all(), (kind, where.keys())
            else:
                assert torch.isnan(row[17]) and torch.equal(torch.cat([row[:17], row[18:]]), torch.cat([be[:17], be[18:]]))
    # the gradients of that row are not numbers either, and those of the others are what they were
    ds = random((2, 5, D), F32, 4)
    want, got = (ttt.block_norm_bwd(t, ds, None, gamma_post=ga, beta_post=be, kind="layer")[0] for t in (x, bad))
    assert torch.isnan(got[1, 3]).all()
    got[1, 3] = want[1, 3]
    assert torch.equal(got, want)


# the gradients read a row ahead, but no row behind its sequence's last token and no tensor that is not there: rows of nothing
# between rows of tokens, several to a workgroup, with NaN in all that has no business in the result
@pytest.mark.parametrize("D,dtype,res_dtype", [(72, BF, F32), (768, BF, BF), (2048, F32, BF), (2056, BF, F32), (4104, BF, F32)])
@pytest.mark.parametrize("given", ["s", "y", "all"])
def test_norm_backward_between_rows_of_nothing(ttt, D, dtype, res_dtype, given):
    B, T = 37, 61
    lens = torch.tensor([(0, 61, 1, 30, 60)[b % 5] for b in range(B)], dtype=torch.int32, device="cuda")
    live = (torch.arange(T, device="cuda") < lens[:, None])[..., None]
    rows = lambda seed, to: random((B, T, D), to, seed).where(live, float("nan"))  # noqa: E731
    p = lambda seed: random((D,), F32, seed, 0.1, 1.0)  # noqa: E731
    x, ds, dy = rows(1, dtype), None if given == "y" else rows(2, res_dtype), None if given == "s" else rows(3, dtype)
    more = {} if given == "s" else dict(gamma_pre=p(4))
    if given == "all":
        more.update(res=rows(5, res_dtype), z=rows(6, dtype), alpha=p(7), gamma_post=p(8), beta_post=p(9), kind="layer")
    ws = torch.full((ttt.block_norm_workspace_bytes(x) // 4,), float("nan"), device="cuda")
    got = ttt.block_norm_bwd(x, ds, dy, lens=lens, workspace=ws, **more)
    for g in got:
        assert g is None or torch.isfinite(g).all()
    cut = lambda t, b: None if t is None else t[b:b + 1, :int(lens[b])] if t.dim() == 3 else t  # noqa: E731
    for b in (1, 2, 3, 18, 33, 36):
        part = {k: cut(v, b) if torch.is_tensor(v) else v for k, v in more.items()}
        alone = ttt.block_norm_bwd(cut(x, b), cut(ds, b), cut(dy, b), **part)
        for g, a in zip(got[:3], alone[:3]):
            if g is not None:
                assert torch.equal(cut(g, b), a) and not g[b, int(lens[b]):].any()


# A = -inf: exp(step A) is 0 for a step of 1e-36 and more and 1 for a step of 0, in one segment, in several, token by token and
# backward; with softplus steps below e^-87 count as 0
@pytest.mark.parametrize("T", [5, 700])
def test_a_decay_that_keeps_nothing(ttt, T):
    steps = torch.tensor([0.0, 1e-36, 1e-20, 0.1, 0.0, 2e-36], device="cuda")
    keeps = (steps == 0).float()
    B, D, N = 1, len(steps), 3
    dt = torch.zeros(B, T, D, device="cuda")
    dt[:, T // 2] = steps  # all other steps are 0
    u, bc = random((B, T, D), F32, 1), torch.zeros(B, 1, T, N, device="cuda")
    A, h0, dh = torch.full((D, N), -INF, device="cuda"), random((B, D, N), F32, 2), random((B, D, N), F32, 3)
    y, h = ttt.selective_scan_fwd(u, dt, A, bc, bc, h0=h0)
    assert torch.equal(h, h0 * keeps[:, None]) and not y.any()
    state = h0.clone()
    ttt.selective_scan_decode(u, dt, A, bc, bc, state)
    assert torch.equal(state, h)
    got = ttt.selective_scan_bwd(u, dt, A, bc, bc, torch.zeros_like(u), h0=h0, dh_final=dh)
    assert torch.equal(got[8], dh * keeps[:, None]) and torch.isfinite(got[2]).all()
    raw = torch.tensor([-200.0, -80.0, -20.0, 0.0, -90.0, 50.0], device="cuda")
    wide = torch.full((B, T, D), -200.0, device="cuda")
    wide[:, T // 2] = raw
    _, h = ttt.selective_scan_fwd(u, wide, A, bc, bc, h0=h0, softplus=True)
    assert torch.equal(h, h0 * (raw < -87).float()[:, None])


# more rows than workgroups: the forward's second pass over its loop, teams whose places for sums come round again, rows of
# nothing in between
@pytest.mark.parametrize("case", [
    (6, 1501, 136, BF, F32, "layer", True, False, True, True, True, True, True, True, "late", "dense"),
    (6, 1501, 520, BF, BF, "rms", True, True, True, False, True, True, False, True, "early", "slice"),
    (6, 1501, 500, F32, F32, "layer", True, False, True, True, True, True, True, True, "early", "odd"),
    (6, 801, 1032, F32, BF, "layer", True, False, True, True, True, True, True, True, "late", "dense"),
    (6, 601, 2056, BF, F32, "layer", False, False, True, True, True, True, True, True, "early", "dense"),
    (1, 1100, 4104, BF, F32, "layer", True, True, True, True, True, True, True, True, None, "dense"),
    (1, 1100, 4101, BF, BF, "rms", True, False, True, False, True, True, False, True, None, "odd"),
])
def test_norm_forward_more_rows_than_workgroups(ttt, case):
    small.test_norm_forward(ttt, case)


@pytest.mark.parametrize("case", [
    (1, 700, 4104, BF, BF, "layer", True, True, True, True, True, True, True, True, None, "dense"),
    (1, 700, 4101, F32, F32, "rms", True, False, True, False, True, True, False, True, None, "odd"),
    (6, 301, 2056, F32, BF, "layer", True, False, True, True, True, True, True, True, "late", "slice"),
])
def test_norm_backward_more_rows_than_workgroups(ttt, case):
    small.test_norm_backward(ttt, case)


def segment(B, T, D, dtype):
    """Tokens that a thread of the convolution's gradients walks."""
    return min(max(T * B * -(-D // (8 if dtype == BF else 4)) >> 17, 16), 128)


# longer walks than 16 tokens, as training has them, up to the longest of 128: dx and the state's gradient of every sequence
# against that sequence alone, where walks are 16 tokens long; the sums over tokens against 64 bits on a few channels
@pytest.mark.parametrize("B,T,D,K,dtype,out,silu,walk", [
    (8, 2048, 1536, 4, BF, BF, True, 24), (6, 1501, 1540, 3, F32, F32, True, 26), (10, 5003, 2056, 4, BF, F32, False, 98),
    (40, 3301, 1032, 2, BF, BF, True, 128)])
def test_conv_gradients_of_long_walks(ttt, B, T, D, K, dtype, out, silu, walk):
    assert segment(B, T, D, dtype) == walk and segment(1, T, D, dtype) == 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s, to=F32, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(to)  # noqa: E731
    lens = torch.tensor([(T, T // 2, walk * 8 + 1, 0, T - 1, 1)[b % 6] for b in range(B)], dtype=torch.int32, device="cuda")
    c = dict(x=mk(B, T, D, to=dtype), w=mk(D, K, std=0.5), dy=mk(B, T, D, to=out), bias=mk(D), state=mk(B, K - 1, D, to=dtype),
             dstate_final=mk(B, K - 1, D, to=out))
    dx, dw, db, dst = ttt.short_conv_bwd(**c, silu=silu, lens=lens)
    for b in sorted({0, 1, 2, 3, 4, 5, B - 1}):
        one = {k: v[b:b + 1] if k in ("x", "dy", "state", "dstate_final") else v for k, v in c.items()}
        alone = ttt.short_conv_bwd(**one, silu=silu, lens=lens[b:b + 1])
        assert torch.equal(dx[b:b + 1], alone[0]) and torch.equal(dst[b:b + 1], alone[3])
    cut = slice(D - 9, D)
    part = {k: (v[cut] if k in ("w", "bias") else v[..., cut]).cpu() for k, v in c.items()}
    ref, size = bt.conv_grads(**part, act=silu, lens=lens.cpu())
    deep = bt.conv(part["x"], part["w"], part["bias"], part["state"], lens=lens.cpu(), magnitudes=True)[2].max().item()
    # as for short walks; a term goes through the rest of its walk and its workgroup's 8 walks, the last sum is in 64 bits
    roundings = 2 * K + 8 + (20 + deep if silu else 0)
    for n, a, r, s in zip(("dx", "dw", "dbias", "dstate"), (dx[..., cut], dw[cut], db[cut], dst[..., cut]), ref, size):
        bt.check(n, a, r, s, roundings + (walk + 8 if n in ("dw", "dbias") else 0))


# The bounds of the tests over types and layouts allow every rounding its worst; this one asks for what they come to: no further
# from 64 bits than 8 times what plain fp32 operations are, which add the same terms in another order, and 2^-22 of the largest
# value for results that those happen to hit
@pytest.mark.parametrize("B,T,D,N,G,gate", [(2, 60, 24, 16, 1, True), (1, 300, 70, 16, 2, False), (3, 700, 12, 4, 1, True), (2, 333, 40, 32, 1, True)])
def test_scan_is_as_good_as_plain_fp32(ttt, B, T, D, N, G, gate):
    _, _, c, g = small.scan_case(B, T, D, N, G, F32, F32, True, gate, True, True, True, None, "dense", 21)
    dy, dh = random((B, T, D), F32, 22), random((B, D, N), F32, 23)
    names = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")

    def plain(dtype):
        p = {n: None if c[n] is None else c[n].to(dtype).requires_grad_() for n in names}
        step = torch.nn.functional.softplus(p["dt"] + p["dt_bias"])
        Bx, Cx = (p[n].repeat_interleave(D // G, 1) for n in ("Bm", "Cm"))
        h, ys = p["h0"], []
        for t in range(T):
            h = torch.exp(step[:, t, :, None] * p["A"]) * h + (step[:, t] * p["u"][:, t])[..., None] * Bx[:, :, t]
            ys.append((h * Cx[:, :, t]).sum(-1))
        y = torch.stack(ys, 1) + p["D"] * p["u"]
        if gate:
            y = y * bt.silu(p["z"])
        leaves = [v for v in p.values() if v is not None]
        return [y.detach(), h.detach(), *torch.autograd.grad([y, h], leaves, [dy.cpu().to(dtype), dh.cpu().to(dtype)])]

    exact, own = plain(torch.float64), plain(F32)
    grads = ttt.selective_scan_bwd(**g, dy=dy, dh_final=dh, softplus=True)
    order = [0, 1, 2, 3, 4, 5, 6, 7, 8] if gate else [0, 1, 2, 3, 4, 5, 7, 8]
    got = [*ttt.selective_scan_fwd(**g, softplus=True), *(grads[i] for i in order)]
    for n, a, r, f in zip(["y", "h", *(n for n in names if c[n] is not None)], got, exact, own):
        off, ref = (a.cpu().double() - r).abs().max().item(), (f.double() - r).abs().max().item()
        print(f"{n}: off {off:.2e}, plain fp32 {ref:.2e}, largest {r.abs().max().item():.1e}", flush=True)
        assert off <= 8 * ref + 2.0 ** -22 * r.abs().max().item(), n


# small and large rows without eps: as far as mean squares of 1e-37 and 1e38 the result does not depend on their size
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 1.0, 2.0 ** 60])
def test_norm_of_small_and_large_rows(ttt, kind, scale):
    x, ga, dy = random((2, 3, 200), F32, 1), random((200,), F32, 2, 0.1, 1.0), random((2, 3, 200), F32, 3)
    _, y = ttt.block_norm_fwd(x * scale, gamma_pre=ga, kind=kind, eps=0.0)
    ref = bt.norm_rounded(x.cpu(), None, None, None, None, None, ga.cpu(), None, kind, 0.0, False)[1]
    bt.check_rounded("y", y, ref)
    dx = ttt.block_norm_bwd(x * scale, None, dy, gamma_pre=ga, kind=kind, eps=0.0)[0]
    ref = bt.norm_rounded(x.cpu(), None, None, None, None, None, ga.cpu(), None, kind, 0.0, False, dy=dy.cpu())[0]
    bt.check_rounded("dx", dx * scale, ref)
