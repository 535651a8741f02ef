"""Rotary positions on the GPU against the rotation in 64 bits.  An output is
scale (a cos - b sin): its two products, the sum, the scaled cosine and sine (each
rounded, scaled and off by the angle's rounding of at most pi 2^-24) put at most
12 x 2^-24 of scale (|a| + |b|) on it, and the store half a step of its type."""
import itertools

import pytest

from attn_testutil import check, turn

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


def tol(x, ref, freqs, layout, scale, dtype):
    n = freqs.shape[0]
    size = x.double().abs()
    pair = torch.zeros_like(size)
    first, second = ((slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    pair[..., first] = pair[..., second] = size[..., first] + size[..., second]
    return torch.finfo(dtype).eps / 2 * ref.abs() + 12 * 2.0 ** -24 * scale * pair + 1e-30


def make(B, H, Hkv, T, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H, T, d, generator=gen).to(dtype), torch.randn(B, Hkv, T, d, generator=gen).to(dtype))


# d, rot: whole head, half of it, an odd number of pairs, one pair, none; rows that are no multiple of 16 bytes
SIZES = [(64, 64), (64, 32), (64, 62), (128, 128), (16, 16), (32, 16), (64, 2), (64, 0), (30, 12), (7, 6), (256, 64),
         (24, 22), (40, 34), (12, 10), (20, 8), (64, 48), (36, 24)]


@pytest.mark.parametrize("layout,dtype", list(itertools.product(["half", "interleaved"], [BF16, F32])))
@pytest.mark.parametrize("d,rot", SIZES)
def test_sizes(ttt, d, rot, layout, dtype):
    freqs, _ = ttt.rotary_freqs(rot)
    scale = 1.25
    for B, H, Hkv, T in ((2, 3, 1, 9), (1, 5, 0, 1), (3, 1, 2, 130)):
        q, k = make(B, H, Hkv, T, d, dtype, seed=T)
        pos = torch.randint(0, 1 << 20, (B, T), generator=torch.Generator().manual_seed(T))
        for back in (False, True):
            call = ttt.rotary_bwd if back else ttt.rotary
            got = call(q.to(DEV), k.to(DEV) if Hkv else None, pos.to(DEV), freqs.to(DEV), layout, scale)
            assert (got[1] is None) == (Hkv == 0)
            for x, y in zip((q, k), got):
                if y is not None:
                    ref = turn(x, pos, freqs, layout, scale, inverse=back)
                    check(f"d {d} rot {rot}", y, ref, tol(x, ref, freqs, layout, scale, dtype))
                    assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("start", [0, -5, 1_000_003, (1 << 40) + 12345])
def test_far_positions(ttt, start):
    q, k = make(2, 4, 4, 33, 64, F32)
    freqs, s = ttt.rotary_freqs(64, scaling="yarn", factor=16.0)
    each = start + torch.arange(33).expand(2, 33)
    got = ttt.rotary(q.to(DEV), k.to(DEV), start, freqs.to(DEV), scale=s)
    # the 64-bit products of position and frequency: 2^-53 of an angle each side, 3e-4 radians at 2^40
    far = 4 * 2.0 ** -53 * abs(start)
    for x, y in zip((q, k), got):
        ref = turn(x, each, freqs, "half", s)
        check("far", y, ref, tol(x, ref, freqs, "half", s, F32) + far * s * 2 * x.double().abs().amax())
    # the same positions said in other ways
    for pos in (torch.full((2,), start), each, each.contiguous()):
        again = ttt.rotary(q.to(DEV), k.to(DEV), pos.to(DEV), freqs.to(DEV), scale=s)
        assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_layouts_and_in_place(ttt, layout):
    B, H, T, d = 2, 4, 37, 64
    q, k = (x.to(DEV) for x in make(B, H, H, T, d, BF16))
    freqs = ttt.rotary_freqs(48, device=DEV)[0]
    ref = ttt.rotary(q, k, 11, freqs, layout)
    qc, kc = q.clone(), k.clone()
    got = ttt.rotary(qc, kc, 11, freqs, layout, out=(qc, kc))
    assert got[0] is qc and torch.equal(qc, ref[0]) and torch.equal(kc, ref[1])
    qc = q.clone()  # one of the two in place
    got = ttt.rotary(qc, k, 11, freqs, layout, out=(qc, torch.empty_like(k)))
    assert torch.equal(qc, ref[0]) and torch.equal(got[1], ref[1])
    packed = torch.stack([x.transpose(1, 2) for x in (q, k, q)], 2)  # [B, T, 3, H, d]
    pq, pk = (packed[:, :, i].transpose(1, 2) for i in (0, 1))
    got = ttt.rotary(pq, pk, 11, freqs, layout)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    ttt.rotary(pq, pk, 11, freqs, layout, out=(pq, pk))
    assert torch.equal(pq, ref[0]) and torch.equal(pk, ref[1]) and torch.equal(packed[:, :, 2].transpose(1, 2), q)
    odd = torch.cat([q[..., :1], q], -1)[..., 1:]  # rows two bytes off
    assert torch.equal(ttt.rotary(odd, None, 11, freqs, layout)[0], ref[0])
    with pytest.raises(ttt.TTTError) as e:
        ttt.rotary(q, q, 11, freqs, layout, out=(q, q))
    assert e.value.status == 5


@pytest.mark.parametrize("d,rot", [(64, 62), (24, 22), (16, 10)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_halves_in_place(ttt, d, rot, dtype):
    """both, and only one, of q and k in place, with rows that end inside a workgroup's last piece"""
    freqs = ttt.rotary_freqs(rot, device=DEV)[0]
    q, k = (x.to(DEV) for x in make(3, 5, 2, 211, d, dtype))
    ref = ttt.rotary(q, k, 7, freqs)
    qc, kc = q.clone(), k.clone()
    ttt.rotary(qc, kc, 7, freqs, out=(qc, kc))
    assert torch.equal(qc, ref[0]) and torch.equal(kc, ref[1])
    qc = q.clone()
    got = ttt.rotary(qc, k, 7, freqs, out=(qc, torch.empty_like(k)))
    assert torch.equal(qc, ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rest_of_the_head_is_passed_on(ttt, layout):
    """infinities and NaN beside and behind the turned elements stay where they are"""
    for d, rot in ((64, 16), (64, 30), (64, 32), (9, 4)):
        q = torch.randn(1, 2, 5, d, device=DEV)
        q[..., rot:] = torch.tensor([float("inf"), float("nan"), -float("inf")], device=DEV).repeat(d)[:d - rot]
        y = ttt.rotary(q, None, 3, ttt.rotary_freqs(rot, device=DEV)[0], layout)[0]
        assert torch.isfinite(y[..., :rot]).all() and torch.equal(y[..., rot:].nan_to_num(7.0), q[..., rot:].nan_to_num(7.0))


def test_many_heads_and_few(ttt):
    """the heads of one token dealt out over workgroups"""
    freqs = ttt.rotary_freqs(64, device=DEV)[0]
    for B, H, Hkv in ((1, 37, 5), (1, 1, 1), (700, 2, 1)):
        q, k = make(B, H, Hkv, 1, 64, BF16, seed=B)
        pos = torch.arange(B)[:, None] * 7
        got = ttt.rotary(q.to(DEV), k.to(DEV), pos.to(DEV), freqs)
        for x, y in zip((q, k), got):
            ref = turn(x, pos, freqs.cpu())
            check("heads", y, ref, tol(x, ref, freqs, "half", 1.0, BF16))


def test_nothing_to_do(ttt):
    freqs = ttt.rotary_freqs(64, device=DEV)[0]
    q, k = make(0, 2, 2, 4, 64, BF16)
    assert ttt.rotary(q.to(DEV), k.to(DEV), 0, freqs)[0].shape == (0, 2, 4, 64)
    q, k = make(2, 2, 2, 0, 64, BF16)
    assert ttt.rotary(q.to(DEV), k.to(DEV), 0, freqs)[1].shape == (2, 2, 0, 64)


def test_stream_and_graph(ttt):
    q, k = (x.to(DEV) for x in make(2, 4, 2, 65, 64, BF16))
    freqs = ttt.rotary_freqs(64, device=DEV)[0]
    ref = ttt.rotary(q, k, 3, freqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q2 = q.clone()
    got = ttt.rotary(q2, k, 3, freqs, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    pos = torch.zeros(2, dtype=torch.int64, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ttt.rotary(q, k, pos, freqs)
    for p in (3, 50, 0):
        pos.fill_(p)
        want = ttt.rotary(q, k, p, freqs)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_gradient_is_the_adjoint(ttt):
    """<dy, rotary(x)> = <rotary_bwd(dy), x>: the rotation is linear.  Both sides are sums of terms of size
    scale |dy| |pair of x|, each off by 12 roundings."""
    gen = torch.Generator().manual_seed(5)
    x, dy = torch.randn(2, 3, 40, 32, generator=gen), torch.randn(2, 3, 40, 32, generator=gen)
    freqs = ttt.rotary_freqs(24, device=DEV)[0]
    for layout in ("half", "interleaved"):
        y = ttt.rotary(x.to(DEV), None, 9, freqs, layout, 1.5)[0].double().cpu()
        dx = ttt.rotary_bwd(dy.to(DEV), None, 9, freqs, layout, 1.5)[0].double().cpu()
        bound = 2 * 13 * 2.0 ** -24 * 1.5 * 2 * (dy.abs().amax(-1) * x.abs().amax(-1) * 32).sum().item()
        assert abs((dy * y).sum() - (dx * x).sum()) <= bound


def test_offsets_past_32_bits(ttt):
    wide = torch.zeros(20000, 1 << 17, device=DEV, dtype=BF16)
    q = wide[:, :64][None, None]
    q.copy_(torch.randn(1, 1, 20000, 64, device=DEV).to(BF16))
    freqs = ttt.rotary_freqs(64, device=DEV)[0]
    ref = ttt.rotary(q.contiguous(), None, 0, freqs)[0]
    out = wide[:, 64:128][None, None]
    ttt.rotary(q, None, 0, freqs, out=(out, None))
    assert torch.equal(out, ref)


@pytest.mark.parametrize("d,rot", [(48, 48), (80, 80), (96, 96), (96, 30), (1040, 64), (2056, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_q_alone_and_k_alone(ttt, d, rot, dtype):
    """rows that fill no workgroup evenly, without a k and without a q, out of place and in place"""
    freqs = ttt.rotary_freqs(rot)[0]
    f = freqs.to(DEV)
    for B, H, T in ((3, 5, 211), (1, 1, 1), (2, 4, 64)):
        q, _ = make(B, H, 1, T, d, dtype, seed=T)
        ref = turn(q, 9 + torch.arange(T).expand(B, T), freqs)
        got = ttt.rotary(q.to(DEV), None, 9, f)[0]
        check("q", got, ref, tol(q, ref, freqs, "half", 1.0, dtype))
        none = torch.empty(B, 0, T, d, dtype=dtype, device=DEV)
        assert torch.equal(ttt.rotary(none, q.to(DEV), 9, f)[1], got)
        here = q.to(DEV)
        ttt.rotary(here, None, 9, f, out=(here, None))
        check("in place", here, ref, tol(q, ref, freqs, "half", 1.0, dtype))


@pytest.mark.parametrize("start", [1, 77, 100_003])
def test_sine_and_cosine_keep_their_relative_accuracy(ttt, start):
    """The pair (1, 0) becomes (cos, sin).  Near whole and half turns, where the sine is small, and near quarter turns,
    where the cosine is: each within 6 x 2^-24 of itself (two steps of the fp32 functions, one of the correction), and the
    64-bit angle's own rounding, 2^-52 of it on either side."""
    gen = torch.Generator().manual_seed(start)
    quarter = torch.randint(-4, 5, (4096,), generator=gen).double()
    off = torch.exp(-14 * torch.rand(4096, generator=gen, dtype=torch.float64)) * torch.where(
        torch.rand(4096, generator=gen) < 0.5, -1.0, 1.0)
    freqs = (quarter * torch.pi / 2 + off) / start
    angle = start * freqs
    q = torch.zeros(1, 1, 1, 8192)
    q[..., :4096] = 1
    y = ttt.rotary(q.to(DEV), None, start, freqs.to(DEV))[0].cpu().double().view(2, 4096)
    for name, got, ref in (("cos", y[0], torch.cos(angle)), ("sin", y[1], torch.sin(angle))):
        check(name, got, ref, 6 * 2.0 ** -24 * ref.abs() + 4 * 2.0 ** -52 * (1 + angle.abs()))
