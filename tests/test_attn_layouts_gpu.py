"""Linear attention and rotary positions in places that interleave: slices within the heads of one
projection, as inputs, as outputs and in place."""
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


def _packed(B, T, H, d, dtype, order, seed):
    """Three [B, H, T, d] views of one buffer laid out in the given order of b, t, h and the three."""
    gen = torch.Generator().manual_seed(seed)
    sizes = dict(b=B, t=T, h=H, x=3)
    buf = torch.randn(*(sizes[n] for n in order), d, generator=gen).to(dtype).to(DEV)
    views = buf.permute(*(order.index(n) for n in "xbht"), 4)
    return buf, [views[i] for i in range(3)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("order", ["bthx", "bhtx", "btxh", "bxht"])
@pytest.mark.parametrize("T", [50, 300])
def test_gradients_in_one_buffer(ttt, order, dtype, T):
    B, H, d = 2, 3, 32
    _, (q, k, v) = _packed(B, T, H, d, dtype, order, seed=T)
    g = torch.tensor([-0.1, 0.0, -2.0], device=DEV)
    dz = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    ref = ttt.linear_attn_bwd(*(x.contiguous() for x in (q, k, v)), g, dz)
    _, places = _packed(B, T, H, d, dtype, order, seed=0)
    got = ttt.linear_attn_bwd(q, k, v, g, dz, out=(*places, torch.empty_like(ref[3]), torch.empty_like(ref[4])))
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
    # the forward's Z in the place that Q's gradient had, beside inputs of the same buffer
    buf, (q, k, z) = _packed(B, T, H, d, dtype, order, seed=T + 1)
    keep = q.clone(), k.clone()
    want = ttt.linear_attn_fwd(q.contiguous(), k.contiguous(), v, g, out_dtype=dtype)[0]
    assert torch.equal(ttt.linear_attn_fwd(q, k, v, g, z=z)[0], want)
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("order", ["bthx", "bhtx"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 30), (24, 22), (96, 96)])
def test_rotary_in_place_within_heads(ttt, order, layout, d, rot):
    buf, (q, k, v) = _packed(2, 67, 4, d, BF16, order, seed=d)
    keep = v.clone()
    f = ttt.rotary_freqs(rot, device=DEV)[0]
    want = ttt.rotary(q.contiguous(), k.contiguous(), 5, f, layout)
    ttt.rotary(q, k, 5, f, layout, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)
