"""The short convolution, the selective scan and the block norm where a value, a length or a walk is at an end of its range."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32 = torch.float32
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
