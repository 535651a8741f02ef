"""The short convolution, the selective scan and the block norm at the sizes where another form of their kernels runs: rows in
16-byte pieces whose tiles end inside, many sequences, long walks, more rows than workgroups."""
import pytest

import block_testutil as bt
import test_block_gpu as small

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


SCAN = [  # as in the small cases; channels in eights, states in fours, ends inside tiles of 16, 32 and 64
    (6, 61, 72, 16, 1, BF, BF, True, True, True, True, True, "late", "dense"),
    (6, 97, 136, 12, 1, BF, F32, True, True, True, True, True, "early", "slice"),
    (2, 77, 80, 20, 1, F32, F32, True, True, True, True, True, None, "slice"),
    (1, 93, 144, 32, 2, BF, BF, False, True, True, True, True, None, "dense"),
    (3, 50, 16, 4, 2, F32, BF, True, True, False, True, True, "late", "dense"),
    (6, 701, 72, 16, 1, BF, BF, True, True, True, True, True, "late", "dense"),
    (6, 531, 48, 8, 2, F32, F32, True, True, True, True, True, "early", "dense"),
]


@pytest.mark.parametrize("case", SCAN)
def test_scan_forward(ttt, case):
    small.test_scan_forward(ttt, case)


@pytest.mark.parametrize("case", SCAN)
def test_scan_backward(ttt, case):
    small.test_scan_backward(ttt, case)


@pytest.mark.parametrize("case", [c for c in SCAN if c[1] <= 100])
def test_scan_tokens(ttt, case):
    small.test_scan_tokens(ttt, case)


# lengths where the gradients go from one segment to two, three, ..., and where the last has one token
@pytest.mark.parametrize("T", [63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 161, 192, 193, 257])
def test_scan_segments(ttt, T):
    case = (2, T, 40, 16, 1, F32, F32, True, True, True, True, True, None, "dense")
    small.test_scan_forward(ttt, case)
    small.test_scan_backward(ttt, case)
    ends = (6, T, 8, 4, 1, F32, F32, True, True, True, True, True, "late", "dense")
    small.test_scan_forward(ttt, ends)
    small.test_scan_backward(ttt, ends)


@pytest.mark.parametrize("case", [
    (6, 1501, 136, BF, F32, "layer", True, False, True, True, True, True, True, True, "late", "dense"),
    (6, 1501, 520, BF, BF, "rms", True, True, True, False, True, True, False, True, "early", "slice"),
    (1, 300, 4104, BF, F32, "rms", True, False, True, False, False, True, False, True, None, "dense"),
])
def test_norm_backward_more_rows_than_workgroups(ttt, case):
    small.test_norm_backward(ttt, case)


def random(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def ragged(B, T):
    return torch.tensor([(T, 0, T - 1, T // 2, 1)[i % 5] for i in range(B)], dtype=torch.int32, device="cuda")


# many tiles of 8 tokens, ends inside them; a few sequences alone have the same bits
@pytest.mark.parametrize("B,T,D,K,dtype,with_lens", [
    (37, 7300, 256, 4, BF, True), (300, 28000, 4, 3, F32, False), (260, 33000, 1, 2, BF, True)])
def test_conv_long_walk(ttt, B, T, D, K, dtype, with_lens):
    x, w, bias = random((B, T, D), dtype, 1), random((D, K), F32, 2, 0.5), random((D,), F32, 3)
    state, lens = random((B, K - 1, D), dtype, 4), ragged(B, T) if with_lens else None
    y, last = ttt.short_conv_fwd(x, w, bias=bias, state=state, silu=True, lens=lens)
    for at in (0, B // 2, B - 5):
        cut = slice(at, at + 5)
        part = None if lens is None else lens[cut].contiguous()
        y1, last1 = ttt.short_conv_fwd(x[cut], w, bias=bias, state=state[cut].contiguous(), silu=True, lens=part)
        assert torch.equal(y[cut], y1) and torch.equal(last[cut], last1)
    c = dict(x=x[:2].cpu(), w=w.cpu(), bias=bias.cpu(), state=state[:2].cpu())
    part = None if lens is None else lens[:2].cpu()
    size = bt.conv(**c, lens=part, magnitudes=True)[0]
    bt.check("y", y[:2], bt.conv(**c, act=True, lens=part)[0], size * 1.1, K + 1 + 16 + size.max().item())


# many sequences; a few of them alone have the same bits
@pytest.mark.parametrize("B,T,N,dtype", [(37, 1, 16, BF), (33, 3, 12, F32), (35, 2, 5, BF)])
def test_scan_tokens_of_many(ttt, B, T, N, dtype):
    D = 4096
    u, z = random((B, T, D), dtype, 1), random((B, T, D), dtype, 2)
    dt, A = random((B, T, D), dtype, 3, 0.7, -2.0), -(random((D, N), F32, 4).abs() * 3 + 0.01)
    Bm, Cm = random((B, 1, T, N), dtype, 5), random((B, 1, T, N), dtype, 6)
    skip, bias, h0 = random((D,), F32, 7), random((D,), F32, 8, 0.3), random((B, D, N), F32, 9)
    lens = ragged(B, T)
    h = h0.clone()
    y = ttt.selective_scan_decode(u, dt, A, Bm, Cm, h, D=skip, z=z, dt_bias=bias, softplus=True, lens=lens)
    for at in (0, B - 3):
        cut = slice(at, at + 3)
        h1 = h0[cut].clone()
        y1 = ttt.selective_scan_decode(u[cut], dt[cut], A, Bm[cut], Cm[cut], h1, D=skip, z=z[cut], dt_bias=bias, softplus=True,
                                       lens=lens[cut].contiguous())
        assert torch.equal(y[cut], y1) and torch.equal(h[cut], h1)
    c = dict(u=u, dt=dt, A=A, Bm=Bm, Cm=Cm, D=skip, z=z, dt_bias=bias, h0=h0)
    c = {k: v.cpu() for k, v in c.items()}
    ref, size = (bt.scan(**c, softplus=True, lens=lens.cpu(), magnitudes=m) for m in (False, True))
    k = bt.scan_roundings(T, N, D)[0]
    bt.check("y", y, ref[0], size[0], k)
    bt.check("h", h, ref[1], size[1], k)


# 2^18 pieces of channels are where a thread takes four sequences; the last takes fewer
@pytest.mark.parametrize("B,T,D,K,dtype", [(259, 1, 8192, 4, BF), (258, 2, 4096, 3, F32), (2051, 1, 1020, 2, BF)])
def test_conv_tokens_of_many(ttt, B, T, D, K, dtype):
    assert B * -(-D // (8 if dtype == BF else 4)) >= 1 << 18 and B % 4
    x, w, bias = random((B, T, D), dtype, 1), random((D, K), F32, 2, 0.5), random((D,), F32, 3)
    state0, lens = random((B, K - 1, D), dtype, 4), ragged(B, T)
    state = state0.clone()
    y = ttt.short_conv_decode(x, w, state, bias=bias, silu=True, lens=lens)
    c = dict(x=x.cpu(), w=w.cpu(), bias=bias.cpu(), state=state0.cpu())
    size = bt.conv(**c, lens=lens.cpu(), magnitudes=True)[0]
    ref, last, _ = bt.conv(**c, act=True, lens=lens.cpu())
    bt.check("y", y, ref, size * 1.1, K + 1 + 16 + size.max().item())
    assert torch.equal(state.cpu().double(), last)
