"""Where a NaN or an infinity in the inputs of linear attention may come out, and that all else
keeps its bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
B, H, HKV, D = 2, 4, 2, 32


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as m
    m.lib()
    return m


def _case(T, dtype, lens):
    gen = torch.Generator().manual_seed(T)
    r = lambda h: torch.randn(B, h, T, D, generator=gen).to(dtype).to(DEV)  # noqa: E731
    c = dict(q=r(H), k=r(HKV), v=r(HKV), dz=r(H))
    more = dict(log_decay=torch.tensor([-0.01, 0.0, -1.0, float("-inf")], device=DEV),
                w0=torch.randn(B, H, D, D, generator=gen).to(DEV),
                lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))
    return c, more


def _run(ttt, c, more, dw):
    z, w = ttt.linear_attn_fwd(c["q"], c["k"], c["v"], **more, out_dtype=c["q"].dtype)
    dq, dk, dv, dg, dw0 = ttt.linear_attn_bwd(c["q"], c["k"], c["v"], dz=c["dz"], dw_final=dw, **more)
    return dict(z=z, w=w, dq=dq, dk=dk, dv=dv, dg=dg, dw0=dw0)


def _reach(n, T, t, length):
    """Tokens of each output that input n's token t reaches: those that depend on it, and its block of 16."""
    i = torch.arange(T)
    at_or_after, up_to, own = i >= t, i <= t, i == t
    block = i // 16 == t // 16
    back = (length - 1 - i).div(16, rounding_mode="floor") == (length - 1 - t) // 16
    none = torch.zeros(T, dtype=torch.bool)
    return {"q": dict(z=own, dq=none, dk=up_to | back, dv=up_to),
            "k": dict(z=at_or_after, dq=at_or_after | block, dk=none, dv=own),
            "v": dict(z=at_or_after | block, dq=at_or_after, dk=own, dv=none),
            "dz": dict(z=none, dq=own, dk=up_to, dv=up_to | back)}[n]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,lens,tokens", [(70, None, (0, 20, 37, 69)), (450, None, (3, 200, 449)), (90, [77, 30], (5, 40, 76))])
def test_reach(ttt, dtype, T, lens, tokens):
    c, more = _case(T, dtype, lens)
    dw = torch.randn(B, H, D, D, generator=torch.Generator().manual_seed(2)).to(DEV)
    clean = _run(ttt, c, more, dw)
    length = T if lens is None else lens[0]
    for n in ("q", "k", "v", "dz"):
        for t in tokens:
            for bad in (float("nan"), float("inf")):
                x = c[n].clone()
                head = 1  # (of q and dz: key / value head 0; of k and v: query heads 2 and 3)
                x[0, head, t, 5] = bad
                got = _run(ttt, {**c, n: x}, more, dw)
                query = [head] if n in ("q", "dz") else [2, 3]
                shared = [head // 2] if n in ("q", "dz") else [head]
                reach = _reach(n, T, t, length)
                for name, y in got.items():
                    same = (y == clean[name]) & torch.isfinite(y)
                    heads = shared if name in ("dk", "dv") else query
                    if name in reach:
                        same[0, heads] |= (reach[name][:length].nonzero().flatten().to(DEV)[:, None] ==
                                           torch.arange(T, device=DEV)).any(0)[:, None]
                        if reach[name][t] and t < length:  # it does not get lost
                            assert not torch.isfinite(y[0, heads, t]).all(), (n, t, bad, name)
                    elif name == "dg" or (name == "w") == (n in ("k", "v")):  # (W_final: of K, V; dW0: of Q, dZ)
                        same[0, heads] = True
                    assert same.all(), (n, t, bad, name)


@pytest.mark.parametrize("n", ["q", "k", "v"])
def test_reach_in_decode(ttt, n):
    """Tokens before it keep their bits, and with q all others do."""
    T, t = 11, 6
    c, more = _case(T, BF16, None)

    def run(c):
        w = more["w0"].clone()
        return ttt.linear_attn_decode(c["q"], c["k"], c["v"], more["log_decay"], w), w

    clean, cw = run(c)
    x = c[n].clone()
    x[0, 1, t, 5] = float("nan")
    z, w = run({**c, n: x})
    heads = [1] if n == "q" else [2, 3]
    same = z == clean
    assert not torch.isfinite(z[0, heads, t]).all()
    same[0, heads, t:(t + 1 if n == "q" else T)] = True
    assert same.all()
    same = w == cw
    if n != "q":
        same[0, heads] = True
    assert same.all()


def test_padding_reaches_nothing(ttt):
    """Rows behind a sequence's end, from the first of them on, in every tensor at once"""
    T, lens = 90, [77, 30]
    c, more = _case(T, BF16, lens)
    clean = _run(ttt, c, more, None)
    dirty = {n: x.clone() for n, x in c.items()}
    for x in dirty.values():
        for b, m in enumerate(lens):
            x[b, :, m:] = float("nan")
    got = _run(ttt, dirty, more, None)
    assert all(torch.equal(got[n], clean[n]) for n in clean)


@pytest.mark.parametrize("T", [70, 450])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lowest_values_without_a_score(ttt, dtype, T):
    """Tokens whose k is zero and whose v holds the type's lowest and largest values, as a mask may leave them: nothing of
    them in Z and W_final.  The same of dK, dV and dW0 with zeros in dz or q and such values in the other.  (Not of dQ:
    there such a v is in the score, dz.v, which overflows.)"""
    c, more = _case(T, dtype, None)
    more["log_decay"] = torch.tensor([-0.01, 0.0, -1.0, -0.1], device=DEV)
    gone = torch.zeros(T, dtype=torch.bool)
    gone[[0, 3, 17, 18, 40, T - 1]] = True
    most = torch.finfo(dtype).max
    edge = torch.where(torch.arange(D) % 2 == 0, -most, most).to(dtype).to(DEV)

    def put(n, x):
        y = c[n].clone()
        y[:, :, gone] = x
        return y

    clean, held = ({**c, "k": put("k", 0), "v": put("v", x)} for x in (0, edge))
    a, b = (_run(ttt, x, more, None) for x in (clean, held))
    for n in ("z", "w"):
        assert torch.equal(a[n], b[n]), n
    for zero, full, names in (("dz", "q", ("dk", "dw0")), ("q", "dz", ("dv", "dw0"))):
        a, b = (_run(ttt, {**c, zero: put(zero, 0), full: put(full, x)}, more, None) for x in (0, edge))
        for n in names:
            assert torch.equal(a[n], b[n]), (zero, n)
