"""The bounds of test_attn_bits_gpu.py, on the CPU: products of bf16 parts in 64 bits, with two parts beyond them
and with three within."""
import pytest

torch = pytest.importorskip("torch")
from test_attn_bits_gpu import A, additions, bound, coherent  # noqa: E402


def parts(x, n):
    got, rest = [], x.double()
    for _ in range(n):
        got.append(rest.float().bfloat16().double())
        rest = rest - got[-1]
    return got


def product(a, b, n):
    """a @ b over the part pairs (p, q) with p + q < n; every sum in 64 bits"""
    pa, pb = parts(a, n), parts(b, n)
    return sum(pa[p] @ pb[q] for p in range(n) for q in range(n) if p + q < n)


def test_parts_of_the_value():
    p = [x.item() for x in parts(torch.tensor(A, dtype=torch.float64), 3)]
    assert p == [1.0, 2.0 ** -8 - 2.0 ** -15, 2.0 ** -17 - 2.0 ** -23] and torch.tensor(A).double().item() == A


@pytest.mark.parametrize("d,T", [(16, 32), (64, 32), (128, 32)])
def test_two_parts_are_beyond_the_bound(d, T):
    """One chunk's outputs, the state's update and the decay's gradient"""
    gen = torch.Generator().manual_seed(d)
    q, k, v, dz = (coherent(gen, T, d) for _ in range(4))
    n = additions(d, T)
    i = torch.arange(T)
    dist = (i[:, None] - i).clamp(min=0).double()
    low = torch.tril(torch.ones(T, T, dtype=torch.float64))
    off = {}
    for parts_ in (2, 3, 8):  # 8: all of it
        s = product(q, k.T, parts_) * low
        z = product(s.float() if parts_ < 8 else s, v, parts_)
        dg = (dist * s * product(dz, v.T, parts_)).sum()
        off[parts_] = dict(z=z, w=product(v.T, k, parts_), dg=dg)
    for name in ("z", "w", "dg"):
        two, three = ((off[m][name] / off[8][name] - 1).abs() for m in (2, 3))
        assert two.min() > bound(n[name]) > 20 * three.max(), (name, two.min(), three.max(), bound(n[name]))
