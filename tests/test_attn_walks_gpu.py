"""Linear attention over many chunks in one workgroup, and over offsets past 32 bits, against the
recurrence in 64 bits."""
import pytest

from attn_testutil import attn, attn_grads, check, tolerance

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
NAMES = ("z", "w", "dq", "dk", "dv", "dg", "dw0")


@pytest.fixture(scope="module")
def ttt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import test_sequence_layer_amd as m
    m.lib()
    return m


def against(ttt, got, c, dz, dw):
    """the outputs of one part of a batch, and its inputs on the CPU"""
    d, T = c["q"].shape[3], c["q"].shape[2]
    out = dz.dtype
    ab = {n: x.abs() if torch.is_tensor(x) and n not in ("log_decay", "lens") else x for n, x in c.items()}
    ref = (*attn(**c), *attn_grads(**c, dz=dz, dw_final=dw))
    size = (*attn(**ab), *attn_grads(**c, dz=dz, dw_final=dw, magnitudes=True))
    group = c["q"].shape[1] // c["k"].shape[1]
    for name, y, r, a in zip(NAMES, got, ref, size):
        check(name, y, r, tolerance(r, a, d, T, out if name in ("z", "dq", "dk", "dv") else F32, group=group))


# so many chains that none is cut into segments (more than 32768 / d / 2; the backward fewer): 31, 15 and 63 chunks a walk
@pytest.mark.parametrize("B,H,Hkv,T,d,dtype,lens", [(2, 264, 132, 1000, 64, BF16, [1000, 777]), (1, 264, 264, 490, 128, BF16, None),
                                                    (1, 132, 132, 490, 128, F32, [489]), (1, 514, 257, 2016, 32, F32, None),
                                                    (1, 1030, 1030, 700, 16, BF16, None)])
def test_long_walks(ttt, B, H, Hkv, T, d, dtype, lens):
    gen = torch.Generator().manual_seed(T)
    r = lambda h, std=1.0: (torch.randn(B, h, T, d, generator=gen) * std).to(dtype)  # noqa: E731
    q, k, v, dz = r(H), r(Hkv, d ** -0.5), r(Hkv), r(H)
    g = -torch.exp2(-10 * torch.rand(H, generator=gen))
    w0, dw = torch.randn(B, H, d, d, generator=gen), torch.randn(B, H, d, d, generator=gen)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    assert ttt.linear_attn_workspace_bytes(q, k, out_dtype=dtype) == 0  # (no states: one walk a chain)
    need = ttt.linear_attn_workspace_bytes(q, k, out_dtype=dtype, backward=True)
    assert need == 0 if H == Hkv else need >= 2 * B * H * T * d * 4
    on = [x.to(DEV) for x in (q, k, v, g)]
    more = dict(w0=w0.to(DEV), lens=None if n is None else n.to(DEV))
    z, w = ttt.linear_attn_fwd(*on, **more, out_dtype=dtype)
    got = (z, w, *ttt.linear_attn_bwd(*on, dz.to(DEV), dw_final=dw.to(DEV), **more))
    group = H // Hkv
    for b in range(B):
        for j in sorted({0, Hkv // 2, Hkv - 1}):  # a key / value head and its query heads
            hs = slice(j * group, (j + 1) * group)
            c = dict(q=q[b:b + 1, hs], k=k[b:b + 1, j:j + 1], v=v[b:b + 1, j:j + 1], log_decay=g[hs], w0=w0[b:b + 1, hs],
                     lens=None if n is None else n[b:b + 1])
            part = [x[b:b + 1, j:j + 1] if name in ("dk", "dv") else x[b:b + 1, hs]
                    for name, x in zip(NAMES, got)]
            against(ttt, part, c, dz[b:b + 1, hs], dw[b:b + 1, hs])


def test_offsets_past_32_bits(ttt):
    """Rows 2^17 elements apart, 20000 tokens: every tensor and every output reaches beyond 2^31 elements."""
    T, d = 20000, 16
    wide = torch.zeros(T, 1 << 17, device=DEV, dtype=BF16)
    gen = torch.Generator().manual_seed(3)
    place = lambda i: wide[:, 64 * i:64 * i + d][None, None]  # noqa: E731
    c = {n: torch.randn(1, 1, T, d, generator=gen).to(BF16) for n in ("q", "k", "v", "dz")}
    for i, n in enumerate(c):
        place(i).copy_(c[n])
    g = torch.tensor([-0.01])
    dw = torch.randn(1, 1, d, d, generator=gen)
    q, k, v, dz = (place(i) for i in range(4))
    z, w = ttt.linear_attn_fwd(q, k, v, g.to(DEV), z=place(4))
    out = (place(5), place(6), place(7), torch.empty(1, 1, device=DEV), torch.empty(1, 1, d, d, device=DEV))
    got = ttt.linear_attn_bwd(q, k, v, g.to(DEV), dz, dw_final=dw.to(DEV), out=out)
    against(ttt, (z, w, *got), dict(q=c["q"], k=c["k"], v=c["v"], log_decay=g), c["dz"], dw)
    # nothing beside the outputs' columns
    mask = torch.ones(1 << 17, dtype=torch.bool, device=DEV)
    for i in range(8):
        mask[64 * i:64 * i + d] = False
    assert not any(bool((rows[:, mask] != 0).any()) for rows in wide.split(1000))
