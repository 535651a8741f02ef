"""Host-side checks of the linear-attention and rotary entry points, without a GPU:
the C ABI through ttt_*_validate with fake (never dereferenced) addresses, and what
the Python binding refuses."""
import ctypes

import pytest

import test_sequence_layer_amd as ttt

OK, NULL, SHAPE, DTYPE, UNSUP, ALIAS, ALIGN, HIP, STRIDE, FLAGS, POS, WORKSPACE, SCRATCH = range(13)
GB = 1 << 30
S = ttt.Strides
L = ttt.lib()


def desc(B=2, H=4, Hkv=2, T=64, d=64, ind=1, outd=1, flags=0, scale=1.0, reserved=0, wstride=0, **strides):
    q, k = S(H * T * d, T * d, d), S(Hkv * T * d, T * d, d)
    s = dict(q=q, k=k, v=k, z=q, dq=q, dk=k, dv=k)
    s.update(strides)
    return ttt.LinearAttnDesc(B, H, Hkv, T, d, ind, outd, flags, scale, reserved, wstride,
                              *(s[x] for x in ("q", "k", "v", "z", "dq", "dk", "dv")))


FWD = dict(q=GB, k=2 * GB, v=3 * GB, g=4 * GB, w0=5 * GB, lens=6 * GB, z=7 * GB, wf=8 * GB, ws=9 * GB, wsb=GB)
BWD = dict(q=GB, k=2 * GB, v=3 * GB, g=4 * GB, w0=5 * GB, lens=6 * GB, dz=7 * GB, dwf=8 * GB, dq=10 * GB, dk=11 * GB,
           dv=12 * GB, dg=13 * GB, dw0=14 * GB, ws=15 * GB, wsb=GB)
DEC = dict(q=GB, k=2 * GB, v=3 * GB, g=4 * GB, lens=6 * GB, rope=None, z=7 * GB, w=8 * GB)


def fwd(d, **over):
    a = {**FWD, **over}
    return L.ttt_linear_attn_fwd_validate(None if d is None else ctypes.byref(d), *a.values())


def bwd(d, **over):
    a = {**BWD, **over}
    return L.ttt_linear_attn_bwd_validate(None if d is None else ctypes.byref(d), *a.values())


def dec(d, **over):
    a = {**DEC, **over}
    r = a["rope"]
    a["rope"] = None if r is None else ctypes.byref(r)
    return L.ttt_linear_attn_decode_validate(None if d is None else ctypes.byref(d), *a.values())


def rope(pos=20 * GB, sb=1, st=0, off=0, freqs=21 * GB, rot=64, inter=0, scale=1.0, reserved=0):
    return ttt.Rope(pos, sb, st, off, freqs, rot, inter, scale, reserved)


def rdesc(B=2, H=4, Hkv=2, T=64, d=64, dtype=1, flags=0, reserved=0, **strides):
    q, k = S(H * T * d, T * d, d), S(Hkv * T * d, T * d, d)
    s = dict(q=q, k=k, qo=q, ko=k)
    s.update(strides)
    return ttt.RotaryDesc(B, H, Hkv, T, d, dtype, flags, reserved, s["q"], s["k"], s["qo"], s["ko"])


def rot(d, r, q=GB, k=2 * GB, qo=3 * GB, ko=4 * GB):
    return L.ttt_rotary_validate(None if d is None else ctypes.byref(d), None if r is None else ctypes.byref(r), q, k, qo,
                                 ko)


@pytest.mark.parametrize("call", [fwd, bwd, dec])
def test_valid_calls(call):
    for ind in (0, 1):
        for outd in (0, 1):
            for d in (16, 32, 64, 128):
                assert call(desc(d=d, ind=ind, outd=outd)) == OK
    assert call(desc(), lens=None) == OK
    assert call(desc(T=1)) == OK and call(desc(T=61)) == OK
    assert call(desc(H=6, Hkv=1)) == OK


@pytest.mark.parametrize("call", [fwd, bwd, dec])
def test_desc_refusals(call):
    assert call(None) == NULL
    for kw in (dict(B=-1), dict(T=-1), dict(d=0), dict(H=4, Hkv=3), dict(H=4, Hkv=0), dict(H=2, Hkv=4),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(B=1 << 20, H=1 << 20, Hkv=1 << 20)):
        assert call(desc(**kw)) == SHAPE, kw
    big = S(1 << 36, 1 << 36, 64)
    assert call(desc(T=(1 << 30) + 1, q=big, k=big, v=big, z=big, dq=big, dk=big, dv=big)) == SHAPE
    assert call(desc(ind=2)) == DTYPE and call(desc(outd=-1)) == DTYPE
    assert call(desc(flags=1)) == FLAGS and call(desc(reserved=1)) == FLAGS
    assert call(desc(wstride=64)) == STRIDE
    assert call(desc(d=48)) == UNSUP and call(desc(d=256)) == UNSUP


@pytest.mark.parametrize("call,names", [(fwd, ("q", "k", "v", "g", "z", "wf")),
                                        (bwd, ("q", "k", "v", "g", "dz", "dq", "dk", "dv", "dg", "dw0")),
                                        (dec, ("q", "k", "v", "g", "z", "w"))])
def test_null_and_empty(call, names):
    for n in names:
        assert call(desc(), **{n: None}) == NULL, n
    none = {n: None for n in names}
    assert call(desc(B=0), **none) == OK
    assert call(desc(H=0, Hkv=0), **none) == OK
    # no tokens: only the state and the decay are looked at
    keep = {"g", "wf", "w", "dg", "dw0"}
    assert call(desc(T=0), **{n: None for n in names if n not in keep}) == OK
    assert call(desc(T=0), g=None) == NULL


def test_strides():
    d = 64
    ok = S(64 * 4 * d, d, 4 * d)  # [B, T, H, d]
    okk = S(64 * 2 * d, d, 2 * d)
    for call in (fwd, bwd, dec):
        assert call(desc(q=ok, k=okk, v=okk, z=ok, dq=ok, dk=okk, dv=okk)) == OK
        assert call(desc(q=S(-64, 0, 0))) == STRIDE
        assert call(desc(k=S(0, 0, 0))) == OK              # inputs may repeat
        assert call(desc(k=S(1 << 60, 0, 0))) == STRIDE    # beyond any memory
    assert fwd(desc(z=S(0, 64 * d, d))) == STRIDE          # outputs may not
    assert fwd(desc(z=S(4 * 64 * d, 64 * d, d - 8))) == STRIDE
    assert dec(desc(z=S(0, 64 * d, d))) == STRIDE
    assert bwd(desc(dq=S(0, 64 * d, d))) == STRIDE and bwd(desc(dv=S(0, 64 * d, d))) == STRIDE
    # strides of dimensions of size 1 carry nothing
    assert fwd(desc(B=1, H=1, Hkv=1, T=1, q=S(-5, -7, -1), k=S(3, 3, 3), v=S(1, 1, 1), z=S(0, 0, 0))) == OK


def test_alignment():
    for call, names in ((fwd, ("q", "k", "v", "z", "w0", "wf")), (bwd, ("q", "k", "v", "dz", "dq", "dk", "dv", "w0", "dwf",
                                                                        "dw0"))):
        for n in names:
            base = (FWD if call is fwd else BWD)[n]
            assert call(desc(), **{n: base + 8}) == ALIGN, n
        assert call(desc(), g=4 * GB + 2) == ALIGN and call(desc(), lens=6 * GB + 2) == ALIGN
    assert fwd(desc(q=S(4 * 64 * 68, 64 * 68, 68))) == ALIGN
    # single tokens come from anywhere
    assert dec(desc(q=S(4 * 64 * 67, 64 * 67, 67)), q=GB + 2) == OK
    assert dec(desc(), q=GB + 1) == ALIGN and dec(desc(), w=8 * GB + 4) == ALIGN


def test_workspace():
    few = desc(B=1, H=1, Hkv=1, T=4096)
    for backward, call in ((0, fwd), (1, bwd)):
        need = L.ttt_linear_attn_workspace_bytes(ctypes.byref(few), backward)
        assert need > 0
        assert call(few, wsb=need) == OK and call(few, wsb=need - 1) == WORKSPACE
        assert call(few, ws=None) == WORKSPACE and call(few, ws=9 * GB + 8) == WORKSPACE
        many = desc(B=64, H=16, Hkv=16, T=64)
        assert L.ttt_linear_attn_workspace_bytes(ctypes.byref(many), backward) == 0
        assert call(many, ws=None, wsb=0) == OK
    shared = desc(B=64, H=16, Hkv=8, T=64)  # the parts of shared heads
    assert L.ttt_linear_attn_workspace_bytes(ctypes.byref(shared), 1) >= 2 * 64 * 16 * 64 * 64 * 4
    assert L.ttt_linear_attn_workspace_bytes(ctypes.byref(desc(d=20)), 0) == -1
    assert L.ttt_linear_attn_workspace_bytes(None, 0) == -1


def test_alias():
    for n in ("q", "k", "v", "g", "lens", "w0"):
        assert fwd(desc(), z=FWD[n]) == ALIAS, n
    for n in ("q", "k", "v", "g", "lens"):
        assert fwd(desc(), wf=FWD[n]) == ALIAS, n
    assert fwd(desc(), wf=FWD["z"]) == ALIAS
    assert fwd(desc(), wf=FWD["w0"]) == ALIAS                                   # a shared W0
    each = desc(wstride=4 * 64 * 64)
    assert fwd(each, wf=FWD["w0"]) == OK                                        # in place
    assert fwd(each, wf=FWD["w0"] + 64) == ALIAS
    few = dict(B=1, H=1, Hkv=1, T=4096)
    for n in ("q", "k", "v", "g", "lens", "w0", "z", "wf"):
        assert fwd(desc(**few), ws=FWD[n]) == ALIAS, n
    for o in ("dq", "dk", "dv", "dg", "dw0"):
        for n in ("q", "k", "v", "g", "w0", "lens", "dz", "dwf"):
            assert bwd(desc(), **{o: BWD[n]}) == ALIAS, (o, n)
    for o, p in (("dq", "dk"), ("dk", "dv"), ("dq", "dg"), ("dg", "dw0"), ("dv", "dw0")):
        assert bwd(desc(), **{o: BWD[p]}) == ALIAS, (o, p)
    for n in ("q", "k", "v", "g", "lens", "z"):
        assert dec(desc(), w=DEC[n]) == ALIAS, n
    assert dec(desc(), z=DEC["q"]) == ALIAS


def test_gradients_as_slices_of_one_buffer():
    """dq, dk, dv as [B, T, 3, H, d] slices: ranges that interleave without sharing an element."""
    H, T, d = 4, 64, 64
    s = S(T * 3 * H * d, d, 3 * H * d)
    args = dict(Hkv=H, dq=s, dk=s, dv=s)
    base = 40 * GB
    assert bwd(desc(**args), dq=base, dk=base + 2 * H * d, dv=base + 4 * H * d) == OK
    assert bwd(desc(**args), dq=base, dk=base + 2 * H * d - 16, dv=base + 4 * H * d) == ALIAS
    assert bwd(desc(**args), dq=base, dk=base + 2 * H * d, dv=base + 4 * H * d + 16) == ALIAS  # into the next row
    # [B, 3, H, T, d]
    s = S(3 * H * T * d, T * d, d)
    n = 2 * H * T * d
    args = dict(Hkv=H, dq=s, dk=s, dv=s)
    assert bwd(desc(**args), dq=base, dk=base + n, dv=base + 2 * n) == OK
    assert bwd(desc(**args), dq=base, dk=base + n - 128, dv=base + 2 * n) == ALIAS


def test_rope_refusals():
    ok = desc()
    assert dec(ok, rope=rope()) == OK
    for kw in (dict(rot=63), dict(rot=-2), dict(rot=66), dict(scale=float("nan"))):
        assert dec(ok, rope=rope(**kw)) == SHAPE and rot(rdesc(), rope(**kw)) == SHAPE, kw
    for kw in (dict(sb=-1), dict(st=-1)):
        assert dec(ok, rope=rope(**kw)) == STRIDE and rot(rdesc(), rope(**kw)) == STRIDE, kw
    for kw in (dict(inter=2), dict(reserved=1)):
        assert dec(ok, rope=rope(**kw)) == FLAGS and rot(rdesc(), rope(**kw)) == FLAGS, kw
    assert dec(ok, rope=rope(freqs=None)) == NULL
    assert dec(ok, rope=rope(freqs=None, rot=0)) == OK
    assert dec(ok, rope=rope(pos=None, off=7)) == OK
    assert dec(ok, rope=rope(pos=20 * GB + 4)) == ALIGN and dec(ok, rope=rope(freqs=21 * GB + 4)) == ALIGN
    assert dec(ok, rope=rope(), w=20 * GB) == ALIAS and dec(ok, rope=rope(), z=21 * GB) == ALIAS


def test_rotary_refusals():
    r = rope()
    assert rot(rdesc(), r) == OK and rot(None, r) == NULL and rot(rdesc(), None) == NULL
    assert rot(rdesc(d=100), r) == OK and rot(rdesc(flags=1), r) == OK
    for kw in (dict(B=-1), dict(d=0), dict(T=-3), dict(Hkv=-1)):
        assert rot(rdesc(**kw), r) == SHAPE, kw
    assert rot(rdesc(dtype=2), r) == DTYPE and rot(rdesc(flags=2), r) == FLAGS and rot(rdesc(reserved=1), r) == FLAGS
    for n in ("q", "k", "qo", "ko"):
        assert rot(rdesc(), r, **{n: None}) == NULL
        assert rot(rdesc(), r, **{n: 9 * GB + 1}) == ALIGN
    assert rot(rdesc(Hkv=0), r, k=None, ko=None) == OK
    assert rot(rdesc(B=0), r, q=None, k=None, qo=None, ko=None) == OK
    assert rot(rdesc(qo=S(0, 64, 64 * 4)), r) == STRIDE and rot(rdesc(q=S(0, 0, 0)), r) == OK
    # in place, and not quite
    assert rot(rdesc(), r, qo=GB, ko=2 * GB) == OK
    assert rot(rdesc(), r, qo=GB) == OK
    assert rot(rdesc(), r, qo=GB + 128) == ALIAS
    assert rot(rdesc(qo=S(64, 2 * 64 * 64, 2 * 64)), r, qo=GB) == ALIAS    # another layout over q
    assert rot(rdesc(), r, qo=2 * GB) == ALIAS and rot(rdesc(), r, ko=GB) == ALIAS and rot(rdesc(), r, ko=3 * GB) == ALIAS
    assert rot(rdesc(Hkv=4), r, k=GB, qo=GB, ko=GB) == ALIAS               # q and k the same tensor, both in place
    # q and k in place within one [B, T, 3, H, d] buffer
    s = S(64 * 3 * 4 * 64, 64, 3 * 4 * 64)
    packed = rdesc(Hkv=4, q=s, k=s, qo=s, ko=s)
    assert rot(packed, r, q=GB, k=GB + 2 * 4 * 64, qo=GB, ko=GB + 2 * 4 * 64) == OK
    assert rot(packed, r, q=GB, k=GB + 4 * 64, qo=GB, ko=GB + 4 * 64) == ALIAS


# ---- the Python binding ----------------------------------------------------------

torch = pytest.importorskip("torch")


def test_python_refusals():
    q, k, g = torch.zeros(2, 4, 8, 16), torch.zeros(2, 2, 8, 16), torch.zeros(4)
    f = ttt.rotary_freqs(16)[0]
    with pytest.raises(ValueError, match="on the GPU"):
        ttt.linear_attn_fwd(q, k, k, g)
    with pytest.raises(ValueError, match="on the GPU"):
        ttt.rotary(q, k, 0, f)
    with pytest.raises(ValueError, match="dtype"):
        ttt.linear_attn_fwd(q, k.bfloat16(), k, g)
    with pytest.raises(ValueError, match="share"):
        ttt.linear_attn_fwd(q, k[:, :1].expand(2, 3, 8, 16), k[:, :1].expand(2, 3, 8, 16), g)
    with pytest.raises(ValueError, match="expected"):
        ttt.linear_attn_fwd(q, k[:, :, :7], k, g)
    with pytest.raises(ValueError, match="log_decay"):
        ttt.linear_attn_fwd(q, k, k, g[:3])
    with pytest.raises(TypeError, match="log_decay"):
        ttt.linear_attn_fwd(q, k, k, g.double())
    with pytest.raises(ValueError, match="lens"):
        ttt.linear_attn_fwd(q, k, k, g, lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="lens"):
        ttt.linear_attn_fwd(q, k, k, g, lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="w0"):
        ttt.linear_attn_fwd(q, k, k, g, w0=torch.zeros(2, 16, 16))
    with pytest.raises(ValueError, match=r"\[B, H, T, d\]"):
        ttt.linear_attn_fwd(q[0], k, k, g)
    with pytest.raises(ValueError, match="expected"):
        ttt.rotary(q, k[:, :, :7], 0, f)


def test_rotary_freqs():
    f, s = ttt.rotary_freqs(8)
    assert f.dtype == torch.float64 and s == 1.0 and torch.allclose(f, 10000.0 ** -(torch.arange(4).double() / 4))
    f2, s = ttt.rotary_freqs(8, scaling="linear", factor=4.0)
    assert s == 1.0 and torch.allclose(f2, f / 4)
    # the base raised: the fastest pair as it was, the slowest slowed by the factor
    f3, s = ttt.rotary_freqs(8, scaling="ntk", factor=4.0)
    assert s == 1.0 and f3[0] == 1.0 and torch.allclose(f3[-1], f[-1] / 4)
    f4, s = ttt.rotary_freqs(64, scaling="yarn", factor=4.0, original=2048)
    g4 = ttt.rotary_freqs(64)[0]
    assert abs(s - (0.1 * torch.log(torch.tensor(4.0)).item() + 1)) < 1e-6
    assert f4[0] == g4[0] and f4[-1] == g4[-1] / 4 and ((f4 <= g4) & (f4 >= g4 / 4)).all()
    assert ttt.rotary_freqs(0)[0].numel() == 0 and ttt.rotary_freqs(2, scaling="ntk", factor=2.0)[0].tolist() == [1.0]
    for bad in (dict(rot=7), dict(rot=-2), dict(rot=8, scaling="cubic"), dict(rot=8, factor=2.0),
                dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, scaling="yarn", factor=2.0, beta_fast=1.0)):
        with pytest.raises(ValueError):
            ttt.rotary_freqs(**bad)


def test_threads_of_a_launch():
    # 2^32 threads are refused, one workgroup less than that many is not
    far = {n: (i + 1) << 44 for i, n in enumerate(["q", "k", "v", "g", "w0", "lens", "z", "wf", "ws", "dz", "dwf", "dq",
                                                   "dk", "dv", "dg", "dw0", "w", "qo", "ko"])}
    take = lambda names: {n: far[n] for n in names.split()}
    f = {**take("q k v g w0 lens z wf ws"), "wsb": 1 << 43}
    b = {**take("q k v g w0 lens dz dwf dq dk dv dg dw0 ws"), "wsb": 1 << 43}
    n = 1 << 20
    assert fwd(desc(B=n, H=16, Hkv=16, T=1), **f) == SHAPE
    assert fwd(desc(B=n - 1, H=16, Hkv=16, T=1), **f) == OK
    assert dec(desc(B=n, H=16, Hkv=16, T=1), **take("q k v g lens z w")) == SHAPE
    assert dec(desc(B=n - 1, H=16, Hkv=16, T=1), **take("q k v g lens z w")) == OK
    assert bwd(desc(B=n // 3 + 1, H=16, Hkv=16, T=1), **b) == SHAPE
    assert bwd(desc(B=n // 3, H=16, Hkv=16, T=1), **b) == OK
    # the sums over shared heads: B Hkv T d / 2 threads, and one for each decay's gradient
    assert bwd(desc(B=1, H=4, Hkv=2, T=1 << 26), **b) == SHAPE
    assert bwd(desc(B=1, H=4, Hkv=2, T=(1 << 26) - 16), **b) == OK
    assert bwd(desc(B=1, H=4, Hkv=4, T=1 << 26), **b) == OK
    r = rope(pos=None, sb=0, freqs=50 << 44)
    assert rot(rdesc(B=1, H=1, Hkv=1, T=1 << 26), r, **take("q k qo ko")) == SHAPE
    assert rot(rdesc(B=1, H=1, Hkv=1, T=(1 << 26) - 4), r, **take("q k qo ko")) == OK


def test_few_chains_are_walked_in_segments():
    """A workspace of one state a segment and chain (three in the backward, and the decay's sums)."""
    def segments(backward, **kw):
        d = desc(Hkv=kw["H"], outd=kw.get("ind", 1), **kw)
        need = L.ttt_linear_attn_workspace_bytes(ctypes.byref(d), backward)
        state = d.B * d.H * d.d * d.d * 4
        return need // (3 * state if backward else state)
    for backward in (0, 1):
        for T, n in ((1, 0), (352, 0), (353, 3), (384, 3), (512, 4), (1 << 20, 64)):
            assert segments(backward, B=1, H=2, T=T) == n, (backward, T)
        for T, n in ((160, 0), (161, 2), (288, 3), (289, 4)):
            assert segments(backward, B=1, H=2, T=T, ind=0) == n
            assert segments(backward, B=1, H=2, T=T, d=128) == n
    for d, n in ((16, 64), (32, 32), (64, 16), (128, 8)):
        assert segments(0, B=2, H=16, T=1 << 16, d=d) == n
    for d, n in ((16, 20), (32, 12), (64, 10), (128, 7)):
        assert segments(1, B=2, H=16, T=1 << 16, d=d) == n
    assert segments(0, B=32, H=16, T=1 << 16) == 0 == segments(1, B=21, H=16, T=1 << 16)


def test_gradients_interleaved_within_heads():
    """dq, dk, dv as [B, T, H, 3, d] slices, as a projection that keeps each head's three together leaves them."""
    H, T, d = 4, 64, 64
    s = S(T * 3 * H * d, 3 * d, 3 * H * d)
    base, n = 40 * GB, 2 * d
    for B in (1, 2):
        args = dict(B=B, Hkv=H, dq=s, dk=s, dv=s)
        assert bwd(desc(**args), dq=base, dk=base + n, dv=base + 2 * n) == OK
        assert bwd(desc(**args), dq=base + 2 * n, dk=base, dv=base + n) == OK
        assert bwd(desc(**args), dq=base, dk=base + n - 16, dv=base + 2 * n) == ALIAS
        assert bwd(desc(**args), dq=base, dk=base + n, dv=base + 2 * n + 16) == ALIAS      # into the next head's dq
    # [B, H, T, 3, d]
    s = S(T * 3 * H * d, T * 3 * d, 3 * d)
    args = dict(Hkv=H, dq=s, dk=s, dv=s)
    assert bwd(desc(**args), dq=base, dk=base + n, dv=base + 2 * n) == OK
    assert bwd(desc(**args), dq=base, dk=base + n, dv=base + 2 * n + 16) == ALIAS
    # [B, T, Hkv, group + 2, d] with one key / value head: q's four heads, then k, then v
    s = S(T * 6 * d, d, 6 * d)
    args = dict(Hkv=1, dq=s, dk=s, dv=s)
    assert bwd(desc(**args), dq=base, dk=base + 4 * n, dv=base + 5 * n) == OK
    assert bwd(desc(**args), dq=base, dk=base + 3 * n, dv=base + 5 * n) == ALIAS
    # one behind the other, of other strides
    q = S(H * T * d, T * d, d)
    assert bwd(desc(Hkv=H, dq=q, dk=S(T * H * d, d, H * d), dv=q), dq=base, dk=base + 2 * 2 * H * T * d,
               dv=base + 4 * 2 * H * T * d) == OK
    # the same first token, other strides between tokens: row 3 of one is row 1 of the other
    assert bwd(desc(B=1, H=1, Hkv=1, dq=S(0, 0, d), dk=S(0, 0, 3 * d)), dq=base, dk=base + 2 * 3 * d) == ALIAS


def test_rotary_in_place_within_heads():
    """q and k of a [B, T, H, 3, d] projection turned where they are"""
    H, T, d = 4, 64, 64
    s = S(T * 3 * H * d, 3 * d, 3 * H * d)
    p = rdesc(Hkv=H, q=s, k=s, qo=s, ko=s)
    r = rope()
    assert rot(p, r, q=GB, k=GB + 2 * d, qo=GB, ko=GB + 2 * d) == OK
    assert rot(p, r, q=GB, k=GB + 2 * d, qo=GB + 2 * d, ko=GB) == ALIAS
    assert rot(p, r, q=GB, k=GB + d, qo=GB, ko=GB + d) == ALIAS
    # k's output in the third place
    assert rot(p, r, q=GB, k=GB + 2 * d, qo=GB, ko=GB + 4 * d) == OK
    assert rot(p, r, q=GB, k=GB + 2 * d, qo=GB, ko=GB + 5 * d) == ALIAS


def test_apart_is_apart():
    """Random slices of one buffer against the elements themselves: never accepted where one is shared, and what is
    refused without one is not of the kinds that the header names (slices of the same rows)."""
    import random
    rng = random.Random(3)
    seen = {OK: 0, ALIAS: 0}
    for _ in range(3000):
        B, H, T, d = rng.choice([1, 2]), rng.choice([1, 2, 3]), rng.choice([1, 2, 3]), 16
        def strides():
            order, s, span = rng.sample("bht", 3), {}, d
            for a in order:
                s[a] = span + d * rng.choice([0, 0, 1, 2])
                span = s[a] + {"b": B, "h": H, "t": T}[a] * s[a] - s[a] if {"b": B, "h": H, "t": T}[a] > 1 else span
            return S(s["b"], s["h"], s["t"])
        a = strides()
        b = a if rng.random() < 0.7 else strides()
        off = rng.randrange(0, 20) * (d // 2)
        def cells(s, at):
            return {at + x * s.b + y * s.h + z * s.t + i for x in range(B) for y in range(H) for z in range(T) for i in range(d)}
        def ok(s):
            return len(cells(s, 0)) == B * H * T * d
        if not (ok(a) and ok(b)):
            continue
        got = bwd(desc(B=B, H=H, Hkv=H, T=T, d=d, dq=a, dk=b, dv=S(H * T * d, T * d, d)), dq=40 * GB, dk=40 * GB + 2 * off)
        if got == STRIDE:
            continue
        seen[got] += 1
        if cells(a, 0) & cells(b, off):
            assert got == ALIAS, (B, H, T, [a.b, a.h, a.t], [b.b, b.h, b.t], off)
    assert min(seen.values()) > 100, seen


def way(d, r, q=GB, k=2 * GB, qo=3 * GB, ko=4 * GB):
    return L.ttt_rotary_kernel_name(ctypes.byref(d), ctypes.byref(r), q, k, qo, ko)


def test_rotary_kernels():
    """Only rows at any address, or of more than 256 pieces, go element by element: an absent q or k takes no part in the
    choice, and turning in place makes no difference."""
    assert way(rdesc(), rope()) == b"ttt_rotary_halves" and way(rdesc(), rope(inter=1)) == b"ttt_rotary_interleaved"
    assert way(rdesc(), rope(rot=62)) == b"ttt_rotary_odd_halves"
    for d in (48, 80, 96, 160):  # 256 is no multiple of d / 8 pieces of bf16
        r = rope(rot=d)
        assert way(rdesc(d=d), r) == b"ttt_rotary_odd_halves"
        assert way(rdesc(d=d, Hkv=0), r, k=None, ko=None) == b"ttt_rotary_odd_halves"
        assert way(rdesc(d=d, H=0), r, q=None, qo=None) == b"ttt_rotary_odd_halves"
        assert way(rdesc(d=d, Hkv=0), r, k=None, ko=None, qo=GB) == b"ttt_rotary_odd_halves"
        assert way(rdesc(d=d), r, ko=2 * GB) == b"ttt_rotary_odd_halves"
    assert way(rdesc(d=2048), rope(rot=62)) == b"ttt_rotary_odd_halves"
    assert way(rdesc(d=2056), rope(rot=62)) == b"ttt_rotary_pairs"
    assert way(rdesc(), rope(), q=GB + 2) == b"ttt_rotary_pairs"
    assert way(rdesc(Hkv=0, k=S(3, 5, 7), ko=S(1, 1, 1)), rope(), k=6, ko=2) == b"ttt_rotary_halves"
    assert way(rdesc(), rope(rot=63)) is None and way(rdesc(B=0), rope()) is None
    assert way(rdesc(), rope(rot=0), qo=GB, ko=2 * GB) is None
