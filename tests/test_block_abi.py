"""Host-side checks of the short convolution, the selective scan and the block norm, without a GPU: the C ABI through
ttt_*_validate with fake (never dereferenced) addresses, and what the Python binding refuses."""
import ctypes

import pytest
import torch

import test_sequence_layer_amd as ttt

OK, NULL, SHAPE, DTYPE, UNSUP, ALIAS, ALIGN, HIP, STRIDE, FLAGS, POS, WORKSPACE, SCRATCH = range(13)
GB = 1 << 30
S = ttt.Strides
L = ttt.lib()
P = ctypes.byref


def rows(T, D):
    return S(T * D, 7, D)  # (h is not looked at)


def conv_desc(B=2, T=64, D=64, K=4, ind=1, outd=1, flags=1, reserved=0, **st):
    s = dict(dict.fromkeys(("x", "y", "dx"), rows(T, D)), **st)
    return ttt.ShortConvDesc(B, T, D, K, ind, outd, flags, reserved, s["x"], s["y"], s["dx"])


def scan_desc(B=2, T=64, D=64, N=16, G=2, ind=1, outd=1, flags=1, **st):
    r, b = rows(T, D), S(G * T * N, T * N, N)
    s = dict(dict.fromkeys(("u", "dt", "z", "y", "du", "ddt", "dz"), r), Bm=b, Cm=b, dBm=b, dCm=b)
    s.update(st)
    return ttt.SelectiveScanDesc(B, T, D, N, G, ind, outd, flags, *(s[x] for x in ("u", "dt", "z", "y", "Bm", "Cm", "du", "ddt",
                                                                                   "dz", "dBm", "dCm")))


def norm_desc(B=2, T=64, D=64, ind=1, rd=0, flags=1, eps=1e-6, reserved=0, **st):
    names = ("x", "z", "res", "s", "y", "dx", "dz", "dres")
    s = dict(dict.fromkeys(names, rows(T, D)), **st)
    return ttt.BlockNormDesc(B, T, D, ind, rd, flags, eps, reserved, *(s[x] for x in names))


def call(f, names):
    base = {n: (i + 1) * GB for i, n in enumerate(names)}
    if "wsb" in base:
        base["wsb"] = GB

    def run(d, **over):
        a = {**base, **over}
        return f(None if d is None else P(d), *a.values())

    run.base, run.names = base, names
    return run


CONV = ("x", "w", "bias", "state", "lens")
conv_fwd = call(L.ttt_short_conv_fwd_validate, CONV + ("y", "sf"))
conv_bwd = call(L.ttt_short_conv_bwd_validate, CONV + ("dy", "dsf", "dx", "dw", "dbias", "ds", "ws", "wsb"))
conv_dec = call(L.ttt_short_conv_decode_validate, ("x", "w", "bias", "lens", "y", "state"))
SCAN = ("u", "dt", "A", "Bm", "Cm", "D", "z", "bias", "h0", "lens")
scan_fwd = call(L.ttt_selective_scan_fwd_validate, SCAN + ("y", "h", "ws", "wsb"))
scan_bwd = call(L.ttt_selective_scan_bwd_validate, SCAN + ("dy", "dh", "du", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "ws", "wsb"))
scan_dec = call(L.ttt_selective_scan_decode_validate, ("u", "dt", "A", "Bm", "Cm", "D", "z", "bias", "lens", "y", "h"))
NORM = ("x", "z", "res", "alpha", "gp", "bp", "gn")
norm_fwd = call(L.ttt_block_norm_fwd_validate, NORM + ("bn", "lens", "s", "y"))
norm_bwd = call(L.ttt_block_norm_bwd_validate, NORM + ("lens", "ds", "dy", "dx", "dz", "dres", "da", "dgp", "dbp", "dgn", "dbn", "ws", "wsb"))

EVERY = [(conv_desc, c) for c in (conv_fwd, conv_bwd, conv_dec)] + [(scan_desc, c) for c in (scan_fwd, scan_bwd, scan_dec)] + [
    (norm_desc, c) for c in (norm_fwd, norm_bwd)]
OPTIONAL = {"bias", "state", "lens", "sf", "dsf", "dbias", "ds", "D", "h0", "dh", "dD", "db", "dh0", "z", "dz", "res", "alpha",
            "bp", "bn", "dres", "da", "dgp", "dbp", "dgn", "dbn"}


def needed(c):
    must = [n for n in c.names if n not in OPTIONAL and n not in ("ws", "wsb")]
    if c is conv_dec:
        must.append("state")
    return [n for n in must if not (c in (norm_fwd, norm_bwd) and n in ("gp", "gn", "s", "y", "dy"))]


@pytest.mark.parametrize("desc,c", EVERY)
def test_valid_calls(desc, c):
    for ind in (0, 1):
        for other in (0, 1):
            d = desc(ind=ind, **({"rd": other} if desc is norm_desc else {"outd": other}))
            assert c(d) == OK
    assert c(desc(T=1)) == OK and c(desc(T=61, D=62)) == OK and c(desc(flags=0)) == OK
    for n in c.names:
        if n in OPTIONAL - {"z", "dz"} and not (c is conv_dec and n == "state"):
            assert c(desc(), **{n: None}) == OK, n


@pytest.mark.parametrize("desc,c", EVERY)
def test_desc_refusals(desc, c):
    assert c(None) == NULL
    for kw in (dict(B=-1), dict(T=-1), dict(D=0), dict(B=1 << 30, T=1 << 29)):
        assert c(desc(**kw)) == SHAPE, kw
    big = S(1 << 40, 0, 64)
    names = [n for n, _ in desc()._fields_ if isinstance(getattr(desc(), n), S)]
    assert c(desc(T=(1 << 30) + 1, **{n: big for n in names})) == SHAPE
    assert c(desc(ind=2)) == DTYPE and c(desc(**{"rd" if desc is norm_desc else "outd": -1})) == DTYPE
    assert c(desc(flags=4)) == FLAGS
    if desc is not scan_desc:
        assert c(desc(reserved=1)) == FLAGS
    if desc is conv_desc:
        assert c(desc(K=1)) == UNSUP and c(desc(K=5)) == UNSUP and c(desc(K=0)) == SHAPE
    if desc is scan_desc:
        assert c(desc(N=33)) == UNSUP and c(desc(N=0)) == SHAPE and c(desc(G=3)) == SHAPE and c(desc(G=0)) == SHAPE
    if desc is norm_desc:
        assert c(desc(D=8193)) == UNSUP
        for eps in (-1.0, float("nan"), float("inf")):
            assert c(desc(eps=eps)) == SHAPE


@pytest.mark.parametrize("desc,c", EVERY)
def test_null_and_empty(desc, c):
    for n in needed(c):
        assert c(desc(), **{n: None}) == NULL, n
    keep = {"ws", "wsb", "w", "dw", "A", "dA", "h"}
    nothing = {n: None for n in c.names if n not in keep}
    assert c(desc(B=0), **nothing) == OK
    if c is conv_dec:
        nothing.pop("state")
    assert c(desc(T=0), **nothing) == OK


def test_null_of_the_norm():
    for c in (norm_fwd, norm_bwd):
        assert c(norm_desc(), gp=None) == NULL             # beta without gamma
        assert c(norm_desc(), gp=None, bp=None) == OK
    assert norm_fwd(norm_desc(), s=None) == OK and norm_fwd(norm_desc(), s=None, y=None) == NULL
    assert norm_fwd(norm_desc(), y=None, gn=None, bn=None) == OK and norm_fwd(norm_desc(), gn=None, bn=None) == NULL
    assert norm_fwd(norm_desc(), y=None, gn=None) == NULL
    assert norm_bwd(norm_desc(), ds=None) == OK and norm_bwd(norm_desc(), dy=None, gn=None) == OK
    assert norm_bwd(norm_desc(), ds=None, dy=None) == NULL and norm_bwd(norm_desc(), gn=None) == NULL
    assert norm_bwd(norm_desc(), z=None) == NULL and norm_bwd(norm_desc(), dz=None) == NULL
    assert norm_bwd(norm_desc(), z=None, dz=None) == OK
    assert scan_bwd(scan_desc(), z=None) == NULL and scan_bwd(scan_desc(), dz=None) == NULL
    assert scan_bwd(scan_desc(), z=None, dz=None) == OK and scan_fwd(scan_desc(), z=None) == OK


@pytest.mark.parametrize("desc,c", EVERY)
def test_strides(desc, c):
    d = desc()
    out = {"y", "s"} if c in (conv_fwd, conv_dec, scan_fwd, scan_dec, norm_fwd) else {"dx", "du", "ddt", "dz", "dBm", "dCm", "dres"}
    grads = {"dx", "du", "ddt", "dz", "dBm", "dCm", "dres"}
    for n, _ in d._fields_:
        st = getattr(d, n)
        if not isinstance(st, S) or (n in grads and n not in out):
            continue
        assert c(desc(**{n: S(-1, st.h, st.t)})) == STRIDE, n
        assert c(desc(**{n: S(1 << 60, st.h, st.t)})) == STRIDE, n
        # inputs may repeat, outputs may not
        assert c(desc(**{n: S(0, st.h, st.t)})) == (STRIDE if n in out else OK), n
        assert c(desc(**{n: S(st.b, st.h, 0)})) == (STRIDE if n in out else OK), n
    # strides of dimensions of size 1 carry nothing
    names = [n for n, _ in d._fields_ if isinstance(getattr(d, n), S)]
    more = {"G": 1} if desc is scan_desc else {}
    assert c(desc(B=1, T=1, **more, **{n: S(-5, -3, -1) for n in names})) == OK


@pytest.mark.parametrize("desc,c", EVERY)
def test_alignment_is_the_elements(desc, c):
    d = desc(ind=0, **({"rd": 0} if desc is norm_desc else {"outd": 0}))
    for n in c.names:
        if n in ("wsb",):
            continue
        if n == "ws":
            assert c(d, ws=c.base["ws"] + 8) == (WORKSPACE if c is not scan_fwd or d.T > 4096 else OK)
            continue
        assert c(d, **{n: c.base[n] + 2}) == ALIGN, n
        assert c(d, **{n: c.base[n] + 4}) == OK, n


@pytest.mark.parametrize("desc,c", EVERY)
def test_alias(desc, c):
    outs = {conv_fwd: ("y", "sf"), conv_bwd: ("dx", "dw", "dbias", "ds", "ws"), conv_dec: ("y", "state"), scan_fwd: ("y", "h"),
            scan_bwd: ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "ws"), scan_dec: ("y", "h"),
            norm_fwd: ("s", "y"), norm_bwd: ("dx", "dz", "dres", "da", "dgp", "dbp", "dgn", "dbn", "ws")}[c]
    for o in outs:
        for n in c.names:
            if n in (o, "wsb") or (c is scan_fwd and (o, n) == ("h", "ws")):
                continue
            want = ALIAS
            if (c is scan_fwd and (o, n) == ("h", "h0")) or (c is norm_fwd and (o, n) == ("s", "res")):
                want = OK  # the state and the residual stream may go on in place
            if n == "ws" and c is scan_fwd:
                continue
            assert c(desc(), **{o: c.base[n]}) == want, (o, n)
    if c is norm_fwd:
        assert c(desc(s=S(64 * 80, 0, 80)), s=c.base["res"]) == ALIAS  # (not the same strides)
        assert c(desc(), s=c.base["res"] + 4) == ALIAS
    if c is scan_fwd:
        assert c(desc(), h=c.base["h0"] + 4) == ALIAS


def test_slices_of_one_row():
    """Halves of a projection, and outputs beside each other in one buffer."""
    half = S(64 * 128, 0, 128)
    assert conv_fwd(conv_desc(x=half, y=half), y=conv_fwd.base["x"] + 128) == OK
    assert conv_fwd(conv_desc(x=half, y=half), y=conv_fwd.base["x"] + 126) == ALIAS
    bc = S(2 * 64 * 32, 64 * 32, 32)
    d = scan_desc(dBm=bc, dCm=bc, du=half, dz=half)
    assert scan_bwd(d, dC=scan_bwd.base["dB"] + 32, dz=scan_bwd.base["du"] + 128) == OK
    assert scan_bwd(d, dC=scan_bwd.base["dB"] + 30) == ALIAS
    assert norm_bwd(norm_desc(dx=half, dz=half), dz=norm_bwd.base["dx"] + 128) == OK


def test_workspace():
    for d, c, need in ((conv_desc(T=4096), conv_bwd, L.ttt_short_conv_workspace_bytes(P(conv_desc(T=4096)))),
                       (scan_desc(T=4096), scan_fwd, L.ttt_selective_scan_workspace_bytes(P(scan_desc(T=4096)), 0)),
                       (scan_desc(T=4096), scan_bwd, L.ttt_selective_scan_workspace_bytes(P(scan_desc(T=4096)), 1)),
                       (norm_desc(), norm_bwd, L.ttt_block_norm_workspace_bytes(P(norm_desc())))):
        assert need > 0
        assert c(d, wsb=need) == OK and c(d, wsb=need - 1) == WORKSPACE
        assert c(d, ws=None) == WORKSPACE and c(d, ws=c.base["ws"] + 8) == WORKSPACE
    assert L.ttt_selective_scan_workspace_bytes(P(scan_desc(B=64, D=4096)), 0) == 0
    for f, d in ((L.ttt_short_conv_workspace_bytes, conv_desc(K=9)), (L.ttt_block_norm_workspace_bytes, norm_desc(D=0))):
        assert f(P(d)) == -1
    assert L.ttt_selective_scan_workspace_bytes(P(scan_desc(N=64)), 0) == -1


def test_launch_limits():
    big = S(1 << 38, 0, 8)
    assert conv_fwd(conv_desc(B=64, T=1 << 30, D=8, x=big, y=big)) == SHAPE
    assert scan_dec(scan_desc(B=1 << 25, T=1, D=64, N=4, G=1, u=rows(1, 64))) == SHAPE


# ------------------------------------------------------------- the binding --

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_wants_the_gpu():
    f = torch.float32
    for run in (lambda: ttt.short_conv_fwd(z(1, 2, 8), z(8, 4, dtype=f)),
                lambda: ttt.selective_scan_fwd(z(1, 2, 8), z(1, 2, 8), z(8, 4, dtype=f), z(1, 1, 2, 4), z(1, 1, 2, 4)),
                lambda: ttt.block_norm_fwd(z(1, 2, 8))):
        with pytest.raises(ValueError, match="GPU"):
            run()


def conv_args(**over):
    f = torch.float32
    a = dict(x=z(2, 5, 8), w=z(8, 4, dtype=f), bias=z(8, dtype=f), state=z(2, 3, 8), lens=z(2, dtype=torch.int32),
             out_dtype=torch.bfloat16, silu=True, y=z(2, 5, 8))
    a.update(over)
    return ttt._conv_call(**a)


def scan_args(**over):
    f = torch.float32
    a = dict(u=z(2, 5, 8), dt=z(2, 5, 8), A=z(8, 4, dtype=f), Bm=z(2, 2, 5, 4), Cm=z(2, 2, 5, 4), D=z(8, dtype=f), z=z(2, 5, 8),
             dt_bias=z(8, dtype=f), h0=z(2, 8, 4, dtype=f), softplus=True, lens=None, y=z(2, 5, 8))
    a.update(over)
    return ttt._scan_call(**a)


def norm_args(**over):
    f = torch.float32
    p = z(8, dtype=f)
    a = dict(x=z(2, 5, 8), z=z(2, 5, 8), res=z(2, 5, 8, dtype=f), alpha=p, gamma_post=p, beta_post=p, gamma_pre=p, beta_pre=p,
             kind="rms", eps=1e-6, gate_first=False, lens=None, s=z(2, 5, 8, dtype=f), y=z(2, 5, 8), res_dtype=f)
    a.update(over)
    return ttt._norm_call(**a)


def test_binding_refusals():
    f, i64 = torch.float32, torch.int64
    conv_args(), scan_args(), norm_args()
    for make, over in ((conv_args, dict(x=z(5, 8))), (conv_args, dict(w=z(7, 4, dtype=f))), (conv_args, dict(w=z(8, 4))),
                       (conv_args, dict(bias=z(7, dtype=f))), (conv_args, dict(state=z(2, 4, 8))),
                       (conv_args, dict(state=z(2, 3, 8, dtype=f))), (conv_args, dict(lens=z(3, dtype=torch.int32))),
                       (conv_args, dict(y=z(2, 5, 9))), (conv_args, dict(x=z(2, 8, 5).transpose(1, 2))),
                       (conv_args, dict(w=z(4, 8, dtype=f).t())),
                       (scan_args, dict(dt=z(2, 5, 9))), (scan_args, dict(dt=z(2, 5, 8, dtype=f))), (scan_args, dict(u=z(5, 8))),
                       (scan_args, dict(A=z(8, 5, dtype=f))), (scan_args, dict(Bm=z(2, 3, 5, 4))), (scan_args, dict(Cm=z(2, 2, 5, 3))),
                       (scan_args, dict(Bm=z(2, 5, 4))), (scan_args, dict(h0=z(2, 4, 8, dtype=f))), (scan_args, dict(D=z(8))),
                       (scan_args, dict(z=z(2, 4, 8))), (scan_args, dict(Bm=z(2, 2, 4, 5).transpose(2, 3))),
                       (norm_args, dict(z=z(2, 5, 9))), (norm_args, dict(res=z(2, 5, 8))), (norm_args, dict(alpha=z(9, dtype=f))),
                       (norm_args, dict(gamma_pre=z(8))), (norm_args, dict(kind="batch")), (norm_args, dict(x=z(2, 8)))):
        with pytest.raises(ValueError):
            make(**over)
    for make in (conv_args, scan_args, norm_args):
        with pytest.raises(TypeError):
            make(lens=z(2, dtype=i64))


def test_binding_workspace_bytes():
    x, w = z(2, 300, 64), z(64, 4, dtype=torch.float32)
    assert ttt.short_conv_workspace_bytes(x, w) == L.ttt_short_conv_workspace_bytes(P(conv_desc(T=300)))
    b = z(2, 2, 300, 16)
    for back in (False, True):
        assert ttt.selective_scan_workspace_bytes(x, b, back) == L.ttt_selective_scan_workspace_bytes(P(scan_desc(T=300)), back)
    assert ttt.block_norm_workspace_bytes(x) == L.ttt_block_norm_workspace_bytes(P(norm_desc(T=300)))
