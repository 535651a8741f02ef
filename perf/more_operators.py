"""What the selective scan, the short convolution and the block norm are measured on.

The three are what stands around a sequence layer's state: the block norm joins a
block's output to the residual stream and normalises it for the next block, the short
convolution mixes each channel with its last few tokens, and the selective scan carries
a state per channel whose decay and input depend on the token:

    h_t = exp(dt_t A) h_{t-1} + dt_t B_t u_t,   y_t = C_t h_t + D u_t

``run`` computes them in elementary torch operations, or through the package where
``own`` is true.
"""
import math

import torch

own = False


def listed():
    return [
        # one short user prompt at the 125M layer's width (12 heads of 64, doubled): every launch and its latency shows
        scan("scan_prompt_short", "scan_fwd", B=1, T=67, D=1536),
        # prompts at the 1.3B layer's width (32 heads of 64, doubled) and its full length
        scan("scan_prompt_l1p3b", "scan_fwd", B=4, T=8192, D=4096),
        # a padded fp32 batch of odd length and width, two groups of channels, every sequence with a state of its own
        scan("scan_prompt_ragged_f32", "scan_fwd", B=3, T=1009, D=500, N=8, G=2, dtype="f32", out="f32", h0=True,
             ragged=True, gate=False),
        # training steps: the 125M layer, and a padded fp32 batch with states
        scan("scan_grad_l125m", "scan_bwd", B=8, T=2048, D=1536),
        scan("scan_grad_ragged_f32", "scan_bwd", B=3, T=531, D=200, N=16, G=2, dtype="f32", out="f32", h0=True, ragged=True),
        # one token for each of 512 running sequences of the 1.3B layer
        scan("scan_token_512", "scan_decode", B=512, T=1, D=4096, h0=True),
        # the convolution before the scan: prompts at the 1.3B layer's width as a slice of a wider projection, the 125M
        # layer's training step, one token for each of 512 sequences
        conv("conv_prompt_l1p3b", "conv_fwd", B=4, T=8192, D=4096, sliced=True),
        conv("conv_grad_l125m", "conv_bwd", B=8, T=2048, D=1536),
        conv("conv_token_512", "conv_decode", B=512, T=1, D=4096, state=True),
        # the join of two blocks: one token for each of 16 sequences, prompts with an fp32 residual stream, the 125M
        # layer's training step
        norm("norm_token_16", "norm_fwd", B=16, T=1, D=2048),
        norm("norm_prompt_l1p3b", "norm_fwd", B=4, T=8192, D=2048, res="f32"),
        norm("norm_grad_l125m", "norm_bwd", B=8, T=2048, D=768, kind="layer", bias=True),
    ]


def scan(name, op, B, T, D, N=16, G=1, dtype="bf16", out="bf16", h0=False, ragged=False, gate=True, softplus=True):
    return dict(name=name, op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, out=out, h0=h0, ragged=ragged, gate=gate,
                softplus=softplus)


def conv(name, op, B, T, D, K=4, dtype="bf16", out="bf16", silu=True, bias=True, state=False, ragged=False, sliced=False):
    return dict(name=name, op=op, B=B, T=T, D=D, K=K, dtype=dtype, out=out, silu=silu, bias=bias, state=state,
                ragged=ragged, sliced=sliced)


def norm(name, op, B, T, D, kind="rms", dtype="bf16", res="bf16", bias=False, gate=True, gate_first=False, ragged=False):
    return dict(name=name, op=op, B=B, T=T, D=D, kind=kind, dtype=dtype, res=res, bias=bias, gate=gate,
                gate_first=gate_first, ragged=ragged)


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_decode", "conv_fwd", "conv_bwd", "conv_decode",
                     "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    out = rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32"
    ragged = rng.random() < 0.3
    flip = lambda: rng.random() < 0.5  # noqa: E731
    D = rng.choice([_spread(rng, 1, 4096), 64 * _spread(rng, 1, 64), 8 * _spread(rng, 1, 512)])
    if op == "scan_decode" or op == "conv_decode":
        B, T = _spread(rng, 1, 512), rng.choice([1, 1, 1, 2, 5])
    else:
        B = _spread(rng, 1, 16)
        most = {"scan_fwd": 1 << 26, "scan_bwd": 1 << 24, "conv_fwd": 1 << 27, "conv_bwd": 1 << 24, "norm_fwd": 1 << 26,
                "norm_bwd": 1 << 23}[op]
        T = _spread(rng, 1, max(1, min(16384, most // (B * D))))
    if op.startswith("scan"):
        G = rng.choice([1, 1, 2, 4])
        D = -(-D // G) * G
        N = rng.choice([16, 16, 8, 32, _spread(rng, 1, 32)])
        if B * T * D * N > (1 << 30 if op == "scan_fwd" else 1 << 28):
            N = 16
        c = scan("", op, B, T, D, N, G, dtype, out, op == "scan_decode" or flip(), ragged, flip(), flip())
    elif op.startswith("conv"):
        c = conv("", op, B, T, D, rng.choice([2, 3, 4, 4]), dtype, out, flip(), flip(), op == "conv_decode" or flip(), ragged,
                 flip())
    else:
        gate = flip()
        c = norm("", op, B, T, D, rng.choice(["rms", "layer"]), dtype, rng.choice([dtype, "f32"]), flip(), gate,
                 gate and flip(), ragged)
    del c["name"]
    return c


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _made(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, T, D, op = case["B"], case["T"], case["D"], case["op"]

    def normal(*shape, std=1.0, mean=0.0, to="f32"):
        x = torch.randn(shape, generator=gen, device="cuda")
        return (x if std == 1.0 and mean == 0.0 else x * std + mean).to(TYPES[to])

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"case": case, "lens": None}
    if case["ragged"]:
        s["lens"] = torch.randint(T // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    to = case["dtype"]
    if op.startswith("scan"):
        N, G, out = case["N"], case["G"], case["out"]
        s["u"] = normal(B, T, D, to=to)
        # steps from a thousandth to a tenth, moved by the token
        step = torch.exp(uniform(D) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step)) if case["softplus"] else None
        s["dt"] = normal(B, T, D, std=0.5, to=to) if case["softplus"] else (uniform(B, T, D) * step).to(TYPES[to])
        # decays 1 to N per unit of time, a little off
        s["A"] = -(torch.arange(1, N + 1, device="cuda") * (1 + 0.1 * uniform(D, N)))
        # B and C as the projection that makes them leaves them: slices of one row
        rows = normal(B, T, G, 2 * N, to=to).transpose(1, 2)
        s["B"], s["C"] = rows[..., :N], rows[..., N:]
        s["D"] = normal(D, std=0.1, mean=1.0)
        s["z"] = normal(B, T, D, to=to) if case["gate"] else None
        s["h0"] = normal(B, D, N) if case["h0"] else None
        if op == "scan_bwd":
            s["dy"] = normal(B, T, D, to=out)
            s["dh"] = normal(B, D, N) if case["h0"] else None
    elif op.startswith("conv"):
        K = case["K"]
        s["x"] = normal(B, T, 2 * D, to=to)[..., :D] if case["sliced"] else normal(B, T, D, to=to)
        s["w"] = normal(D, K, std=K ** -0.5)
        s["bias"] = normal(D, std=0.1) if case["bias"] else None
        s["state"] = normal(B, K - 1, D, to=to) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, T, D, to=case["out"])
            s["dstate"] = normal(B, K - 1, D, to=case["out"]) if case["state"] else None
    else:
        s["x"] = normal(B, T, D, to=to)
        s["z"] = normal(B, T, D, to=to) if case["gate"] else None
        s["res"] = normal(B, T, D, std=2.0, to=case["res"])
        s["alpha"] = normal(D, std=0.05, mean=0.2)
        s["post"], s["pre"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1, mean=1.0)
        s["post_b"], s["pre_b"] = (normal(D, std=0.1), normal(D, std=0.1)) if case["bias"] else (None, None)
        if op == "norm_bwd":
            s["ds"], s["dy"] = normal(B, T, D, to=case["res"]), normal(B, T, D, to=to)
    return s


def prepare(case, seed):
    return _made(case, seed)


# ---------------------------------------------------------------- plain form --

def _live(s):
    """[B, T, 1], or None: which rows belong to their sequence."""
    c = s["case"]
    if s["lens"] is None:
        return None
    return (torch.arange(c["T"], device="cuda") < s["lens"][:, None])[..., None]


def _kept(x, live):
    return x if live is None else torch.where(live, x, 0.0)


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _doubling(a, x):
    """h_t = a_t h_{t-1} + x_t over dimension 0, in log2(T) sweeps."""
    k, T = 1, x.shape[0]
    while k < T:
        x = torch.cat([x[:k], x[k:] + a[k:] * x[:-k]])
        if 2 * k < T:
            a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return x


def _plain_scan(s):
    c = s["case"]
    B, T, D, N, G = (c[x] for x in "BTDNG")
    live = _live(s)
    u, dt = s["u"].float(), s["dt"].float()
    if s["dt_bias"] is not None:
        raw = dt + s["dt_bias"]
        dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    u, dt = _kept(u, live), _kept(dt, live)
    Bm, Cm = s["B"].float(), s["C"].float()
    if live is not None:  # rows behind the end hold anything
        Bm, Cm = torch.where(live[:, None], Bm, 0.0), torch.where(live[:, None], Cm, 0.0)
    z = None if s["z"] is None else _kept(s["z"].float(), live)
    up = None
    if c["op"] == "scan_bwd":
        up = _kept(s["dy"].float(), live)
    if c["op"] == "scan_decode":
        y, h = _plain_tokens(s, u, dt, Bm, Cm, z)
        return _kept(y, live).to(TYPES[c["out"]]), s["h0"].copy_(h)
    # as many sequences at a time as keep a state per token in a few GB
    some = max(1, (1 << 28) // (T * D * N))
    got = []
    for i in range(0, B, some):
        cut = slice(i, i + some)
        got.append(_plain_sequences(s, *(None if x is None else x[cut] for x in (u, dt, Bm, Cm, z, up, s["h0"])), s["A"], s["D"],
                                    None if up is None or s["dh"] is None else s["dh"][cut]))
    out = TYPES[c["out"]]
    if up is None:
        y, h = torch.cat([x[0] for x in got]), torch.cat([x[1] for x in got])
        return _kept(y, live).to(out), h
    du, ddt, dA, dB, dC, dD, dz, dh0 = (None if x[0] is None else torch.cat(x) for x in zip(*got))
    db = None
    if s["dt_bias"] is not None:
        ddt = _kept(ddt * _sigmoid(raw), live)
        db = ddt.sum((0, 1), dtype=torch.float64).float()
    grads = [du.to(out), ddt.to(out), dA.sum(0, dtype=torch.float64).float(), dB.to(out), dC.to(out),
             dD.sum(0, dtype=torch.float64).float()]
    return grads + [x for x in (None if dz is None else dz.to(out), db, dh0 if s["h0"] is not None else None) if x is not None]


def _plain_tokens(s, u, dt, Bm, Cm, z):
    """A few tokens from the state s["h0"]: the recurrence itself."""
    c = s["case"]
    h, ys = s["h0"], []
    share = torch.arange(c["D"], device="cuda") // (c["D"] // c["G"])
    for t in range(c["T"]):
        h = torch.exp(dt[:, t, :, None] * s["A"]) * h + (dt[:, t] * u[:, t])[..., None] * Bm[:, share, t]
        ys.append((h * Cm[:, share, t]).sum(-1) + s["D"] * u[:, t])
    y = torch.stack(ys, 1)
    return (y if z is None else y * (z * _sigmoid(z))), h


def _plain_sequences(s, u, dt, Bm, Cm, z, up, h0, A, Dv, dh):
    """Some sequences, in [T, sequence, D, N]; the parameters' gradients stay per sequence."""
    c = s["case"]
    T, D, N, G = (c[x] for x in "TDNG")
    n = u.shape[0]
    share = torch.arange(D, device="cuda") // (D // G)
    u, dt, z, up = (None if x is None else x.transpose(0, 1) for x in (u, dt, z, up))  # [T, n, D]
    a = torch.exp(dt[..., None] * A)
    Bt, Ct = Bm.permute(2, 0, 1, 3)[:, :, share], Cm.permute(2, 0, 1, 3)[:, :, share]
    x = (dt * u)[..., None] * Bt
    if h0 is not None:
        x[0] += a[0] * h0
    h = _doubling(a, x)
    del x
    y = (h * Ct).sum(-1) + Dv * u
    if up is None:
        if z is not None:
            y = y * (z * _sigmoid(z))
        return y.transpose(0, 1), h[-1].clone()
    dz = None
    if z is not None:
        sig = _sigmoid(z)
        dz = (up * y * (sig * (1 + z * (1 - sig)))).transpose(0, 1)
        up = up * (z * sig)
    dC = (up[..., None] * h).view(T, n, G, D // G, N).sum(3).permute(1, 2, 0, 3)
    g = up[..., None] * Ct
    if dh is not None:
        g[-1] += dh
    after = torch.cat([a[1:], torch.ones_like(a[:1])])
    g = _doubling(after.flip(0), g.flip(0)).flip(0)
    del after
    dB = (g * (dt * u)[..., None]).view(T, n, G, D // G, N).sum(3).permute(1, 2, 0, 3)
    dx = (g * Bt).sum(-1)
    g = g * a
    dh0 = g[0].clone()
    before = torch.zeros_like(h[:1]) if h0 is None else h0[None]
    g = g * torch.cat([before, h[:-1]])
    ddt = (g * A).sum(-1) + dx * u
    return ((dx * dt + Dv * up).transpose(0, 1), ddt.transpose(0, 1), (g * dt[..., None]).sum(0), dB, dC, (up * u).sum(0), dz, dh0)


def _plain_conv(s):
    c = s["case"]
    B, T, D, K, out = c["B"], c["T"], c["D"], c["K"], TYPES[c["out"]]
    live = _live(s)
    x = _kept(s["x"].float(), live)
    first = torch.zeros(B, K - 1, D, device="cuda") if s["state"] is None else s["state"].float()
    rows = torch.cat([first, x], 1)  # row j is the input of token j - (K - 1)
    pre = sum(s["w"][:, j] * rows[:, j:j + T] for j in range(K))
    if s["bias"] is not None:
        pre = pre + s["bias"]
    ends = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"].long()
    last = (ends[:, None] + torch.arange(K - 1, device="cuda"))[..., None].expand(B, K - 1, D)
    if c["op"] != "conv_bwd":
        y = pre * _sigmoid(pre) if c["silu"] else pre
        state = rows.gather(1, last).to(TYPES[c["dtype"]])
        if c["op"] == "conv_decode":
            state = s["state"].copy_(state)
        return _kept(y, live).to(out), state
    g = _kept(s["dy"].float(), live)
    if c["silu"]:
        sig = _sigmoid(pre)
        g = g * sig * (1 + pre * (1 - sig))
    dw = torch.stack([(g * rows[:, j:j + T]).sum((0, 1), dtype=torch.float64) for j in range(K)], 1).float()
    db = g.sum((0, 1), dtype=torch.float64).float()
    drows = torch.zeros_like(rows)
    for j in range(K):
        drows[:, j:j + T] += s["w"][:, j] * g
    if s["dstate"] is not None:
        drows.scatter_add_(1, last, s["dstate"].float())
    dx = _kept(drows[:, K - 1:], live)
    got = [dx.to(out), dw]
    if s["bias"] is not None:
        got.append(db)
    if s["state"] is not None:
        got.append(drows[:, :K - 1].to(out))
    return got


def _normed(x, gamma, beta, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    return y if beta is None else y + beta


def _plain_norm(s):
    c = s["case"]
    live = _live(s)
    kind, dt, rt = c["kind"], TYPES[c["dtype"]], TYPES[c["res"]]
    back = c["op"] == "norm_bwd"
    names = [n for n in ("x", "z", "res", "alpha", "post", "post_b", "pre", "pre_b") if s[n] is not None]
    v = dict.fromkeys(("z", "post_b", "pre_b"))
    for n in names:
        t = s[n].float()
        if n in ("x", "z", "res"):
            t = _kept(t, live)
        v[n] = t.detach().clone().requires_grad_() if back else t
    o = v["x"]
    gate = None if v["z"] is None else v["z"] * _sigmoid(v["z"])
    if gate is not None and c["gate_first"]:
        o = o * gate
    o = _normed(o, v["post"], v["post_b"], kind)
    if gate is not None and not c["gate_first"]:
        o = o * gate
    r = v["res"] + v["alpha"] * o
    y = _normed(r, v["pre"], v["pre_b"], kind)
    if not back:
        return _kept(r, live).to(rt), _kept(y, live).to(dt)
    ups = [_kept(s["ds"].float(), live), _kept(s["dy"].float(), live)]
    got = torch.autograd.grad([r, y], [v[n] for n in names], ups)
    types = {"x": dt, "z": dt, "res": rt}
    return [_kept(g, live).to(types[n]) if n in types else g for n, g in zip(names, got)]


def _plain(s):
    op = s["case"]["op"]
    return (_plain_scan if op.startswith("scan") else _plain_conv if op.startswith("conv") else _plain_norm)(s)


# ------------------------------------------------------------ the operators --

def _framework(s):
    import test_sequence_layer_amd as ttt

    c = s["case"]
    op, lens = c["op"], s["lens"]
    if op.startswith("scan"):
        args = s["u"], s["dt"], s["A"], s["B"], s["C"]
        more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=c["softplus"], lens=lens)
        if op == "scan_fwd":
            return ttt.selective_scan_fwd(*args, h0=s["h0"], out_dtype=TYPES[c["out"]], **more)
        if op == "scan_decode":
            return ttt.selective_scan_decode(*args, s["h0"], out_dtype=TYPES[c["out"]], **more), s["h0"]
        du, ddt, dA, dB, dC, dD, dz, db, dh0 = ttt.selective_scan_bwd(*args, s["dy"], h0=s["h0"], dh_final=s["dh"], **more)
        got = [du, ddt, dA, dB, dC, dD] + ([dz] if c["gate"] else []) + ([db] if s["dt_bias"] is not None else [])
        return got + ([dh0] if s["h0"] is not None else [])
    if op.startswith("conv"):
        more = dict(bias=s["bias"], silu=c["silu"], lens=lens)
        if op == "conv_fwd":
            return ttt.short_conv_fwd(s["x"], s["w"], state=s["state"], out_dtype=TYPES[c["out"]], **more)
        if op == "conv_decode":
            return ttt.short_conv_decode(s["x"], s["w"], s["state"], out_dtype=TYPES[c["out"]], **more), s["state"]
        dx, dw, db, dstate = ttt.short_conv_bwd(s["x"], s["w"], s["dy"], state=s["state"], dstate_final=s["dstate"], **more)
        return [dx, dw] + ([db] if s["bias"] is not None else []) + ([dstate] if s["state"] is not None else [])
    args = dict(res=s["res"], z=s["z"], alpha=s["alpha"], gamma_post=s["post"], beta_post=s["post_b"], gamma_pre=s["pre"],
                beta_pre=s["pre_b"], kind=c["kind"], eps=EPS, gate_first=c["gate_first"], lens=lens)
    if op == "norm_fwd":
        return ttt.block_norm_fwd(s["x"], **args)
    got = ttt.block_norm_bwd(s["x"], s["ds"], s["dy"], **args)
    return [g for g in got if g is not None]


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    B, T, D, op = case["B"], case["T"], case["D"], case["op"]
    size = {"bf16": 2, "f32": 4}
    i = size[case["dtype"]]
    live = 0.75 if case["ragged"] else 1.0  # half to all of a padded row is tokens
    n = B * T * D
    if op.startswith("scan"):
        o, N, G = size[case["out"]], case["N"], case["G"]
        state = 4 * B * D * N
        rows = (3 if case["gate"] else 2) * n * i * live + 2 * B * G * T * N * i * live
        params = 4 * D * (N + 1 + case["softplus"])
        if op != "scan_bwd":
            return {"bytes": rows + params + n * o + state * (2 if case["h0"] else 1), "flops": 7 * n * live * N}
        grads = n * o * live + (3 if case["gate"] else 2) * n * o + 2 * B * G * T * N * o
        return {"bytes": rows + 2 * params + grads + (3 * state if case["h0"] else 0), "flops": 22 * n * live * N}
    if op.startswith("conv"):
        o, K = size[case["out"]], case["K"]
        params, state = 4 * D * (K + case["bias"]), B * (K - 1) * D
        if op != "conv_bwd":
            return {"bytes": n * i * live + n * o + params + state * i * (2 if case["state"] else 1), "flops": 2 * K * n * live}
        return {"bytes": n * i * live + n * o * live + n * o + 2 * params + (state * (i + 2 * o) if case["state"] else 0),
                "flops": 6 * K * n * live}
    r = size[case["res"]]
    rows = (2 if case["gate"] else 1) * n * i
    params = 4 * D * (5 if case["bias"] else 3)
    if op == "norm_fwd":
        return {"bytes": rows * live + n * r * live + n * (r + i) + params, "flops": 16 * n * live}
    return {"bytes": rows * (1 + live) + n * r * (1 + 2 * live) + n * i * live + 2 * params, "flops": 40 * n * live}


# ------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    s = _made(case, seed)
    op = case["op"]
    return (_exact_scan if op.startswith("scan") else _exact_conv if op.startswith("conv") else _exact_norm)(s)


def _exact_scan(s):
    """Token by token from the recurrence itself."""
    c = s["case"]
    B, T, D, N, G = (c[x] for x in "BTDNG")
    u, raw, A, Dv = s["u"].double(), s["dt"].double(), s["A"].double(), s["D"].double()
    # log(1 + e^x), and its slope
    dt, slope = raw, None
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"].double()
        dt, slope = torch.logaddexp(raw, torch.zeros_like(raw)), torch.exp(-torch.logaddexp(-raw, torch.zeros_like(raw)))
    each = D // G
    Bm, Cm = (s[n].double().permute(2, 0, 1, 3).repeat_interleave(each, 2) for n in "BC")  # [T, B, D, N]
    live = None
    if s["lens"] is not None:
        live = torch.arange(T, device="cuda")[:, None] < s["lens"]  # [T, B]
    h = torch.zeros(B, D, N, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    y = torch.zeros(B, T, D, dtype=torch.float64, device="cuda")
    back = c["op"] == "scan_bwd"
    hs = [h]
    for t in range(T):
        new = h * torch.exp(dt[:, t, :, None] * A) + (dt[:, t] * u[:, t])[..., None] * Bm[t]
        h = new if live is None else torch.where(live[t][:, None, None], new, h)
        if back:
            hs.append(h)
        y[:, t] = (h * Cm[t]).sum(-1)
    y = y + Dv * u
    gate = None
    if s["z"] is not None:
        z = s["z"].double()
        gate = z / (1 + torch.exp(-z))
    if not back:
        y = y if gate is None else y * gate
        return y if live is None else torch.where(live.T[..., None], y, 0.0), h
    up = s["dy"].double()
    if live is not None:
        up = torch.where(live.T[..., None], up, 0.0)
    dz = None
    if gate is not None:
        sig = 1 / (1 + torch.exp(-z))
        dz = up * y * (sig + gate * (1 - sig))
        up = up * gate
    du, ddt = up * Dv, torch.zeros_like(u)
    dA = torch.zeros(D, N, dtype=torch.float64, device="cuda")
    dB, dC = (torch.zeros(T, B, G, N, dtype=torch.float64, device="cuda") for _ in range(2))
    g = torch.zeros_like(h) if s["dh"] is None else s["dh"].double()
    for t in reversed(range(T)):
        a = torch.exp(dt[:, t, :, None] * A)
        on = 1.0 if live is None else live[t].double()[:, None, None]
        g = g + up[:, t, :, None] * Cm[t] * on
        m = g * on
        dC[t] = (hs[t + 1] * up[:, t, :, None]).view(B, G, each, N).sum(2)
        dB[t] = (m * (dt[:, t] * u[:, t])[..., None]).view(B, G, each, N).sum(2)
        x = (m * Bm[t]).sum(-1)
        q = m * a * hs[t]
        du[:, t] += x * dt[:, t]
        ddt[:, t] = x * u[:, t] + (q * A).sum(-1)
        dA += (q * dt[:, t, :, None]).sum(0)
        g = g * a if live is None else torch.where(live[t][:, None, None], g * a, g)
    got = [du, ddt if slope is None else ddt * slope, dA, dB.permute(1, 2, 0, 3), dC.permute(1, 2, 0, 3), (up * u).sum((0, 1))]
    if dz is not None:
        got.append(dz)
    if slope is not None:
        got.append((ddt * slope).sum((0, 1)))
    return got + ([g] if s["h0"] is not None else [])


def _exact_conv(s):
    """Token by token from the window of its last inputs; gradients by differentiating that."""
    c = s["case"]
    B, T, D, K = (c[x] for x in "BTDK")
    back = c["op"] == "conv_bwd"
    leaf = lambda x: x.double().clone().requires_grad_(back)  # noqa: E731
    x, w = leaf(s["x"]), leaf(s["w"])
    bias = None if s["bias"] is None else leaf(s["bias"])
    state = None if s["state"] is None else leaf(s["state"])
    ends = [T] * B if s["lens"] is None else s["lens"].tolist()
    ys, lasts = [], []
    for b in range(B):
        first = x.new_zeros(K - 1, D) if state is None else state[b]
        rows = torch.cat([first, x[b, :ends[b]]])
        windows = rows.unfold(0, K, 1)[:ends[b]] if ends[b] else x.new_zeros(0, D, K)  # [tokens, D, K]
        pre = (windows * w).sum(-1)
        if bias is not None:
            pre = pre + bias
        y = pre / (1 + torch.exp(-pre)) if c["silu"] else pre
        ys.append(torch.cat([y, y.new_zeros(T - ends[b], D)]))
        lasts.append(rows[ends[b]:])
    y, last = torch.stack(ys), torch.stack(lasts)
    if not back:
        return y, last
    leaves = [x, w] + [t for t in (bias, state) if t is not None]
    outs, ups = [y], [s["dy"].double()]
    if s["dstate"] is not None:
        outs, ups = outs + [last], ups + [s["dstate"].double()]
    return list(torch.autograd.grad(outs, leaves, ups, materialize_grads=True))


def _exact_norm(s):
    """Forward from the mean and the variance; gradients by the norm's own formula, back to front."""
    c = s["case"]
    layer = c["kind"] == "layer"
    d = {k: None if s.get(k) is None else s[k].double()
         for k in ("x", "z", "res", "alpha", "post", "post_b", "pre", "pre_b", "ds", "dy")}
    live = None
    if s["lens"] is not None:
        live = (torch.arange(c["T"], device="cuda") < s["lens"][:, None])[..., None].double()
        for k in ("x", "z", "res", "ds", "dy"):
            d[k] = None if d[k] is None else d[k] * live

    def forward(x, gamma, beta):
        mean = x.mean(-1, keepdim=True) if layer else 0.0
        unit = (x - mean) * torch.rsqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
        return unit, unit * gamma + (0.0 if beta is None else beta)

    def back(x, unit, gamma, g):
        mean = x.mean(-1, keepdim=True) if layer else 0.0
        inv = torch.rsqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
        h = g * gamma
        dx = h - unit * (h * unit).mean(-1, keepdim=True)
        if layer:
            dx = dx - h.mean(-1, keepdim=True)
        return dx * inv

    x, gate = d["x"], None
    if d["z"] is not None:
        sig = torch.sigmoid(d["z"])
        gate = d["z"] * sig
    first = gate is not None and c["gate_first"]
    o = x * gate if first else x
    unit1, n1 = forward(o, d["post"], d["post_b"])
    v = n1 * gate if gate is not None and not first else n1
    r = d["res"] + d["alpha"] * v
    unit2, y = forward(r, d["pre"], d["pre_b"])
    if c["op"] == "norm_fwd":
        return (r, y) if live is None else (r * live, y * live)
    rows = (0, 1)
    dr = d["ds"] + back(r, unit2, d["pre"], d["dy"])
    dv = dr * d["alpha"]
    dgate = None
    dn = dv
    if gate is not None and not first:
        dn, dgate = dv * gate, dv * n1
    do = back(o, unit1, d["post"], dn)
    dx = do
    if first:
        dx, dgate = do * gate, do * x
    got = [dx]
    if gate is not None:
        got.append(dgate * (sig + gate * (1 - sig)))
    got += [dr, (dr * v).sum(rows), (dn * unit1).sum(rows)]
    if d["post_b"] is not None:
        got.append(dn.sum(rows))
    got.append((d["dy"] * unit2).sum(rows))
    if d["pre_b"] is not None:
        got.append(d["dy"].sum(rows))
    return got
