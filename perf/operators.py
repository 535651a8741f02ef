"""What the linear-attention and rotary-position operators are measured on.

Linear attention with a decay lambda_h = exp(log_decay_h) per head: the state is
W_t = lambda W_{t-1} + v_t k_t^T and the output z_t = scale W_t q_t, with the
state laid out as the TTT layer's (z = W q).  Rotary positions turn the pairs of
q and k by position * frequency.  ``run`` computes both in elementary torch
operations, or through the package where ``own`` is true.
"""
import math

import torch

own = False

CHUNK = 64  # tokens per block of the plain form


def listed():
    return [
        # one short user prompt at the 125M layer's heads: every launch and its latency shows
        attn("prompt_short", "fwd", B=1, H=12, T=67, d=64),
        # the 125M layer's prompt batch, fp32 outputs, continuing from one learned initial state
        attn("prompt_l125m", "fwd", B=8, H=12, T=2048, d=64, out="f32", w0="shared"),
        # the 1.3B layer at its full length, q, k, v as the projections leave them ([B, T, H, d])
        attn("prompt_l1p3b", "fwd", B=16, H=32, T=8192, d=64, layout="bthd"),
        # two long documents: few chains, many tokens
        attn("prompt_long", "fwd", B=2, H=32, T=32768, d=64),
        # a padded fp32 batch of odd length, wide heads, shared key/value heads, every sequence with a state of its own
        attn("prompt_ragged_f32", "fwd", B=3, H=10, kv=5, T=1009, d=128, dtype="f32", out="f32", w0="each", ragged=True),
        # training steps: the 125M layer, a padded fp32 batch with shared key/value heads, the 1.3B layer at 2048 tokens
        attn("grad_l125m", "bwd", B=8, H=12, T=2048, d=64, w0="shared"),
        attn("grad_ragged_f32", "bwd", B=3, H=6, kv=2, T=531, d=32, dtype="f32", out="f32", w0="each", ragged=True),
        attn("grad_l1p3b_2k", "bwd", B=16, H=32, T=2048, d=64, layout="bthd"),
        # one token for each of 16 and 512 running sequences, q and k rotated on the way
        attn("token_16x32", "decode", B=16, H=32, T=1, d=64, w0="each", rope="half", start=8192),
        attn("token_512x32", "decode", B=512, H=32, T=1, d=64, w0="each", rope="half", start=32768),
        # q and k of two long documents, frequencies stretched for the length
        rope("rotary_long", "rotary", B=2, H=32, kv=32, T=32768, d=64, rot=64, pairs="half", scaling="yarn", start=0),
        # the gradient through a rotation of half the head, fp32, far positions
        rope("rotary_grad", "rotary_bwd", B=8, H=12, kv=4, T=2047, d=64, rot=32, pairs="interleaved", dtype="f32",
             scaling="linear", start=1_000_003),
    ]


def attn(name, kind, B, H, T, d, kv=0, dtype="bf16", out="bf16", w0="none", layout="bhtd", ragged=False, rope="none",
         start=0):
    return dict(name=name, kind=kind, B=B, H=H, kv=kv or H, T=T, d=d, dtype=dtype, out=out, w0=w0, layout=layout,
                ragged=ragged, rope=rope, start=start)


def rope(name, kind, B, H, kv, T, d, rot, pairs, scaling, start, dtype="bf16", layout="bhtd"):
    return dict(name=name, kind=kind, B=B, H=H, kv=kv, T=T, d=d, rot=rot, pairs=pairs, dtype=dtype, scaling=scaling,
                start=start, layout=layout)


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "rotary", "rotary_bwd"])
    d = rng.choice([16, 32, 64, 64, 128])
    group = rng.choice([1, 1, 1, 2, 4])
    kv = _spread(rng, 1, 32 // group)
    H = kv * group
    if kind.startswith("rotary"):
        B = _spread(rng, 1, 16)
        T = _spread(rng, 1, max(1, min(32768, (1 << 27) // (B * H * d))))
        c = rope("", kind, B, H, kv, T, d, rot=rng.choice([d, d, d // 2, d - 2]), pairs=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), start=_spread(rng, 1, 1 << 20) - 1,
                 dtype=rng.choice(["bf16", "f32"]), layout=rng.choice(["bhtd", "bthd"]))
    elif kind == "decode":
        B = _spread(rng, 1, max(1, min(512, (1 << 25) // (H * d * d))))
        c = attn("", kind, B, H, rng.choice([1, 1, 1, 2, 5]), d, kv, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                 "each", ragged=rng.random() < 0.3, rope=rng.choice(["none", "half", "interleaved"]),
                 start=_spread(rng, 1, 1 << 18) - 1)
    else:
        B = _spread(rng, 1, 16)
        most = (1 << 26) if kind == "fwd" else (1 << 25)
        T = _spread(rng, 1, max(1, min(32768, most // (B * H * d))))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = attn("", kind, B, H, T, d, kv, dtype, rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32",
                 rng.choice(["none", "shared", "each"]), rng.choice(["bhtd", "bthd"]), rng.random() < 0.3)
    del c["name"]
    return c


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _made(case, seed):
    """The inputs of a case in fp32 and their storage types, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, kv, T, d = (case[x] for x in ("B", "H", "kv", "T", "d"))

    def normal(*shape, std, to):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(TYPES[to])

    def rows(heads, std, to):
        if case["layout"] == "bthd":
            return normal(B, T, heads, d, std=std, to=to).transpose(1, 2)
        return normal(B, heads, T, d, std=std, to=to)

    s = {"case": case}
    unit = d ** -0.5  # views of about unit length
    if case["kind"].startswith("rotary"):
        s["q"], s["k"] = rows(H, unit, case["dtype"]), rows(kv, unit, case["dtype"])
        # every sequence begins somewhere of its own
        s["pos"] = case["start"] + torch.randint(0, 64, (B,), generator=gen, device="cuda")
        s["freqs"], s["mscale"] = _freqs(case["rot"], case["scaling"])
        return s
    s["q"], s["k"], s["v"] = rows(H, unit, case["dtype"]), rows(kv, unit, case["dtype"]), rows(kv, unit, case["dtype"])
    # decays from half a token to a thousand tokens, a little off a fixed ladder
    ladder = 1 + 9 * (torch.arange(H, device="cuda") + torch.rand(H, generator=gen, device="cuda")) / H
    s["log_decay"] = -torch.exp2(-ladder)
    if case["w0"] == "none":
        s["w0"] = None
    else:
        s["w0"] = normal(*([B] if case["w0"] == "each" else []), H, d, d, std=0.02 if case["w0"] == "shared" else 0.2, to="f32")
    s["lens"] = None
    if case["ragged"]:
        s["lens"] = torch.randint(T // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["scale"] = 1.0
    if case["kind"] == "bwd":
        s["dz"] = rows(H, 1.0, case["out"])
        s["dw_final"] = normal(B, H, d, d, std=1.0, to="f32") if case["w0"] == "each" else None
    s["rope"] = None
    if case["rope"] != "none":
        freqs, mscale = _freqs(d, "none")
        pos = case["start"] + torch.randint(0, 64, (B,), generator=gen, device="cuda")
        s["rope"] = (pos, freqs, case["rope"], mscale)
    return s


def prepare(case, seed):
    return _made(case, seed)


def _freqs(rot, scaling, base=10000.0, factor=8.0, original=4096):
    """Radians per position of each pair (fp64) and the factor on the rotated values: plain, positions divided by
    ``factor``, the base raised for it, or (YaRN) the two blended by how often a pair turns within ``original``."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / rot)
    if scaling in ("none", "ntk"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    turns = original * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------- plain form --

def _angles(pos, freqs, T):
    p = pos.to(torch.float64)[:, None] + torch.arange(T, dtype=torch.float64, device=pos.device)
    return p[:, None, :, None] * freqs  # [B, 1, T, rot / 2]


def _turned(x, cos, sin, pairs):
    half = cos.shape[-1]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if pairs == "half":
        a, b = head[..., :half], head[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _plain_rotary(x, pos, freqs, pairs, mscale, back=False):
    t = _angles(pos, freqs, x.shape[2])
    cos, sin = (torch.cos(t) * mscale).float(), (torch.sin(-t if back else t) * mscale).float()
    return _turned(x.float(), cos, sin, pairs)


def _plain_attn(q, k, v, g, w0, lens, scale):
    """z and the last state, [B, H, T, d] fp32 each with as many heads, g [B, H] log decays."""
    B, H, T, d = q.shape
    dev = q.device
    t = torch.arange(T, device=dev)
    left = lens.to(torch.float32)[:, None, None] - 1 - t if lens is not None else (T - 1 - t).float().expand(B, 1, T)
    if lens is not None:
        here = (left >= 0)[..., None]
        q, k, v = (torch.where(here, x, 0.0) for x in (q, k, v))
    size = min(CHUNK, T)
    n = -(-T // size)
    pad = n * size - T
    qc, kc, vc = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, size, d) for x in (q, k, v))
    i = torch.arange(size, device=dev, dtype=torch.float32)
    c = torch.arange(n + 1, device=dev, dtype=torch.float32)
    gap = i[:, None] - i
    decay = torch.where(gap >= 0, torch.exp(g[..., None, None] * gap.clamp(min=0)), 0.0)
    z = (torch.matmul(qc, kc.transpose(-1, -2)) * decay[:, :, None]) @ vc
    # each block's own state, then the states at block starts
    own_state = torch.matmul((vc * torch.exp(g[..., None] * (size - 1 - i))[:, :, None, :, None]).transpose(-1, -2), kc)
    blocks = c[:, None] - 1 - c[:n]
    carry = torch.where(blocks >= 0, torch.exp(g[..., None, None] * size * blocks.clamp(min=0)), 0.0)
    starts = torch.matmul(carry[:, :, :n], own_state.view(B, H, n, d * d)).view(B, H, n, d, d)
    if w0 is not None:
        starts = starts + torch.exp(g[..., None] * size * c[:n])[..., None, None] * w0[:, :, None]
    z = z + torch.exp(g[..., None] * (i + 1))[:, :, None, :, None] * torch.matmul(qc, starts.transpose(-1, -2))
    z = z.reshape(B, H, n * size, d)[:, :, :T] * scale
    last = torch.exp(g[..., None] * left.clamp(min=0))
    w = torch.matmul((v * last[..., None]).transpose(-1, -2), k)
    if w0 is not None:
        w = w + torch.exp(g * (left[:, :, 0] + 1))[..., None, None] * w0
    return z, w


def _plain_token(q, k, v, g, w0, lens, scale):
    """_plain_attn for one token, as the recurrence itself."""
    w = torch.exp(g)[..., None, None] * w0 + v.transpose(-1, -2) * k
    z = torch.matmul(q, w.transpose(-1, -2)) * scale
    if lens is not None:
        live = (lens > 0)[:, None, None, None]
        z, w = torch.where(live, z, 0.0), torch.where(live, w, w0)
    return z, w


def _wide(s):
    c = s["case"]
    group = c["H"] // c["kv"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    g = s["log_decay"].expand(c["B"], c["H"])
    w0 = None if s["w0"] is None else s["w0"].expand(c["B"], c["H"], c["d"], c["d"])
    return q, k, v, g, w0, group


def _plain(s):
    c = s["case"]
    if c["kind"].startswith("rotary"):
        back = c["kind"] == "rotary_bwd"
        return [_plain_rotary(s[x], s["pos"], s["freqs"], c["pairs"], s["mscale"], back).to(TYPES[c["dtype"]]) for x in "qk"]
    q, k, v, g, w0, group = _wide(s)
    out = TYPES[c["out"]]
    if c["kind"] == "decode":
        if s["rope"] is not None:
            pos, freqs, pairs, mscale = s["rope"]
            q, k = _plain_rotary(q, pos, freqs, pairs, mscale), _plain_rotary(k, pos, freqs, pairs, mscale)
    if c["kind"] != "bwd":
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        step = _plain_token if c["kind"] == "decode" and c["T"] == 1 else _plain_attn
        z, w = step(q, k, v, g, w0, s["lens"], s["scale"])
        if c["kind"] == "decode":
            w = s["w0"].copy_(w)
        return z.to(out), w
    leaves = [q, k, v, g] + ([w0] if w0 is not None else [])
    leaves = [x.detach().clone().requires_grad_() for x in leaves]
    q, k, v, g = leaves[:4]
    z, w = _plain_attn(q, k.repeat_interleave(group, 1), v.repeat_interleave(group, 1), g, leaves[4] if w0 is not None else None,
                       s["lens"], s["scale"])
    ends, up = [z], [s["dz"].float()]
    if s["dw_final"] is not None:
        ends, up = ends + [w], up + [s["dw_final"]]
    got = torch.autograd.grad(ends, leaves, up)
    return [x.to(out) for x in got[:3]] + list(got[3:])


# ------------------------------------------------------------ the operators --

def _framework(s):
    import test_sequence_layer_amd as ttt

    c = s["case"]
    if c["kind"] == "rotary":
        return list(ttt.rotary(s["q"], s["k"], s["pos"], s["freqs"], layout=c["pairs"], scale=s["mscale"]))
    if c["kind"] == "rotary_bwd":
        return list(ttt.rotary_bwd(s["q"], s["k"], s["pos"], s["freqs"], layout=c["pairs"], scale=s["mscale"]))
    out = TYPES[c["out"]]
    if c["kind"] == "fwd":
        return ttt.linear_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], w0=s["w0"], scale=s["scale"], lens=s["lens"],
                                   out_dtype=out)
    if c["kind"] == "decode":
        z = ttt.linear_attn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["w0"], scale=s["scale"], lens=s["lens"],
                                   rope=s["rope"], out_dtype=out)
        return z, s["w0"]
    got = ttt.linear_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["dz"], w0=s["w0"], dw_final=s["dw_final"],
                              scale=s["scale"], lens=s["lens"])
    return list(got if s["w0"] is not None else got[:4])


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    B, H, kv, T, d = (case[x] for x in ("B", "H", "kv", "T", "d"))
    size = {"bf16": 2, "f32": 4}
    if case["kind"].startswith("rotary"):
        n = B * (H + kv) * T * d
        return {"bytes": 2 * n * size[case["dtype"]] + 8 * B + 4 * case["rot"], "flops": 3 * n}
    live = 0.75 if case["ragged"] else 1.0  # half to all of a padded row is tokens
    rows_in = B * (H + 2 * kv) * T * d * size[case["dtype"]] * live
    state = 4 * d * d * H
    start = 0 if case["w0"] == "none" else state * (B if case["w0"] == "each" else 1)
    if case["kind"] != "bwd":
        return {"bytes": rows_in + B * H * T * d * size[case["out"]] + start + B * state, "flops": 4 * B * H * T * live * d * d}
    grads = B * (H * live + H + 2 * kv) * T * d * size[case["out"]]  # dz read, dq, dk, dv written
    ends = (B * state if case["w0"] == "each" else 0) + (B * state if case["w0"] != "none" else 0)
    return {"bytes": rows_in + grads + start + ends + 4 * B * H, "flops": 10 * B * H * T * live * d * d}


# ------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    """Token by token from the recurrence itself, in 64 bits."""
    s = _made(case, seed)
    if case["kind"].startswith("rotary"):
        sign = -1.0 if case["kind"] == "rotary_bwd" else 1.0
        return [_exact_turn(s[x].double(), s["pos"], s["freqs"], case["pairs"], s["mscale"], sign) for x in "qk"]
    B, H, T, d = (case[x] for x in ("B", "H", "T", "d"))
    share = torch.arange(H, device="cuda") // (H // case["kv"])
    q, k, v = s["q"].double(), s["k"].double()[:, share], s["v"].double()[:, share]
    if s["rope"] is not None:
        pos, freqs, pairs, mscale = s["rope"]
        q, k = (_exact_turn(x, pos, freqs, pairs, mscale, 1.0) for x in (q, k))
    lam = torch.exp(s["log_decay"].double())[None, :, None, None]
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    live = (torch.arange(T, device="cuda")[:, None] < lens)[..., None, None, None]  # [T, B, 1, 1, 1]
    W = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda")
    if s["w0"] is not None:
        W = W + s["w0"].double()
    scale = s["scale"]
    if case["kind"] != "bwd":
        z = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
        for t in range(T):
            new = W * lam + v[:, :, t, :, None] * k[:, :, t, None, :]
            W = torch.where(live[t], new, W) if case["ragged"] else new
            z[:, :, t] = scale * torch.matmul(W, q[:, :, t, :, None])[..., 0] * live[t][..., 0]
        return z, W
    dz = s["dz"].double() * scale * live[..., 0, 0].permute(1, 2, 0)[..., None]
    dq, dk, dv = (torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda") for _ in range(3))
    U = torch.zeros_like(W)  # dW / d log_decay
    dg = torch.zeros(B, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        newU = lam * (U + W)
        new = W * lam + v[:, :, t, :, None] * k[:, :, t, None, :]
        U, W = (torch.where(live[t], newU, U), torch.where(live[t], new, W)) if case["ragged"] else (newU, new)
        dq[:, :, t] = torch.matmul(dz[:, :, t, None, :], W)[:, :, 0]
        dg += torch.matmul(dz[:, :, t, None, :], torch.matmul(U, q[:, :, t, :, None]))[..., 0, 0]
    G = torch.zeros_like(W) if s["dw_final"] is None else s["dw_final"].double().clone()
    dg += (G * U).sum((-1, -2))
    for t in reversed(range(T)):  # G: the gradient of the state after token t
        G = G + dz[:, :, t, :, None] * q[:, :, t, None, :]
        dk[:, :, t] = torch.matmul(v[:, :, t, None, :], G)[:, :, 0] * live[t][..., 0]
        dv[:, :, t] = torch.matmul(G, k[:, :, t, :, None])[..., 0] * live[t][..., 0]
        G = torch.where(live[t], lam * G, G) if case["ragged"] else lam * G
    dk, dv = (x.view(B, case["kv"], -1, T, d).sum(2) for x in (dk, dv))
    return [dq, dk, dv, dg] + ([G] if s["w0"] is not None else [])


def _exact_turn(x, pos, freqs, pairs, mscale, sign):
    """Each pair as a complex number times e^(i angle)."""
    half, T = freqs.shape[0], x.shape[2]
    at = pos[:, None] + torch.arange(T, device="cuda")
    turn = torch.polar(torch.full((x.shape[0], 1, T, half), float(mscale), dtype=torch.float64, device="cuda"),
                       sign * at[:, None, :, None].double() * freqs)
    y = x.clone()
    first, second = (slice(0, half), slice(half, 2 * half)) if pairs == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    got = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = got.real, got.imag
    return y
