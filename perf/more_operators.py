"""Cases of the operators that complete a block around the recurrences: the
gated linear recurrence (one decay per channel), the norm and rotation of
queries and keys, and the gated feed-forward product.

Each case is one pass through one entry point. ``run`` computes it either in
its plain form (elementary torch operations in fp32, rounded once at the end;
in fp64 where fp32 loses what matters, in the decays, which lie close to one and
act over thousands of tokens, and in the angles of far positions) or, with ``own`` true, through the package's entry points;
``exact`` is the definition once more in fp64, token by token.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_INTERVAL = 16      # tokens between the states that a forward leaves for its backward


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _glr(name, op, B, T, C, dtype, gate=True, normalize=True, lens=False,
         state=False, states=False, extra=0):
    return dict(name=name, op=op, B=B, T=T, C=C, dtype=dtype, gate=gate,
                normalize=normalize, lens=lens, state=state, states=states,
                extra=extra)


def _qk(name, op, B, T, Hq, Hk, D, rot, dtype, norm="rms", weight=True,
        interleaved=False, lens=False, far=False, wide_dy=False):
    return dict(name=name, op=op, B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot,
                dtype=dtype, norm=norm, weight=weight, interleaved=interleaved,
                lens=lens, far=far, wide_dy=wide_dy)


def _ffn(name, op, R, C, F, dtype, act="silu", save=False, extra=0):
    return dict(name=name, op=op, R=R, C=C, F=F, dtype=dtype, act=act, save=save,
                extra=extra)


def listed():
    return [
        # a training batch at the width of a 1.3B layer's values, its states
        # left for the backward pass
        _glr("recurrence prompt", "glr_forward", 4, 4096, 4096, "bf16",
             states=True, extra=64),
        # a padded batch of prompts continued from states, an odd width
        _glr("recurrence ragged fp32", "glr_forward", 3, 1000, 1021, "f32",
             lens=True, state=True),
        # a serving step of 128 sequences, one token each
        _glr("recurrence decode", "glr_decode", 128, 1, 4096, "bf16", state=True),
        # the gradients of a training batch, from the forward's states
        _glr("recurrence backward", "glr_backward", 4, 4096, 4096, "bf16",
             states=True),
        # the gradients of one long sequence, which forms the states itself
        _glr("recurrence backward long", "glr_backward", 1, 9001, 1536, "f32",
             state=True),
        # queries and keys of a 1.3B layer out of one projection
        _qk("rotary prompt", "qk_rotary_forward", 4, 4096, 16, 16, 128, 128,
            "bf16"),
        # one token of 64 sequences far into their contexts, shared keys
        _qk("rotary decode", "qk_rotary_forward", 64, 1, 16, 2, 64, 32, "bf16",
            norm="l2", weight=False, interleaved=True, far=True),
        # the gradients of a training batch, adjoints in fp32 as the delta
        # rule's backward returns them
        _qk("rotary backward", "qk_rotary_backward", 8, 2048, 16, 4, 128, 64,
            "bf16", wide_dy=True),
        # the feed-forward part of a training batch, products kept
        _ffn("feed-forward prompt", "gated_ffn_forward", 8192, 2048, 5632,
             "bf16", save=True),
        # a serving step of 8 sequences: the weights are what is read
        _ffn("feed-forward decode", "gated_ffn_forward", 8, 2048, 5632, "bf16"),
        # the gradients of a training batch
        _ffn("feed-forward backward", "gated_ffn_backward", 8192, 2048, 5632,
             "bf16"),
        # a small fp32 model, odd sizes
        _ffn("feed-forward backward fp32", "gated_ffn_backward", 333, 509, 1366,
             "f32", act="gelu"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_forward", "glr_forward", "glr_decode", "glr_backward",
                     "glr_backward", "qk_rotary_forward", "qk_rotary_forward",
                     "qk_rotary_backward", "gated_ffn_forward",
                     "gated_ffn_forward", "gated_ffn_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("glr"):
        C = rng.choice([_spread(rng, 32, 4096), 64 * _spread(rng, 1, 64)])
        c = _glr("", op, 1, 1, C, dtype, gate=rng.random() < 0.8,
                 normalize=rng.random() < 0.8, lens=rng.random() < 0.4,
                 state=rng.random() < 0.5, states=rng.random() < 0.5,
                 extra=rng.choice([0, 0, 8, 5, 256]))
        if op == "glr_decode":
            c.update(B=_spread(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 5]),
                     lens=False, state=True, states=False)
        else:
            c["T"] = _spread(rng, 1, 9001)
            c["B"] = rng.randint(1, max(1, min(8, (1 << 25) // (C * c["T"]))))
    elif op.startswith("qk"):
        D = rng.choice([32, 64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        c = _qk("", op, rng.randint(1, 4), _spread(rng, 1, 4096),
                Hk * rng.choice([1, 1, 2, 4]), Hk, D,
                rng.choice([D, D, D // 2, 16, 0]), dtype,
                norm=rng.choice(["rms", "rms", "l2", "none"]),
                weight=rng.random() < 0.7, interleaved=rng.random() < 0.4,
                lens=rng.random() < 0.3, far=rng.random() < 0.4,
                wide_dy=op == "qk_rotary_backward" and rng.random() < 0.5)
        if rng.random() < 0.25:  # a serving step
            c.update(B=_spread(rng, 1, 256), T=1, lens=False, far=True)
    else:
        C, F = _spread(rng, 64, 4096), _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            C, F = 64 * max(1, C // 64), 64 * max(1, F // 64)
        most = (8192 * 2048 * 5632) >> (0 if dtype == "bf16" else 3)
        R = _spread(rng, 1, max(1, min(8192, most // (C * F))))
        c = _ffn("", op, R, C, F, dtype, act=rng.choice(["silu", "silu", "gelu",
                                                         "gelu_tanh"]),
                 save=op == "gated_ffn_forward" and rng.random() < 0.5,
                 extra=rng.choice([0, 0, 8, 3]))
    c.pop("name")
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(c, g):
    """Prompt lengths of a padded batch: the first full, the others between
    nothing and everything."""
    u = torch.rand((c["B"],), generator=g, device="cuda")
    n = (u * (c["T"] + 1)).floor().clamp(max=c["T"]).to(torch.int32)
    n[0] = c["T"]
    return n


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = c["op"], _DT[c["dtype"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=c)
    if op.startswith("glr"):
        B, T, C = c["B"], c["T"], c["C"]
        # x and both gates are channel ranges of one projection; decays at an
        # open gate between exp(-1/1000) and exp(-2) a token
        wide = normal(B, T, 3 * C + c["extra"], dtype=dt)
        s.update(x=wide[:, :, :C], r=wide[:, :, C:2 * C],
                 i=wide[:, :, 2 * C:3 * C] if c["gate"] else None,
                 A=-torch.exp(uniform(math.log(1e-3), math.log(2.0), C)),
                 h0=normal(B, C) if c["state"] else None,
                 lengths=_lengths(c, g) if c["lens"] else None, states=None)
        if op == "glr_backward":
            s.update(dy=normal(B, T, C, dtype=dt),
                     dh_T=normal(B, C) if c["state"] else None)
            if c["states"]:
                s["states"] = _glr_forward(dict(s, dy=None))[2]
    elif op.startswith("qk"):
        B, T, Hq, Hk, D = (c[k] for k in ("B", "T", "Hq", "Hk", "D"))
        wide = normal(B, T, (Hq + 2 * Hk) * D, dtype=dt)
        n = c["rot"] // 2
        s.update(q=wide[:, :, :Hq * D], k=wide[:, :, Hq * D:(Hq + Hk) * D],
                 q_weight=1.0 + normal(D, scale=0.1) if c["weight"] else None,
                 k_weight=1.0 + normal(D, scale=0.1) if c["weight"] else None,
                 inv_freq=(10000.0 ** -(torch.arange(n, device="cuda") / max(n, 1))
                           ).float() if n else None,
                 positions=None, lengths=_lengths(c, g) if c["lens"] else None)
        if c["far"]:
            first = (uniform(0, 1, B, 1) * 1e6).to(torch.int32)
            s["positions"] = first + torch.arange(T, device="cuda", dtype=torch.int32)
        if op == "qk_rotary_backward":
            yt = torch.float32 if c["wide_dy"] else dt
            s.update(dq=normal(B, Hq, T, D, dtype=yt), dk=normal(B, Hk, T, D, dtype=yt))
    else:
        R, C, F = c["R"], c["C"], c["F"]
        s.update(x=normal(R, C + c["extra"], dtype=dt)[:, :C],
                 w_gate=normal(F, C, dtype=dt, scale=C ** -0.5),
                 w_up=normal(F, C, dtype=dt, scale=C ** -0.5))
        if op == "gated_ffn_backward":
            x = s["x"].float()
            s.update(gate=(x @ s["w_gate"].float().t()).to(dt),
                     up=(x @ s["w_up"].float().t()).to(dt),
                     dh=normal(R, F, dtype=dt))
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _valid(lengths, T):
    return torch.arange(T, device="cuda")[None, :] < lengths[:, None]


def _walk(a, b):
    """Every h_t = a_t h_{t-1} + b_t of [B, T, C] from zero, by doubling: after
    the step at d, b holds the sums over the last 2 d tokens and a the products
    of their decays (the loop is over the logarithm of T)."""
    d, T = 1, a.shape[1]
    while d < T:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], dim=1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], dim=1)
        d *= 2
    return b


def _glr_terms(s):
    """x, the input gate, the recurrence gate, the log decays, decays and input
    factors in fp64; tokens outside a sequence keep the state and add nothing."""
    x, r = s["x"].double(), s["r"].double()
    i = None if s["i"] is None else s["i"].double()
    if s["lengths"] is not None:
        ok = _valid(s["lengths"], x.shape[1])[:, :, None]
        x = torch.where(ok, x, 0.0)
        r = torch.where(ok, r, 0.0)
        i = None if i is None else torch.where(ok, i, 0.0)
    rho = torch.sigmoid(r)
    la = s["A"].double() * rho
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2.0 * la)) if s["case"]["normalize"] else torch.ones_like(a)
    gi = torch.ones_like(x) if i is None else torch.sigmoid(i)
    if s["lengths"] is not None:
        a, m = torch.where(ok, a, 1.0), torch.where(ok, m, 0.0)
    return x, gi, rho, la, a, m


def _glr_states(s, a, b):
    """h_0 .. h_T as [B, T + 1, C]."""
    h0 = torch.zeros_like(b[:, 0]) if s["h0"] is None else s["h0"].double()
    first = torch.addcmul(b[:, :1], a[:, :1], h0[:, None])
    return torch.cat([h0[:, None], _walk(a, torch.cat([first, b[:, 1:]], dim=1))], dim=1)


def _glr_forward(s):
    c = s["case"]
    x, gi, rho, la, a, m = _glr_terms(s)
    h = _glr_states(s, a, m * (gi * x))
    y = h[:, 1:]
    if s["lengths"] is not None:
        y = torch.where(_valid(s["lengths"], c["T"])[:, :, None], y, 0.0)
    out = (y.to(s["x"].dtype).contiguous(), h[:, -1].float())
    return out + ((h[:, :-1:_INTERVAL].float().contiguous(),) if c["states"] else ())


def _glr_backward(s):
    c = s["case"]
    dtype = s["x"].dtype
    x, gi, rho, la, a, m = _glr_terms(s)
    u = gi * x
    h = _glr_states(s, a, m * u)
    dy = s["dy"].double()
    if s["lengths"] is not None:
        dy = torch.where(_valid(s["lengths"], c["T"])[:, :, None], dy, 0.0)
    last = torch.zeros_like(dy[:, 0]) if s["dh_T"] is None else s["dh_T"].double()
    # g_t = dy_t + a_{t+1} g_{t+1}, from the end
    nxt = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], dim=1)
    src = dy.flip(1)
    src = torch.cat([src[:, :1] + last[:, None], src[:, 1:]], dim=1)
    g = _walk(nxt, src).flip(1)
    du = g * m
    dla = g * (a * h[:, :-1])
    if c["normalize"]:
        # d sqrt(1 - a^2) / d log a = -a^2 / sqrt(1 - a^2)
        dla = dla - torch.where(m > 0, g * u * (a * a / m), 0.0)
    dr = dla * la * (1.0 - rho)
    if s["lengths"] is not None:
        dr = torch.where(_valid(s["lengths"], c["T"])[:, :, None], dr, 0.0)
        dla = torch.where(_valid(s["lengths"], c["T"])[:, :, None], dla, 0.0)
    out = dict(x=(du * gi).to(dtype), r=dr.to(dtype),
               A=(dla * rho).sum((0, 1)).float(), h0=(a[:, 0] * g[:, 0]).float())
    if s["i"] is not None:
        out["i"] = (du * u * (1.0 - gi)).to(dtype)
    return out


def _angles(s):
    """cos and sin [B or 1, T, 1, rot / 2] of the positions, from fp64 angles."""
    T = s["case"]["T"]
    p = (torch.arange(T, device="cuda")[None] if s["positions"] is None
         else s["positions"])
    w = p.double()[:, :, None, None] * s["inv_freq"].double()
    return torch.cos(w).float(), torch.sin(w).float()


def _halves(x, c):
    """The two members of every rotated pair, and the channels behind them."""
    rot = c["rot"]
    if c["interleaved"]:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _joined(u, v, rest, c):
    if c["interleaved"]:
        return torch.cat([torch.stack([u, v], dim=-1).flatten(-2), rest], dim=-1)
    return torch.cat([u, v, rest], dim=-1)


def _turn(x, s, sign):
    c = s["case"]
    if not c["rot"]:
        return x
    cs, sn = _angles(s)
    u, v, rest = _halves(x, c)
    sn = sn * sign
    return _joined(u * cs - v * sn, v * cs + u * sn, rest, c)


def _root(x, c):
    """The reciprocal norm of each head's row."""
    if c["norm"] == "none":
        return torch.ones_like(x[..., :1])
    sq = x.square()
    m = sq.mean(-1, keepdim=True) if c["norm"] == "rms" else sq.sum(-1, keepdim=True)
    return torch.rsqrt(m + _EPS)


def _qk_one(x, weight, s):
    c = s["case"]
    h = x.float().reshape(c["B"], c["T"], -1, c["D"])
    y = h * _root(h, c)
    y = _turn(y if weight is None else y * weight, s, 1.0)
    if s["lengths"] is not None:
        y = torch.where(_valid(s["lengths"], c["T"])[:, :, None, None], y, 0.0)
    return y.permute(0, 2, 1, 3).to(x.dtype).contiguous()


def _qk_one_backward(x, weight, dy, s):
    c = s["case"]
    h = x.float().reshape(c["B"], c["T"], -1, c["D"])
    e = dy.float().permute(0, 2, 1, 3)
    if s["lengths"] is not None:
        ok = _valid(s["lengths"], c["T"])[:, :, None, None]
        h, e = torch.where(ok, h, 0.0), torch.where(ok, e, 0.0)
    e = _turn(e, s, -1.0)
    r = _root(h, c)
    n = h * r
    d_w = None if weight is None else (e.double() * n.double()).sum((0, 1, 2)).float()
    e = e if weight is None else e * weight
    if c["norm"] != "none":
        dot = (n * e).mean(-1, keepdim=True) if c["norm"] == "rms" else (
            n * e).sum(-1, keepdim=True)
        e = e - n * dot
    dx = (r * e).reshape(c["B"], c["T"], -1).to(x.dtype)
    return dx, d_w


def _qk_forward(s):
    return _qk_one(s["q"], s["q_weight"], s), _qk_one(s["k"], s["k_weight"], s)


def _qk_backward(s):
    dq, dwq = _qk_one_backward(s["q"], s["q_weight"], s["dq"], s)
    dk, dwk = _qk_one_backward(s["k"], s["k_weight"], s["dk"], s)
    out = dict(q=dq, k=dk)
    if dwq is not None:
        out.update(q_weight=dwq, k_weight=dwk)
    return out


_RT2, _RT2PI = math.sqrt(0.5), math.sqrt(0.5 / math.pi)
_TANH_IN, _TANH_CUBE = math.sqrt(2.0 / math.pi), 0.044715


def _activated(g, act):
    """The activation of g and its slope."""
    if act == "silu":
        sg = torch.sigmoid(g)
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * _RT2))
        return g * p, p + g * _RT2PI * torch.exp(-0.5 * g * g)
    t = torch.tanh(_TANH_IN * (g + _TANH_CUBE * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * (
        _TANH_IN * (1.0 + 3.0 * _TANH_CUBE * g * g))


def _ffn_forward(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    h = (_activated(g, c["act"])[0] * u).to(dt)
    return (h, g.to(dt), u.to(dt)) if c["save"] else h


def _ffn_backward(s):
    c, dt = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    f, slope = _activated(s["gate"].float(), c["act"])
    dh = s["dh"].float()
    dg, du = dh * s["up"].float() * slope, dh * f
    return dict(x=(dg @ wg + du @ wu).to(dt), w_gate=(dg.t() @ x).to(dt),
                w_up=(du.t() @ x).to(dt))


_PLAIN = {
    "glr_forward": _glr_forward, "glr_decode": _glr_forward,
    "glr_backward": _glr_backward, "qk_rotary_forward": _qk_forward,
    "qk_rotary_backward": _qk_backward, "gated_ffn_forward": _ffn_forward,
    "gated_ffn_backward": _ffn_backward,
}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _own(s):
    import delta_rule_recurrent_scan_amd as osdn
    c = s["case"]
    op = c["op"]
    if op.startswith("glr"):
        k = dict(i=s["i"], normalize=c["normalize"])
        if op == "glr_forward":
            y, h_T, states = osdn.glr_forward(s["x"], s["r"], s["A"], h0=s["h0"],
                                              lengths=s["lengths"],
                                              save=c["states"], **k)
            return (y, h_T, states) if c["states"] else (y, h_T)
        if op == "glr_decode":
            h = torch.empty_like(s["h0"])
            return osdn.glr_decode(s["x"], s["r"], s["A"], s["h0"], h_out=h, **k), h
        d = osdn.glr_backward(s["x"], s["r"], s["A"], s["dy"], h0=s["h0"],
                              dh_T=s["dh_T"], lengths=s["lengths"],
                              states=s["states"], **k)
        return {n: t for n, t in d.items() if t is not None}
    if op.startswith("qk"):
        k = dict(head_dim=c["D"], inv_freq=s["inv_freq"], positions=s["positions"],
                 q_weight=s["q_weight"], k_weight=s["k_weight"],
                 lengths=s["lengths"], norm=c["norm"],
                 interleaved=c["interleaved"], eps=_EPS)
        if op == "qk_rotary_forward":
            return osdn.qk_rotary_forward(s["q"], s["k"], **k)
        d = osdn.qk_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], **k)
        return {n: t for n, t in d.items() if t is not None}
    if op == "gated_ffn_forward":
        h, gate, up = osdn.gated_ffn_forward(s["x"], s["w_gate"], s["w_up"],
                                             activation=c["act"], save=c["save"])
        return (h, gate, up) if c["save"] else h
    return osdn.gated_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["gate"],
                                   s["up"], s["dh"], activation=c["act"])


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    op, e = c["op"], 2 if c["dtype"] == "bf16" else 4
    if op.startswith("glr"):
        B, T, C = c["B"], c["T"], c["C"]
        n, col = B * T * C, B * C * 4
        ins = 3 if c["gate"] else 2
        kept = B * -(-T // _INTERVAL) * C * 4
        if op == "glr_backward":
            return dict(bytes=(2 * ins + 1) * n * e + 8 * C
                        + (3 if c["state"] else 1) * col
                        + (kept if c["states"] else 0), flops=40 * n)
        return dict(bytes=(ins + 1) * n * e + 4 * C
                    + (2 if c["state"] else 1) * col
                    + (kept if c["states"] else 0), flops=16 * n)
    if op.startswith("qk"):
        B, T, D, H = c["B"], c["T"], c["D"], c["Hq"] + c["Hk"]
        n = B * T * H * D
        if op == "qk_rotary_backward":
            return dict(bytes=n * (2 * e + (4 if c["wide_dy"] else e)), flops=16 * n)
        return dict(bytes=2 * n * e, flops=8 * n)
    R, C, F = c["R"], c["C"], c["F"]
    if op == "gated_ffn_forward":
        return dict(bytes=(R * C + 2 * F * C + (3 if c["save"] else 1) * R * F) * e,
                    flops=4 * R * C * F)
    return dict(bytes=(2 * R * C + 4 * F * C + 3 * R * F) * e, flops=8 * R * C * F)


# ---------------------------------------------------------------------------
# The definitions in fp64
# ---------------------------------------------------------------------------

def _exact_glr(s):
    c = s["case"]
    B, T, C = c["B"], c["T"], c["C"]
    A = s["A"].double()
    h = (torch.zeros(B, C, dtype=torch.float64, device="cuda") if s["h0"] is None
         else s["h0"].double())
    n = None if s["lengths"] is None else s["lengths"].long()
    back = c["op"] == "glr_backward"
    before = (torch.zeros(B, T, C, dtype=torch.float64, device="cuda") if back
              else None)
    kept, ys = [], []

    def token(t):
        x = s["x"][:, t].double()
        rho = 1.0 / (1.0 + torch.exp(-s["r"][:, t].double()))
        gi = (torch.ones_like(x) if s["i"] is None
              else 1.0 / (1.0 + torch.exp(-s["i"][:, t].double())))
        la = A * rho
        a = torch.exp(la)
        m = torch.sqrt(-torch.expm1(2 * la)) if c["normalize"] else torch.ones_like(a)
        on = None if n is None else (t < n)[:, None]
        return x, rho, gi, la, a, m, on

    for t in range(T):
        x, rho, gi, la, a, m, on = token(t)
        if t % _INTERVAL == 0 and c["states"] and not back:
            kept.append(h)
        if back:
            before[:, t] = h
        new = a * h + m * gi * x
        h = new if on is None else torch.where(on, new, h)
        if not back:
            ys.append(new if on is None else torch.where(on, new, torch.zeros_like(new)))
    if not back:
        return (torch.stack(ys, dim=1), h) + (
            (torch.stack(kept, dim=1),) if c["states"] else ())
    g = torch.zeros_like(h) if s["dh_T"] is None else s["dh_T"].double()
    dA = torch.zeros(C, dtype=torch.float64, device="cuda")
    out = {k: torch.zeros(B, T, C, dtype=torch.float64, device="cuda")
           for k in ("x", "r") + (() if s["i"] is None else ("i",))}
    for t in range(T - 1, -1, -1):
        x, rho, gi, la, a, m, on = token(t)
        now = g + s["dy"][:, t].double()
        if on is not None:
            now = torch.where(on, now, torch.zeros_like(now))
        d_in = now * m
        d_la = now * a * before[:, t]
        if c["normalize"]:
            part = now * gi * x * a * a / m
            d_la = d_la - torch.where(m > 0, part, torch.zeros_like(part))
        out["x"][:, t] = d_in * gi
        if s["i"] is not None:
            out["i"][:, t] = d_in * x * gi * (1 - gi)
        out["r"][:, t] = d_la * la * (1 - rho)
        dA += (d_la * rho).sum(0)
        g = a * now if on is None else torch.where(on, a * now, g)
    return dict(x=out["x"], r=out["r"], A=dA, h0=g,
                **({} if s["i"] is None else dict(i=out["i"])))


def _exact_qk(s):
    c = s["case"]
    B, T, D, rot = c["B"], c["T"], c["D"], c["rot"]
    p = (torch.arange(T, device="cuda").expand(B, T) if s["positions"] is None
         else s["positions"]).double()
    # the rotation as a matrix on each token's row: y = M x
    eye = torch.eye(D, dtype=torch.float64, device="cuda")
    first = torch.arange(rot // 2, device="cuda")
    i0 = 2 * first if c["interleaved"] else first
    i1 = i0 + (1 if c["interleaved"] else rot // 2)
    back = c["op"] == "qk_rotary_backward"
    ok = None if s["lengths"] is None else (
        torch.arange(T, device="cuda")[None] < s["lengths"].long()[:, None])[..., None, None]

    def turned(v, sign):
        y = v @ eye
        if rot:
            w = p[:, :, None] * s["inv_freq"].double()
            cs, sn = torch.cos(w)[:, :, None], sign * torch.sin(w)[:, :, None]
            a, b = v[..., i0], v[..., i1]
            y = y.index_copy(-1, i0, a * cs - b * sn)
            y = y.index_copy(-1, i1, b * cs + a * sn)
        return y

    def one(name):
        w = s[name + "_weight"]
        w = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
        x = s[name].double().reshape(B, T, -1, D)
        if ok is not None:
            x = torch.where(ok, x, torch.zeros_like(x))
        count = {"rms": D, "l2": 1, "none": 0}[c["norm"]]
        root = (torch.sqrt((x * x).sum(-1, keepdim=True) / count + _EPS) if count
                else torch.ones_like(x[..., :1]))
        if not back:
            y = turned(x / root * w, 1.0)
            if ok is not None:
                y = torch.where(ok, y, torch.zeros_like(y))
            return y.permute(0, 2, 1, 3).contiguous()
        e = s["d" + name].double().permute(0, 2, 1, 3)
        if ok is not None:
            e = torch.where(ok, e, torch.zeros_like(e))
        e = turned(e, -1.0)
        dw = (e * x / root).sum((0, 1, 2))
        e = e * w
        dx = e / root
        if count:
            dx = dx - x * (x * e).sum(-1, keepdim=True) / (count * root ** 3)
        return dx.reshape(B, T, -1), dw

    if not back:
        return one("q"), one("k")
    (dq, dwq), (dk, dwk) = one("q"), one("k")
    out = dict(q=dq, k=dk)
    if s["q_weight"] is not None:
        out.update(q_weight=dwq, k_weight=dwk)
    return out


def _exact_ffn(s):
    c = s["case"]
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()

    def act(v):
        if c["act"] == "silu":
            return v / (1.0 + torch.exp(-v))
        if c["act"] == "gelu":
            return v * torch.special.ndtr(v)
        # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
        z = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v / (1.0 + torch.exp(-2.0 * z))

    def slope(v):
        if c["act"] == "silu":
            p = 1.0 / (1.0 + torch.exp(-v))
            return p + v * p * (1.0 - p)
        if c["act"] == "gelu":
            return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        z = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        p = 1.0 / (1.0 + torch.exp(-2.0 * z))
        return p + v * 2.0 * p * (1.0 - p) * math.sqrt(2 / math.pi) * (1 + 0.134145 * v * v)

    if c["op"] == "gated_ffn_forward":
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        return (act(g) * u, g, u) if c["save"] else act(g) * u
    g, dh = s["gate"].double(), s["dh"].double()
    dg, du = dh * s["up"].double() * slope(g), dh * act(g)
    return dict(x=torch.mm(dg, wg) + torch.mm(du, wu), w_gate=torch.mm(dg.t(), x),
                w_up=torch.mm(du.t(), x))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("glr"):
        if op == "glr_backward":
            s["states"] = None
        return _exact_glr(s)
    return _exact_qk(s) if op.startswith("qk") else _exact_ffn(s)
