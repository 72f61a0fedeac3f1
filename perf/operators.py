"""Cases of the sequence-mixer operators around the recurrences: the short
causal convolution, the selective state space scan, the gated head norm and
the residual norm.

Each case is one pass through one entry point. ``run`` computes it either in
its plain form (elementary torch operations in fp32, rounded once at the end)
or, with ``own`` true, through the package's entry points; ``exact`` is the
definition once more in fp64, token by token or as full score matrices.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_CHUNK = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _ssm(name, op, B, H, G, T, P, N, dtype, lens=False, state=False):
    return dict(name=name, op=op, B=B, H=H, G=G, T=T, P=P, N=N, dtype=dtype,
                lens=lens, state=state)


def _conv(name, op, B, T, H, D, W, dtype, l2norm=False, lens=False, extra=0):
    return dict(name=name, op=op, B=B, T=T, H=H, D=D, W=W, dtype=dtype,
                l2norm=l2norm, lens=lens, extra=extra)


def _gate(name, op, B, H, T, D, dtype, gate_first=False, per_head=False):
    return dict(name=name, op=op, B=B, H=H, T=T, D=D, dtype=dtype,
                gate_first=gate_first, per_head=per_head)


def _res(name, op, R, C, dtype, res, scale=1.0):
    return dict(name=name, op=op, R=R, C=C, dtype=dtype, res=res, scale=scale)


def listed():
    return [
        # a training or prefill batch at the 1.3B-layer head shape
        _ssm("scan prompt", "ssm_forward", 4, 16, 2, 4096, 128, 128, "bf16"),
        # a padded batch of prompts of different lengths, continued from a state
        _ssm("scan ragged fp32", "ssm_forward", 3, 8, 4, 1000, 64, 32, "f32",
             lens=True, state=True),
        # a serving step of 128 sequences, one token each
        _ssm("scan decode", "ssm_decode", 128, 16, 2, 1, 128, 128, "bf16",
             state=True),
        # the gradients of a training batch, keys shared by eight heads
        _ssm("scan backward", "ssm_backward", 4, 16, 2, 2048, 128, 128, "bf16"),
        # the same, one ragged batch in fp32 with a carried state
        _ssm("scan backward ragged", "ssm_backward", 2, 6, 3, 333, 64, 64,
             "f32", lens=True, state=True),
        # keys and queries of a 1.3B layer out of one wide projection, unit rows
        _conv("conv prompt", "short_conv_forward", 4, 4096, 32, 128, 4, "bf16",
              l2norm=True, extra=2176),
        # one token of a single sequence: latency
        _conv("conv decode", "short_conv_decode", 1, 1, 16, 128, 4, "bf16"),
        # the gradients of a training batch of values, padded
        _conv("conv backward", "short_conv_backward", 8, 2048, 16, 128, 4,
              "bf16", lens=True, extra=128),
        # the heads of a layer brought together before its output projection
        _gate("gated norm", "gated_norm_forward", 4, 16, 4096, 128, "bf16"),
        # its gradients, gate before the norm, a weight for every head
        _gate("gated norm backward", "gated_norm_backward", 8, 8, 2048, 64,
              "bf16", gate_first=True, per_head=True),
        # the norm before a block, the residual stream kept in fp32
        _res("residual norm", "residual_norm_forward", 16384, 2048, "bf16",
             "f32"),
        # its gradients, an odd width
        _res("residual norm backward", "residual_norm_backward", 4097, 1021,
             "bf16", "bf16", scale=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ssm_forward", "ssm_forward", "ssm_decode", "ssm_backward",
                     "short_conv_forward", "short_conv_decode",
                     "short_conv_backward", "gated_norm_forward",
                     "gated_norm_backward", "residual_norm_forward",
                     "residual_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("ssm"):
        G = rng.choice([1, 2, 3, 4])
        H = G * rng.choice([1, 2, 4, 5, 8])
        P, N = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        c = _ssm("", op, 1, H, G, 1, P, N, dtype, lens=rng.random() < 0.5,
                 state=rng.random() < 0.5)
        if op == "ssm_decode":
            c.update(B=_spread(rng, 1, 192), T=rng.choice([1, 1, 1, 2, 5]),
                     lens=False, state=True)
            c["B"] = min(c["B"], max(1, 4096 // H))
        else:
            most = 65536 if dtype == "bf16" else 16384
            c["T"] = _spread(rng, 1, 8192)
            c["B"] = rng.randint(1, max(1, min(8, most // (H * c["T"]))))
            c["T"] = min(c["T"], most * 4 // (c["B"] * H))
    elif op.startswith("short_conv"):
        D = rng.choice([32, 64, 128])
        c = _conv("", op, 1, 1, rng.randint(1, 24), D, rng.choice([2, 3, 4]),
                  dtype, l2norm=rng.random() < 0.5,
                  lens=op != "short_conv_decode" and rng.random() < 0.5,
                  extra=rng.choice([0, 0, 8, 5, 256]))
        if op == "short_conv_decode":
            c.update(B=_spread(rng, 1, 256), T=rng.choice([1, 1, 2, 4]))
        else:
            c.update(B=rng.randint(1, 4), T=_spread(rng, 1, 4096))
        if rng.random() < 0.2 and not c["l2norm"]:  # channels without heads
            c.update(H=1, D=rng.randint(1, 2500))
    elif op.startswith("gated_norm"):
        c = _gate("", op, rng.randint(1, 4), rng.randint(1, 20),
                  _spread(rng, 1, 4096), rng.choice([32, 64, 128]), dtype,
                  gate_first=rng.random() < 0.5, per_head=rng.random() < 0.5)
    else:
        c = _res("", op, _spread(rng, 1, 16384), _spread(rng, 16, 2048), dtype,
                 rng.choice(["f32", dtype]), scale=rng.choice([1.0, 0.5, 0.22]))
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
    op = c["op"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=c)
    if op.startswith("ssm"):
        B, H, G, T, P, N = (c[k] for k in ("B", "H", "G", "T", "P", "N"))
        dt = _DT[c["dtype"]]
        # steps between 1/1000 and 1/10 around which the tokens select
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        s.update(x=normal(B, H, T, P, dtype=dt), dt=normal(B, H, T),
                 A=-uniform(1.0, 16.0, H),
                 Bm=normal(B, G, T, N, dtype=dt), Cm=normal(B, G, T, N, dtype=dt),
                 D=normal(H) * 0.1 + 1.0, dt_bias=torch.log(torch.expm1(step)),
                 S0=normal(B, H, P, N, scale=N ** -0.5) if c["state"] else None,
                 lengths=_lengths(c, g) if c["lens"] else None)
        if op == "ssm_backward":
            s.update(dy=normal(B, H, T, P, dtype=dt),
                     dS_T=normal(B, H, P, N, scale=N ** -0.5)
                     if c["state"] else None)
    elif op.startswith("short_conv"):
        B, T, H, D, W = (c[k] for k in ("B", "T", "H", "D", "W"))
        dt, C = _DT[c["dtype"]], H * D
        wide = normal(B, T, C + c["extra"], dtype=dt)
        s.update(x=wide[:, :, :C], weight=normal(C, W, scale=W ** -0.5),
                 bias=normal(C, scale=0.1),
                 state=normal(B, W - 1, C, dtype=dt),
                 lengths=_lengths(c, g) if c["lens"] else None)
        if op == "short_conv_backward":
            s.update(dy=normal(B, H, T, D, dtype=dt),
                     dstate_T=normal(B, W - 1, C, dtype=dt))
    elif op.startswith("gated_norm"):
        B, H, T, D = (c[k] for k in ("B", "H", "T", "D"))
        dt = _DT[c["dtype"]]
        wide = normal(B, T, H * D + 64, dtype=dt)
        shape = (H, D) if c["per_head"] else (D,)
        s.update(x=normal(B, H, T, D, dtype=dt, scale=0.5), z=wide[:, :, :H * D],
                 weight=1.0 + normal(*shape, scale=0.1))
        if op == "gated_norm_backward":
            s.update(dy=normal(B, T, H * D, dtype=dt))
    else:
        R, C = c["R"], c["C"]
        dt, rt = _DT[c["dtype"]], _DT[c["res"]]
        s.update(weight=1.0 + normal(C, scale=0.1))
        if op == "residual_norm_forward":
            s.update(x=normal(R, C, dtype=dt), residual=normal(R, C, dtype=rt))
        else:
            s.update(dy=normal(R, C, dtype=dt), h=normal(R, C, dtype=rt),
                     dh=normal(R, C, dtype=rt))
    return s


# ---------------------------------------------------------------------------
# The plain forms, fp32
# ---------------------------------------------------------------------------

def _valid(lengths, T):
    return torch.arange(T, device="cuda")[None, :] < lengths[:, None]


def _step(dt_raw, bias):
    """softplus of the raw step with its bias, and softplus' slope."""
    v = dt_raw.double() + bias.double()[:, None]
    dt = torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))
    return dt, torch.sigmoid(v)


def _chunks(s, dy=None):
    """The scan's inputs in fp32, padded to whole chunks [.., nc, Q, ..], and
    the decays between tokens, chunk ends and chunks, from fp64 sums."""
    c = s["case"]
    B, H, G, T, P, N = (c[k] for k in ("B", "H", "G", "T", "P", "N"))
    Q = min(_CHUNK, T)
    nc = -(-T // Q)
    dt, slope = _step(s["dt"], s["dt_bias"])
    x, Bm, Cm = s["x"].float(), s["Bm"].float(), s["Cm"].float()
    if s["lengths"] is not None:
        ok = _valid(s["lengths"], T)
        dt = torch.where(ok[:, None], dt, 0.0)
        o4 = ok[:, None, :, None]
        x, Bm, Cm = (torch.where(o4, t, 0.0) for t in (x, Bm, Cm))
        dy = None if dy is None else torch.where(o4, dy, 0.0)
    pad = nc * Q - T

    def cut(t):
        t = torch.nn.functional.pad(t, (0, 0, 0, pad))
        return t.view(*t.shape[:2], nc, Q, t.shape[-1])

    k = dict(Q=Q, nc=nc, T=T, R=H // G, slope=slope, dt64=dt)
    k["x"] = cut(x).view(B, G, H // G, nc, Q, P)
    k["B"], k["C"] = cut(Bm).unsqueeze(2), cut(Cm).unsqueeze(2)
    if dy is not None:
        k["dy"] = cut(dy).view(B, G, H // G, nc, Q, P)
    d = torch.nn.functional.pad(dt, (0, pad)).view(B, G, H // G, nc, Q)
    cum = (d * s["A"].double().view(G, H // G, 1, 1)).cumsum(-1)
    tri = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    k["L"] = torch.exp(torch.where(tri, cum[..., :, None] - cum[..., None, :],
                                   -math.inf)).float()
    k["dt"] = d.float()
    k["entry"] = torch.exp(cum).float()                    # chunk entry .. token
    k["exit"] = torch.exp(cum[..., -1:] - cum).float()     # token .. chunk exit
    # state i (0 is S0, i > 0 leaves chunk i - 1) into the entry of chunk j
    tot = torch.nn.functional.pad(cum[..., -1].cumsum(-1), (1, 0))
    tri = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device="cuda").tril()
    k["between"] = torch.exp(torch.where(
        tri, tot[..., :, None] - tot[..., None, :], -math.inf)).float()
    k["whole"] = torch.exp(cum[..., -1]).float()
    k["S0"] = (torch.zeros(B, G, H // G, 1, P, N, device="cuda")
               if s["S0"] is None else s["S0"].view(B, G, H // G, 1, P, N))
    return k


def _states(k):
    """The states at every chunk's entry and after the last [.., nc + 1, P, N]."""
    w = k["dt"] * k["exit"]
    local = (k["x"] * w[..., None]).transpose(-1, -2) @ k["B"]
    every = torch.cat([k["S0"], local], dim=3)
    return (k["between"] @ every.flatten(-2)).view(every.shape)


def _ssm_forward(s):
    c = s["case"]
    dtype = s["x"].dtype
    k = _chunks(s)
    S = _states(k)
    M = (k["C"] @ k["B"].transpose(-1, -2)) * k["L"] * k["dt"][..., None, :]
    y = M @ k["x"] + k["entry"][..., None] * (k["C"] @ S[:, :, :, :-1].transpose(-1, -2))
    y = y + s["D"].view(c["G"], k["R"], 1, 1, 1) * k["x"]
    y = y.reshape(c["B"], c["H"], -1, c["P"])[:, :, :k["T"]]
    S_T = S[:, :, :, -1].reshape(c["B"], c["H"], c["P"], c["N"])
    return y.to(dtype).contiguous(), S_T.contiguous()


def _ssm_backward(s):
    c = s["case"]
    B, H, G, P, N = (c[k] for k in ("B", "H", "G", "P", "N"))
    dtype = s["x"].dtype
    k = _chunks(s, s["dy"].float())
    x, dy, Bm, Cm, dt = k["x"], k["dy"], k["B"], k["C"], k["dt"]
    A = s["A"].view(G, H // G, 1, 1)
    S = _states(k)[:, :, :, :-1]
    last = (torch.zeros(B, G, H // G, 1, P, N, device="cuda")
            if s["dS_T"] is None else s["dS_T"].view(B, G, H // G, 1, P, N))
    local = (dy * k["entry"][..., None]).transpose(-1, -2) @ Cm
    every = torch.cat([local, last], dim=3)
    adj = (k["between"].transpose(-1, -2) @ every.flatten(-2)).view(every.shape)
    dS0, dS = adj[:, :, :, 0], adj[:, :, :, 1:]   # dS[c]: at chunk c's exit
    CB = Cm @ Bm.transpose(-1, -2)
    dM = dy @ x.transpose(-1, -2)
    K = CB * k["L"]
    Z = dM * k["L"]
    V = Z * CB
    out_x = dS @ Bm.transpose(-1, -2)             # [P, Q]: what x meets at the exit
    dx = (K * dt[..., None, :]).transpose(-1, -2) @ dy
    dx = dx + (k["exit"] * dt)[..., None] * out_x.transpose(-1, -2)
    dx = dx + s["D"].view(G, H // G, 1, 1, 1) * dy
    Zd = Z * dt[..., None, :]
    in_y = S.transpose(-1, -2) @ dy.transpose(-1, -2)   # [N, Q]
    out_B = dS.transpose(-1, -2) @ x.transpose(-1, -2)  # [N, Q]
    dC = Zd @ Bm + k["entry"][..., None] * in_y.transpose(-1, -2)
    dB = Zd.transpose(-1, -2) @ Cm + (k["exit"] * dt)[..., None] * out_B.transpose(-1, -2)
    dB, dC = dB.sum(2), dC.sum(2)
    # the step's own gradient, and the decay's: every pair of a source before
    # a token and a use at or after it
    u = k["exit"] * (out_B.transpose(-1, -2) * Bm).sum(-1)
    w = k["entry"] * (in_y.transpose(-1, -2) * Cm).sum(-1)
    own_dt = V.sum(-2) + u
    Vd = (V * dt[..., None, :]).double().tril(-1)
    pairs = Vd.sum(-1) - Vd.sum(-2)
    g = pairs.flip(-1).cumsum(-1).flip(-1)
    g = g + w.double().flip(-1).cumsum(-1).flip(-1)
    ud = (u * dt).double()
    g = g + ud.cumsum(-1) - ud
    g = g + (k["whole"] * (dS * S).sum((-1, -2))).double()[..., None]
    d_dt = own_dt.double() + A.double() * g
    dA = (g * dt.double()).sum((0, 3, 4)).reshape(H)
    dD = (dy.double() * x.double()).sum((0, 3, 4, 5)).reshape(H)
    T = k["T"]
    d_raw = d_dt.reshape(B, H, -1)[:, :, :T] * k["slope"]
    if s["lengths"] is not None:
        d_raw = torch.where(_valid(s["lengths"], T)[:, None], d_raw, 0.0)

    def tokens(t, heads):
        return t.reshape(B, heads, -1, t.shape[-1])[:, :, :T].to(dtype).contiguous()

    return dict(x=tokens(dx, H), dt=d_raw.float(), A=dA.float(), B=tokens(dB, G),
                C=tokens(dC, G), D=dD.float(), dt_bias=d_raw.sum((0, 2)).float(),
                S0=dS0.reshape(B, H, P, N).contiguous())


def _windows(s):
    """The W inputs that each token's convolution sees [B, T, C, W], fp32, and
    the inputs with the state before them."""
    full = torch.cat([s["state"].float(), s["x"].float()], dim=1)
    return full.unfold(1, s["case"]["W"], 1), full


def _tail(full, s):
    """The last W - 1 inputs of each sequence."""
    c = s["case"]
    if s["lengths"] is None:
        return full[:, c["T"]:]
    at = s["lengths"].long()[:, None] + torch.arange(c["W"] - 1, device="cuda")
    return full.gather(1, at[:, :, None].expand(-1, -1, full.shape[2]))


def _short_conv(s):
    c = s["case"]
    B, T, H, D = (c[k] for k in ("B", "T", "H", "D"))
    win, full = _windows(s)
    u = (win * s["weight"]).sum(-1) + s["bias"]
    y = (u * torch.sigmoid(u)).view(B, T, H, D)
    if c["l2norm"]:
        y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) + _EPS)
    if s["lengths"] is not None:
        y = torch.where(_valid(s["lengths"], T)[:, :, None, None], y, 0.0)
    y = y.permute(0, 2, 1, 3).to(s["x"].dtype).contiguous()
    return y, _tail(full, s).to(s["x"].dtype).contiguous()


def _short_conv_backward(s):
    c = s["case"]
    B, T, H, D, W = (c[k] for k in ("B", "T", "H", "D", "W"))
    C, dtype = H * D, s["x"].dtype
    win, full = _windows(s)
    u = (win * s["weight"]).sum(-1) + s["bias"]
    sg = torch.sigmoid(u)
    dv = s["dy"].float().permute(0, 2, 1, 3)
    if c["l2norm"]:
        v = (u * sg).view(B, T, H, D)
        r = torch.rsqrt(v.square().sum(-1, keepdim=True) + _EPS)
        dv = r * (dv - v * (r * r * (v * dv).sum(-1, keepdim=True)))
    du = dv.reshape(B, T, C) * (sg * (1.0 + u * (1.0 - sg)))
    if s["lengths"] is not None:
        du = torch.where(_valid(s["lengths"], T)[:, :, None], du, 0.0)
    d_w = (du.double()[..., None] * win.double()).sum((0, 1))
    d_b = du.double().sum((0, 1))
    # input t is seen by tokens t .. t + W - 1, through the weights from the last
    around = torch.nn.functional.pad(du, (0, 0, W - 1, W - 1)).unfold(1, W, 1)
    d_full = (around * s["weight"].flip(-1)).sum(-1)
    tail = s["dstate_T"].float()
    if s["lengths"] is None:
        d_full = d_full + torch.nn.functional.pad(tail, (0, 0, T, 0))
    else:
        at = s["lengths"].long()[:, None] + torch.arange(W - 1, device="cuda")
        d_full = d_full.scatter_add(1, at[:, :, None].expand(-1, -1, C), tail)
    return dict(x=d_full[:, W - 1:].to(dtype).contiguous(), weight=d_w.float(),
                bias=d_b.float(), state=d_full[:, :W - 1].to(dtype).contiguous())


def _gated_norm(s):
    c = s["case"]
    B, H, T, D = (c[k] for k in ("B", "H", "T", "D"))
    x = s["x"].float().permute(0, 2, 1, 3)
    z = s["z"].float().reshape(B, T, H, D)
    gate = z * torch.sigmoid(z)
    v = x * gate if c["gate_first"] else x
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS) * s["weight"]
    y = y if c["gate_first"] else y * gate
    return y.reshape(B, T, H * D).to(s["x"].dtype)


def _gated_norm_backward(s):
    c = s["case"]
    B, H, T, D = (c[k] for k in ("B", "H", "T", "D"))
    dtype = s["x"].dtype
    x = s["x"].float().permute(0, 2, 1, 3)
    z = s["z"].float().reshape(B, T, H, D)
    dy = s["dy"].float().view(B, T, H, D)
    sg = torch.sigmoid(z)
    gate, slope = z * sg, sg * (1.0 + z * (1.0 - sg))
    v = x * gate if c["gate_first"] else x
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
    n = v * r
    dn_w = dy if c["gate_first"] else dy * gate
    d_w = (dn_w.double() * n.double()).sum((0, 1) if c["per_head"] else (0, 1, 2))
    dn = dn_w * s["weight"]
    dv = r * (dn - n * (n * dn).mean(-1, keepdim=True))
    if c["gate_first"]:
        dx, dgate = dv * gate, dv * x
    else:
        dx, dgate = dv, dy * n * s["weight"]
    return dict(x=dx.permute(0, 2, 1, 3).to(dtype).contiguous(),
                z=(dgate * slope).reshape(B, T, H * D).to(dtype),
                weight=d_w.float())


def _residual_norm(s):
    h = s["residual"].float() + s["case"]["scale"] * s["x"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS) * s["weight"]
    return y.to(s["x"].dtype), h.to(s["residual"].dtype)


def _residual_norm_backward(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS)
    n = h * r
    d_w = (dy.double() * n.double()).sum(0)
    dn = dy * s["weight"]
    dh = s["dh"].float() + r * (dn - n * (n * dn).mean(-1, keepdim=True))
    return dict(x=(s["case"]["scale"] * dh).to(s["dy"].dtype),
                residual=dh.to(s["h"].dtype), weight=d_w.float())


_PLAIN = {
    "ssm_forward": _ssm_forward, "ssm_decode": _ssm_forward,
    "ssm_backward": _ssm_backward, "short_conv_forward": _short_conv,
    "short_conv_decode": _short_conv, "short_conv_backward": _short_conv_backward,
    "gated_norm_forward": _gated_norm, "gated_norm_backward": _gated_norm_backward,
    "residual_norm_forward": _residual_norm,
    "residual_norm_backward": _residual_norm_backward,
}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _own(s):
    import delta_rule_recurrent_scan_amd as osdn
    c = s["case"]
    op = c["op"]
    if op.startswith("ssm"):
        a = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
        k = dict(D=s["D"], dt_bias=s["dt_bias"])
        if op == "ssm_forward":
            return osdn.ssm_forward(*a, S0=s["S0"], lengths=s["lengths"], **k)
        if op == "ssm_decode":
            S = torch.empty_like(s["S0"])
            return osdn.ssm_decode(*a, s["S0"], S_out=S, **k), S
        return osdn.ssm_backward(*a, s["dy"], S0=s["S0"], dS_T=s["dS_T"],
                                 lengths=s["lengths"], **k)
    if op.startswith("short_conv"):
        k = dict(bias=s["bias"], head_dim=c["D"], l2norm=c["l2norm"], eps=_EPS)
        if op == "short_conv_forward":
            return osdn.short_conv_forward(s["x"], s["weight"], state=s["state"],
                                           lengths=s["lengths"], **k)
        if op == "short_conv_decode":
            state = torch.empty_like(s["state"])
            return osdn.short_conv_decode(s["x"], s["weight"], s["state"],
                                          state_out=state, **k), state
        return osdn.short_conv_backward(s["x"], s["weight"], s["dy"],
                                        state=s["state"], lengths=s["lengths"],
                                        dstate_T=s["dstate_T"], **k)
    if op.startswith("gated_norm"):
        k = dict(eps=_EPS, gate_first=c["gate_first"])
        if op == "gated_norm_forward":
            return osdn.gated_norm_forward(s["x"], s["z"], s["weight"], **k)
        return osdn.gated_norm_backward(s["x"], s["z"], s["weight"], s["dy"], **k)
    if op == "residual_norm_forward":
        return osdn.residual_norm_forward(s["x"], s["weight"], s["residual"],
                                          scale=c["scale"], eps=_EPS)
    return osdn.residual_norm_backward(s["dy"], s["h"], s["weight"], dh=s["dh"],
                                       scale=c["scale"], eps=_EPS)


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
    if op.startswith("ssm"):
        B, H, G, T, P, N = (c[k] for k in ("B", "H", "G", "T", "P", "N"))
        states = (2 if c["state"] else 1) * B * H * P * N * 4
        if op == "ssm_backward":
            # x, dy in, dx out; B, C in, their gradients out; dt and its own
            return dict(bytes=B * T * (3 * H * P * e + 4 * G * N * e + 8 * H)
                        + (states + (B * H * P * N * 4 if c["state"] else 0)),
                        flops=10 * B * H * T * P * N)
        return dict(bytes=B * T * (2 * H * P * e + 2 * G * N * e + 4 * H) + states,
                    flops=4 * B * H * T * P * N)
    if op.startswith("short_conv"):
        n, W = c["B"] * c["T"] * c["H"] * c["D"], c["W"]
        tail = c["B"] * (W - 1) * c["H"] * c["D"] * e
        if op == "short_conv_backward":
            return dict(bytes=3 * n * e + 3 * tail, flops=(6 * W + 20) * n)
        return dict(bytes=2 * n * e + 2 * tail, flops=(2 * W + 12) * n)
    if op.startswith("gated_norm"):
        n = c["B"] * c["H"] * c["T"] * c["D"]
        if op == "gated_norm_backward":
            return dict(bytes=5 * n * e, flops=30 * n)
        return dict(bytes=3 * n * e, flops=12 * n)
    n, r = c["R"] * c["C"], 2 if c["res"] == "bf16" else 4
    if op == "residual_norm_forward":
        return dict(bytes=n * (2 * e + 2 * r), flops=7 * n)
    return dict(bytes=n * (2 * e + 3 * r), flops=15 * n)


# ---------------------------------------------------------------------------
# The definitions, fp64
# ---------------------------------------------------------------------------

def _exact_ssm(c, s, back):
    B, H, G, T, P, N = (c[k] for k in ("B", "H", "G", "T", "P", "N"))
    f = {k: None if s.get(k) is None else s[k].double()
         for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "S0", "dy", "dS_T")}
    if back:
        o = dict(x=torch.zeros_like(f["x"]), dt=torch.zeros_like(f["dt"]),
                 A=torch.zeros_like(f["A"]), B=torch.zeros_like(f["Bm"]),
                 C=torch.zeros_like(f["Cm"]), D=torch.zeros_like(f["D"]),
                 dt_bias=torch.zeros_like(f["A"]),
                 S0=torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda"))
    else:
        y = torch.zeros_like(f["x"])
        S_T = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        for h in range(H):
            g = h // (H // G)
            x, Bt, Ct = f["x"][b, h, :n], f["Bm"][b, g, :n], f["Cm"][b, g, :n]
            v = f["dt"][b, h, :n] + f["dt_bias"][h]
            dt = torch.logaddexp(v, torch.zeros_like(v))
            S0 = (torch.zeros(P, N, dtype=torch.float64, device="cuda")
                  if f["S0"] is None else f["S0"][b, h])
            lam = torch.cumsum(dt * f["A"][h], 0)
            end = lam[-1] if n else torch.zeros((), dtype=torch.float64, device="cuda")
            L = torch.exp(torch.tril(lam[:, None] - lam[None, :]))
            L = torch.tril(L)
            scores = (Ct @ Bt.T) * L
            if not back:
                y[b, h, :n] = (scores @ (dt[:, None] * x) + f["D"][h] * x
                               + torch.exp(lam)[:, None] * (Ct @ S0.T))
                S_T[b, h] = (torch.exp(end) * S0
                             + (torch.exp(end - lam) * dt)[:, None].mul(x).T @ Bt)
                continue
            dy = f["dy"][b, h, :n]
            dS = (torch.zeros_like(S0) if f["dS_T"] is None else f["dS_T"][b, h])
            into, left = torch.exp(lam)[:, None], torch.exp(end - lam)[:, None]
            at_end = left * (Bt @ dS.T)               # what x_j dt_j adds to the loss at the end
            with_x = scores.T @ dy + at_end           # d loss / d (dt_j x_j)
            o["x"][b, h, :n] = dt[:, None] * with_x + f["D"][h] * dy
            pair = (dy @ x.T) * L * dt[None, :]
            o["C"][b, g, :n] += pair @ Bt + into * (dy @ S0)
            o["B"][b, g, :n] += pair.T @ Ct + left * dt[:, None] * (x @ dS)
            # d loss / d (log decay of token t): what crosses from before t to t or after
            cross = torch.tril(pair * (Ct @ Bt.T), -1)
            uses = (into * (dy @ S0) * Ct).sum(1)
            kept = (x * at_end).sum(1) * dt
            suffix = torch.flip(torch.cumsum(torch.flip(
                cross.sum(1) - cross.sum(0) + uses, (0,)), 0), (0,))
            dlam = suffix + torch.cumsum(kept, 0) - kept + torch.exp(end) * (S0 * dS).sum()
            ddt = (with_x * x).sum(1) + f["A"][h] * dlam
            o["dt"][b, h, :n] = ddt * torch.sigmoid(v)
            o["dt_bias"][h] += (ddt * torch.sigmoid(v)).sum()
            o["A"][h] += (dt * dlam).sum()
            o["D"][h] += (dy * x).sum()
            o["S0"][b, h] = torch.exp(end) * dS + (into * dy).T @ Ct
    return o if back else (y, S_T)


def _exact_conv(c, s, back):
    B, T, H, D, W = (c[k] for k in ("B", "T", "H", "D", "W"))
    C = H * D
    w, bias = s["weight"].double(), s["bias"].double()
    full = torch.cat([s["state"], s["x"]], dim=1).double()
    n = (torch.full((B,), T, device="cuda") if s["lengths"] is None
         else s["lengths"].long())
    ok = (torch.arange(T, device="cuda")[None] < n[:, None])[:, :, None]
    u = bias + sum(full[:, k:k + T] * w[:, k] for k in range(W))
    act = torch.nn.functional.silu(u)
    heads = act.view(B, T, H, D)
    norm = (heads.square().sum(-1, keepdim=True) + _EPS).sqrt()
    if not back:
        y = heads / norm if c["l2norm"] else heads
        y = y * ok[..., None]
        tail = torch.stack([full[b, int(n[b]):int(n[b]) + W - 1] for b in range(B)])
        return y.transpose(1, 2).contiguous(), tail
    dv = s["dy"].double().transpose(1, 2)
    if c["l2norm"]:
        y = heads / norm
        dv = (dv - y * (y * dv).sum(-1, keepdim=True)) / norm
    sg = torch.sigmoid(u)
    du = dv.reshape(B, T, C) * (sg + u * sg * (1 - sg)) * ok
    d_full = torch.zeros_like(full)
    d_w = torch.zeros_like(w)
    for k in range(W):
        d_full[:, k:k + T] += du * w[:, k]
        d_w[:, k] = (du * full[:, k:k + T]).sum((0, 1))
    for b in range(B):
        d_full[b, int(n[b]):int(n[b]) + W - 1] += s["dstate_T"][b].double()
    return dict(x=d_full[:, W - 1:], weight=d_w, bias=du.sum((0, 1)),
                state=d_full[:, :W - 1])


def _exact_gate(c, s, back):
    B, H, T, D = (c[k] for k in ("B", "H", "T", "D"))
    x = s["x"].double().transpose(1, 2)
    z = s["z"].double().reshape(B, T, H, D)
    w = s["weight"].double()
    gate = torch.nn.functional.silu(z)
    v = x * gate if c["gate_first"] else x
    rms = (v.square().sum(-1, keepdim=True) / D + _EPS).sqrt()
    if not back:
        y = v / rms * w * (1 if c["gate_first"] else gate)
        return y.reshape(B, T, H * D)
    dy = s["dy"].double().view(B, T, H, D)
    sg = torch.sigmoid(z)
    slope = sg + z * sg * (1 - sg)
    up = dy if c["gate_first"] else dy * gate
    dw = up * v / rms
    a = up * w
    dv = a / rms - v * (a * v).sum(-1, keepdim=True) / (D * rms ** 3)
    dx = dv * gate if c["gate_first"] else dv
    dz = (dv * x if c["gate_first"] else dy * w * v / rms) * slope
    return dict(x=dx.transpose(1, 2), z=dz.reshape(B, T, H * D),
                weight=dw.sum((0, 1)) if c["per_head"] else dw.sum((0, 1, 2)))


def _exact_res(c, s, back):
    w = s["weight"].double()
    if not back:
        h = s["residual"].double() + c["scale"] * s["x"].double()
        return h / (h.square().mean(-1, keepdim=True) + _EPS).sqrt() * w, h
    h, dy = s["h"].double(), s["dy"].double()
    rms = (h.square().mean(-1, keepdim=True) + _EPS).sqrt()
    a = dy * w
    dh = (s["dh"].double() + a / rms
          - h * (a * h).sum(-1, keepdim=True) / (c["C"] * rms ** 3))
    return dict(x=c["scale"] * dh, residual=dh, weight=(dy * h / rms).sum(0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    back = op.endswith("backward")
    if op.startswith("ssm"):
        return _exact_ssm(case, s, back)
    if op.startswith("short_conv"):
        return _exact_conv(case, s, back)
    if op.startswith("gated_norm"):
        return _exact_gate(case, s, back)
    return _exact_res(case, s, back)
