"""The operators in a row, as a layer uses them, against a plain 64-bit
implementation and its gradients: the state space layer that the benchmark
times (residual norm, short convolutions over slices of one projection,
selective scan, gated norm, and all their backward calls), a prompt continued by
single tokens, a padded batch, and short convolutions with their L2 norm before
the delta rule.

Relative L2 errors. A result lies at most 12 roundings to the activations' type
behind the inputs (three convolved inputs, scan, gated norm, and the same back),
each off by at most half a step of its tensor's norm; sums over independent
terms do not raise the relative error of their norm. bf16: 12 * 2^-8. fp32: a
stage's result is a sum of up to 320 terms, 12 * 320 * 2^-24."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import bench
import delta_rule_recurrent_scan_amd as osdn
from parity import rel_l2
from workloads import layers as WL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 12 * 2.0 ** -8, F32: 12 * 320 * 2.0 ** -24}


def leaf(t):
    return t.detach().cpu().double().requires_grad_()


def close(got, ref, tol, what):
    e = rel_l2(got.detach().cpu().double().numpy(), ref.detach().numpy())
    print("%s: %.2e (bound %.2e)" % (what, e, tol), flush=True)
    assert e <= tol, what


def conv(x, w, b, heads, l2=False, state=None, eps=1e-6):
    """x [B,T,C] -> [B,heads,T,C/heads]."""
    B, T, C = x.shape
    W = w.shape[1]
    head = torch.zeros(B, W - 1, C, dtype=x.dtype) if state is None else state
    u = F.conv1d(torch.cat([head, x], 1).transpose(1, 2), w[:, None], b, groups=C)
    v = F.silu(u).transpose(1, 2).reshape(B, T, heads, -1)
    if l2:
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) + eps)
    return v.transpose(1, 2)


def scan(x, dt, A, B, C, D, dt_bias, S=None):
    H, G, T = x.shape[1], B.shape[1], x.shape[2]
    B, C = (t.repeat_interleave(H // G, 1) for t in (B, C))
    s = F.softplus(dt + dt_bias[:, None])
    S = torch.zeros(x.shape[0], H, x.shape[3], B.shape[3], dtype=x.dtype) if S is None else S
    ys = []
    for t in range(T):
        S = (torch.exp(s[:, :, t] * A)[..., None, None] * S + s[:, :, t, None, None]
             * x[:, :, t, :, None] * B[:, :, t, None, :])
        ys.append((S * C[:, :, t, None, :]).sum(-1) + D[:, None] * x[:, :, t])
    return torch.stack(ys, 2), S


def gate(y, z, w, eps=1e-6):
    """y [B,H,T,D], z [B,T,H*D], w [H,D]."""
    B, H, T, D = y.shape
    n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w[:, None]
    return n.transpose(1, 2).reshape(B, T, H * D) * F.silu(z)


def rms(h, w, eps=1e-6):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w


SIZES = [dict(B=2, H=4, G=2, T=70, P=64, N=32, channels=96),
         dict(B=1, H=2, G=2, T=133, P=128, N=128, channels=515),
         dict(B=3, H=6, G=1, T=5, P=32, N=64, channels=128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "T%d" % s["T"])
def test_layer_and_its_gradients(size, dtype):
    w = WL.BY_NAME["ssm-layer"].scaled(dtype=dtype, seed=7, **size)
    a = WL.make_layer(w, DEV)
    step, o = bench.layer_forward(w, a)
    step()
    back, g = bench.layer_backward(w, a, o)
    back()
    torch.cuda.synchronize()

    r = {n: leaf(a[n]) for n in ("residual", "block", "norm", "proj", "dt", "A", "D",
                                 "dt_bias", "gate_norm")}
    cw, cb = [leaf(t) for t in a["conv_w"]], [leaf(t) for t in a["conv_b"]]
    xs = list(torch.split(r["proj"], w.splits, -1))
    c = [conv(xs[i], cw[i], cb[i], n) for i, n in enumerate((w.H, w.G, w.G))]
    y, S = scan(c[0], r["dt"], r["A"], c[1], c[2], r["D"], r["dt_bias"])
    out = gate(y, xs[3], r["gate_norm"])
    h = r["residual"] + r["block"]
    n = rms(h, r["norm"])
    ((out * a["dy"].cpu().double()).sum()
     + (n * a["dnorm"].cpu().double()).sum()).backward()

    tol = TOL[a["proj"].dtype]
    close(o["h"], h, tol, "h")
    close(o["norm"], n, tol, "norm")
    for i in range(3):
        close(o["conv"][i], c[i], tol, "conv %s" % "xBC"[i])
    close(o["y"], y, tol, "y")
    close(o["S"], S, tol, "S_T")
    close(o["out"], out, tol, "out")
    dproj = torch.cat([t["x"] for t in g["conv"]] + [g["gate"]["z"]], -1)
    for i in range(4):
        lo = sum(w.splits[:i])
        cut = slice(lo, lo + w.splits[i])
        close(dproj[..., cut], r["proj"].grad[..., cut], tol, "d proj %s" % "xBCz"[i])
    for i in range(3):
        close(g["conv"][i]["weight"], cw[i].grad, tol, "d conv weight %d" % i)
        close(g["conv"][i]["bias"], cb[i].grad, tol, "d conv bias %d" % i)
    for name in ("dt", "A", "dt_bias"):
        close(g["scan"][name], r[name].grad, tol, "d " + name)
    # dD = sum <dy, x> is no sum of independent terms: dy comes out of the norm,
    # whose gradient is orthogonal to the norm's input y = S C + D x (to eps), so
    # <dy, D x> = -<dy, S C>, and where D x makes up most of y, as it does in the
    # first tokens, the sum is a small rest of its terms. With dy and x each off
    # by tol / 2 of their norms, the sum is off by tol |dy| |x| (Cauchy-Schwarz).
    size = [t.detach().pow(2).sum((0, 2, 3)).sqrt() for t in (g["gate"]["x"].cpu().double(), c[0])]
    err = (g["scan"]["D"].cpu().double() - r["D"].grad).abs()
    assert (err <= tol * size[0] * size[1]).all(), "d D"
    close(g["gate"]["weight"], r["gate_norm"].grad, tol, "d gate norm")
    close(g["norm"]["x"], r["block"].grad, tol, "d block")
    close(g["norm"]["residual"], r["residual"].grad, tol, "d residual")
    close(g["norm"]["weight"], r["norm"].grad, tol, "d norm")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_single_tokens(dtype):
    w = WL.BY_NAME["ssm-layer-decode"].scaled(B=3, H=4, G=2, P=64, N=128, channels=100,
                                              dtype=dtype, seed=9)
    a = WL.make_layer(w, DEV)
    S, tails = leaf(a["S"]), [leaf(t) for t in a["conv_state"]]
    step, o = bench.layer_forward(w, a)
    xs = [t.detach() for t in torch.split(leaf(a["proj"]), w.splits, -1)]
    tol = TOL[a["proj"].dtype]
    for turn in range(3):      # the same token, on the states it moved
        step()
        torch.cuda.synchronize()
        c = []
        for i, n in enumerate((w.H, w.G, w.G)):
            c.append(conv(xs[i], a["conv_w"][i].cpu().double(),
                          a["conv_b"][i].cpu().double(), n, state=tails[i]))
            tails[i] = torch.cat([tails[i], xs[i]], 1)[:, 1:]
        y, S = scan(c[0], a["dt"].cpu().double(), a["A"].cpu().double(), c[1], c[2],
                    a["D"].cpu().double(), a["dt_bias"].cpu().double(), S)
        out = gate(y, xs[3], a["gate_norm"].cpu().double())
        close(o["out"], out, tol, "out of step %d" % turn)
        close(a["S"], S, tol, "S of step %d" % turn)
        for i in range(3):
            close(a["conv_state"][i], tails[i], 0.0, "conv state %d" % i)


@pytest.mark.parametrize("dt", [F32, BF])
def test_prompt_then_tokens_equals_one_sequence(dt):
    """A padded batch of prompts, then three tokens each, against the whole
    sequences in one call: same operands, same functions; both sides lie within
    the bound of the exact result."""
    B, H, G, P, N, W, T = 3, 4, 2, 64, 64, 4, 40
    lens = [40, 17, 0]
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g)
    full = n(B, T + 3, H * P).to(dt).to(DEV)
    Bm, Cm = (n(B, G, T + 3, N).to(dt).to(DEV) for _ in range(2))
    step = n(B, H, T + 3).to(DEV)
    A = -(1 + n(H).abs()).to(DEV)
    cw, cb = n(H * P, W).to(DEV), n(H * P).to(DEV)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)

    x, tail = osdn.short_conv_forward(full[:, :T], cw, cb, lengths=L, head_dim=P)
    cut = lambda t: t[:, :, :T].contiguous()
    y, S = osdn.ssm_forward(x, cut(step), A, cut(Bm), cut(Cm), lengths=L)
    for b, m in enumerate(lens):
        assert not y[b, :, m:].any()
    whole = []
    for b, m in enumerate(lens):
        xb, _ = osdn.short_conv_forward(full[b:b + 1, :m + 3], cw, cb, head_dim=P)
        at = lambda t: t[b:b + 1, :, :m + 3].contiguous()
        whole.append(osdn.ssm_forward(xb, at(step), A, at(Bm), at(Cm)))
        if m:
            assert rel_l2(y[b, :, :m].cpu().double().numpy(),
                          whole[b][0][0, :, :m].cpu().double().numpy()) <= TOL[dt]
    for i in range(3):
        pick = lambda t, dim: torch.stack([t[b].narrow(dim, lens[b] + i, 1)
                                           for b in range(B)]).contiguous()
        xi = osdn.short_conv_decode(pick(full, 0), cw, tail, cb, head_dim=P)
        yi = osdn.ssm_decode(xi, pick(step, 1), A, pick(Bm, 1), pick(Cm, 1), S)
        for b, m in enumerate(lens):
            close(yi[b, :, 0], whole[b][0][0, :, m + i].cpu().double(), TOL[dt],
                  "entry %d, token %d" % (b, i))
    for b in range(B):
        close(S[b], whole[b][1][0].cpu().double(), TOL[dt], "state of entry %d" % b)


def delta(q, k, v, beta, eta):
    """OSDN without a forgetting gate, from S = 0 and d = 1."""
    S = torch.zeros(*v.shape[:2], v.shape[-1], k.shape[-1], dtype=v.dtype)
    d = torch.ones(*k.shape[:2], k.shape[-1], dtype=v.dtype)
    out = []
    for t in range(k.shape[2]):
        kt, bt = k[:, :, t], beta[:, :, t, None]
        u = bt * (v[:, :, t] - (S * kt[..., None, :]).sum(-1))
        S = S + u[..., None] * (d * kt)[..., None, :]
        out.append((S * q[:, :, t, None, :]).sum(-1))
        a = kt * kt
        n, c = a.sum(-1, keepdim=True), (d * a).sum(-1, keepdim=True)
        d = d + eta * bt * (1 - bt * c) / n * a
    return torch.stack(out, 2)


def test_convolutions_and_gated_norm_around_the_delta_rule():
    """q and k convolved and L2 normalised, v convolved, the delta rule, the
    gated norm; back: its fp32 gradients go into the convolutions' backward."""
    B, H, T, D, W, eta = 2, 3, 90, 64, 4, 0.1
    C = H * D
    g = torch.Generator().manual_seed(11)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)
    proj, z, dy = n(B, T, 3 * C), n(B, T, C), n(B, T, C)
    cw, gw = [n(C, W) * 0.5 for _ in range(3)], 1 + 0.1 * n(H, D)
    beta = torch.sigmoid(n(B, H, T))
    xs = [proj[..., i * C:(i + 1) * C] for i in range(3)]
    q, k, v = (osdn.short_conv_forward(xs[i], cw[i], head_dim=D, l2norm=i < 2)[0]
               for i in range(3))
    o, _, _ = osdn.osdn_forward(q, k, v, beta, None, eta)
    out = osdn.gated_norm_forward(o, z, gw)
    gg = osdn.gated_norm_backward(o, z, gw, dy)
    gd = osdn.osdn_backward(q, k, v, beta, gg["x"], eta=eta)
    gc = [osdn.short_conv_backward(xs[i], cw[i], gd["qkv"[i]], head_dim=D,
                                   l2norm=i < 2) for i in range(3)]

    rp, rz, rw, rb = leaf(proj), leaf(z), leaf(gw), leaf(beta)
    rc = [leaf(t) for t in cw]
    rq, rk, rv = (conv(rp[..., i * C:(i + 1) * C], rc[i], None, H, i < 2)
                  for i in range(3))
    ro = delta(rq, rk, rv, rb, eta)
    rout = gate(ro, rz, rw)
    (rout * dy.cpu().double()).sum().backward()
    close(o, ro, TOL[F32], "o")
    close(out, rout, TOL[F32], "out")
    close(gg["z"], rz.grad, TOL[F32], "dz")
    close(gg["weight"], rw.grad, TOL[F32], "d gate norm")
    close(gd["beta"], rb.grad, TOL[F32], "d beta")
    for i in range(3):
        close(gc[i]["x"], rp.grad[..., i * C:(i + 1) * C], TOL[F32], "d proj %d" % i)
        close(gc[i]["weight"], rc[i].grad, TOL[F32], "d conv weight %d" % i)
    assert not np.isnan(out.cpu().numpy()).any()


def test_lengths_outside_the_sequence_are_clamped():
    B, T, H, G, P, N = 3, 70, 2, 1, 64, 32
    g = torch.Generator().manual_seed(13)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)
    out = torch.tensor([-5, T + 9, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    inside = torch.tensor([0, T, T], dtype=torch.int32, device=DEV)
    rows, cw, dy = n(B, T, H * P), n(H * P, 4), n(B, H, T, P)
    a = (n(B, H, T), -(1 + n(H).abs()), n(B, G, T, N), n(B, G, T, N))
    got = []
    for lens in (out, inside):
        x, tail = osdn.short_conv_forward(rows, cw, lengths=lens, head_dim=P)
        y, S = osdn.ssm_forward(x, *a, lengths=lens)
        gs = osdn.ssm_backward(x, *a, dy, lengths=lens)
        gc = osdn.short_conv_backward(rows, cw, gs["x"], lengths=lens, head_dim=P)
        got.append([x, tail, y, S] + list(gs.values()) + list(gc.values()))
    for u, v in zip(*got):
        assert torch.equal(u, v)
