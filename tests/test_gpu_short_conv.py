"""GPU parity of the short causal convolution (forward, decode, backward)
against the fp64 oracle."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import DEV, f64, held, rows
from oracle import mixer as M

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# B, T, H, D, W, dtype, l2norm, extra channels of the row, lengths
CASES = [
    (2, 37, 3, 64, 4, BF, True, 64, None),
    (2, 37, 3, 32, 4, BF, True, 5, [37, 11]),      # rows off 16 bytes
    (1, 1, 1, 128, 4, F32, True, 0, None),
    (3, 70, 5, 32, 3, F32, False, 0, [70, 0, 1]),
    (1, 2, 2, 128, 4, BF, False, 0, None),         # fewer tokens than taps
    (2, 3, 1, 7, 4, F32, False, 2, None),          # an odd width, no heads
    (1, 131, 1, 1001, 2, BF, False, 0, [130]),
    (4, 130, 9, 128, 4, BF, True, 8, [130, 1, 129, 64]),
    (1, 33, 4, 20, 4, BF, False, 0, None),         # heads off 8 channels
]
IDS = ["-".join(str(x) for x in c[:5]) + ("-f32" if c[5] is F32 else "-bf16")
       for c in CASES]


def _inputs(case, seed=0):
    B, T, H, D, W, dt, l2, extra, lens = case
    g = torch.Generator().manual_seed(seed)
    C = H * D
    a = dict(x=rows((B, T, C), dt, g, extra),
             weight=(torch.randn((C, W), generator=g) * W ** -0.5).to(DEV),
             bias=(torch.randn(C, generator=g) * 0.1).to(DEV),
             state=torch.randn((B, W - 1, C), generator=g).to(dt).to(DEV))
    k = dict(head_dim=D, l2norm=l2, eps=1e-6,
             lengths=None if lens is None else torch.tensor(
                 lens, dtype=torch.int32, device=DEV))
    return a, k, g


def _ref_args(a, k):
    lens = None if k["lengths"] is None else k["lengths"].cpu().numpy()
    return ({n: f64(t) for n, t in a.items()},
            dict(lengths=lens, head_dim=k["head_dim"], l2norm=k["l2norm"],
                 eps=k["eps"]))


def _mags(r, kr, H, D):
    """|u| terms and, per head, what an error of u does to y."""
    ab = {n: np.abs(t) for n, t in r.items()}
    kw = dict(kr, l2norm=False)
    y0, _, u = M.short_conv_ref(r["x"], r["weight"], r["bias"], r["state"], **kw)
    _, _, ua = M.short_conv_ref(ab["x"], ab["weight"], ab["bias"], ab["state"], **kw)
    B, T, C = u.shape
    heads = lambda t: t.reshape(B, T, H, D).transpose(0, 2, 1, 3)
    m = 2.0 * heads(ua) * (1 + np.abs(heads(u)))   # silu and its relative error
    norm = np.sqrt((y0 * y0).sum(-1, keepdims=True) + kr["eps"])
    return y0, u, m, norm


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    B, T, H, D, W, dt, l2, extra, lens = case
    print("case:", case, flush=True)
    a, k, _ = _inputs(case)
    y, tail = osdn.short_conv_forward(a["x"], a["weight"], a["bias"], a["state"], **k)
    torch.cuda.synchronize()
    r, kr = _ref_args(a, k)
    ry, rt, _ = M.short_conv_ref(r["x"], r["weight"], r["bias"], r["state"], **kr)
    y0, u, m, norm = _mags(r, kr, H, D)
    if l2:  # an error of any channel moves the row's norm
        m = (m + np.abs(ry) * np.sqrt((m * m).sum(-1, keepdims=True))) / norm + np.abs(ry)
    held(y, ry, m, 4 * W + 48, what="y")
    assert np.array_equal(f64(tail), rt)
    # nothing beyond the inputs: no bias, no state, no activation
    y, tail = osdn.short_conv_forward(a["x"], a["weight"], activation=False,
                                      **dict(k, l2norm=False))
    kr2 = dict(kr, l2norm=False, activation=False)
    ry, rt, _ = M.short_conv_ref(r["x"], r["weight"], **kr2)
    mag, _, _ = M.short_conv_ref(np.abs(r["x"]), np.abs(r["weight"]), **kr2)
    held(y, ry, mag, 2 * W, what="plain y")
    assert np.array_equal(f64(tail), rt)


def test_padding_is_never_used():
    case = (3, 40, 2, 64, 4, BF, True, 8, [40, 7, 0])
    a, k, g = _inputs(case)
    dy = torch.randn((3, 2, 40, 64), generator=g).to(BF).to(DEV)
    y, tail = osdn.short_conv_forward(a["x"], a["weight"], a["bias"], a["state"], **k)
    d = osdn.short_conv_backward(a["x"], a["weight"], dy, a["bias"], a["state"], **k)
    for b, n in enumerate(case[-1]):
        a["x"][b, n:] = float("nan")
        dy[b, :, n:] = float("inf")
    y2, tail2 = osdn.short_conv_forward(a["x"], a["weight"], a["bias"], a["state"], **k)
    d2 = osdn.short_conv_backward(a["x"], a["weight"], dy, a["bias"], a["state"], **k)
    assert torch.equal(y, y2) and torch.equal(tail, tail2)
    for n in d:
        assert torch.equal(d[n], d2[n]), n
    for b, n in enumerate(case[-1]):
        assert not y2[b, :, n:].any() and not d2["x"][b, n:].any()


def test_a_zero_row_and_a_zero_token_axis():
    a, k, _ = _inputs((1, 5, 2, 64, 4, BF, True, 0, None))
    x = torch.zeros_like(a["x"])
    y, _ = osdn.short_conv_forward(x, a["weight"], head_dim=64, l2norm=True)
    assert not y.any()
    d = osdn.short_conv_backward(x, a["weight"], torch.ones_like(y), head_dim=64,
                                 l2norm=True)
    assert all(bool(torch.isfinite(t).all()) for t in d.values())
    # no tokens: the state stays; its adjoint passes through
    x0 = a["x"][:, :0]
    y, tail = osdn.short_conv_forward(x0, a["weight"], a["bias"], a["state"], **k)
    assert y.shape == (1, 2, 0, 64) and torch.equal(tail, a["state"])
    d = osdn.short_conv_backward(x0, a["weight"], y, a["bias"], a["state"],
                                 dstate_T=a["state"], **k)
    assert torch.equal(d["state"], a["state"])
    assert not d["weight"].any() and not d["bias"].any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("W", [2, 4])
def test_decode_continues_forward(dt, W):
    """A prompt, then tokens one, three and one at a time, in place: the bits
    of the whole prompt at once."""
    case = (2, 29, 3, 64, W, dt, True, 16, None)
    a, k, _ = _inputs(case)
    k.pop("lengths")
    want, tail = osdn.short_conv_forward(a["x"], a["weight"], a["bias"], a["state"], **k)
    got, st = osdn.short_conv_forward(a["x"][:, :24], a["weight"], a["bias"],
                                      a["state"], **k)
    out = [got]
    for i, j in ((24, 25), (25, 28), (28, 29)):
        out.append(osdn.short_conv_decode(a["x"][:, i:j], a["weight"], st,
                                          bias=a["bias"], **k))
    assert torch.equal(torch.cat(out, 2), want) and torch.equal(st, tail)
    # the state kept, the new one elsewhere
    before = st.clone()
    nxt = torch.empty_like(st)
    osdn.short_conv_decode(a["x"][:, :1], a["weight"], st, bias=a["bias"],
                           state_out=nxt, **k)
    assert torch.equal(st, before) and not torch.equal(nxt, st)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("dy32", [False, True])
def test_backward(case, dy32):
    B, T, H, D, W, dt, l2, extra, lens = case
    print("case:", case, flush=True)
    a, k, g = _inputs(case, 1)
    C = H * D
    dy = torch.randn((B, H, T, D), generator=g).to(F32 if dy32 else dt).to(DEV)
    dst = torch.randn((B, W - 1, C), generator=g).to(dt).to(DEV)
    got = osdn.short_conv_backward(a["x"], a["weight"], dy, a["bias"], a["state"],
                                   dstate_T=dst, **k)
    torch.cuda.synchronize()
    r, kr = _ref_args(a, k)
    ref = M.short_conv_backward_ref(r["x"], r["weight"], f64(dy), r["bias"],
                                    r["state"], dstate_T=f64(dst), **kr)
    # |dv| terms; du = dv * slope, the slope's own error through u's
    y0, u, m, norm = _mags(r, kr, H, D)
    ady = np.abs(f64(dy))
    if l2:
        v = y0 / norm
        rel = 1 + np.sqrt((m * m).sum(-1, keepdims=True)) / norm
        adv = (ady + np.abs(v) * (np.abs(v) * ady).sum(-1, keepdims=True)) / norm
        adv = adv + (m / norm) * (np.abs(v) * ady).sum(-1, keepdims=True) / norm \
            + np.abs(v) * (m * ady).sum(-1, keepdims=True) / norm ** 2
        adv = adv * rel
    else:
        adv = ady
    adu = (adv * (2 + m)).transpose(0, 2, 1, 3).reshape(B, T, C)
    n = M._lengths(kr["lengths"], B, T)
    mx, ms = np.zeros((B, T, C)), np.zeros((B, W - 1, C))
    mw, mb = np.zeros((C, W)), np.zeros(C)
    for b in range(B):
        full = np.concatenate([r["state"][b], r["x"][b, :n[b]]])
        df = np.zeros_like(full)
        df[n[b]:] += np.abs(f64(dst)[b])
        for t in range(n[b]):
            df[t:t + W] += np.abs(r["weight"].T) * adu[b, t]
            mw += np.abs(full[t:t + W] * adu[b, t]).T
            mb += adu[b, t]
        ms[b], mx[b, :n[b]] = df[:W - 1], df[W - 1:]
    kk = 4 * W + 64
    held(got["x"], ref["x"], mx, kk, what="dx")
    held(got["state"], ref["state"], ms, kk, what="dstate")
    held(got["weight"], ref["weight"], mw, kk + 64, what="dweight")
    held(got["bias"], ref["bias"], mb, kk + 64, what="dbias")


def test_backward_against_differences():
    """The gradient against central differences of the forward itself, fp32."""
    case = (2, 21, 2, 32, 4, F32, True, 0, [21, 9])
    a, k, g = _inputs(case, 2)
    dy = torch.randn((2, 2, 21, 32), generator=g).to(DEV)
    got = osdn.short_conv_backward(a["x"], a["weight"], dy, a["bias"], a["state"], **k)

    def loss(p):
        y, _ = osdn.short_conv_forward(p["x"], p["weight"], p["bias"], p["state"], **k)
        return float((y.double() * dy.double()).sum())
    for n in ("x", "weight", "bias", "state"):
        d = torch.randn(a[n].shape, generator=g).to(DEV)
        h = 2.0 ** -8
        num = (loss(dict(a, **{n: a[n] + h * d})) - loss(dict(a, **{n: a[n] - h * d}))) / (2 * h)
        ana = float((got[n].double() * d.double()).sum())
        # 2^-24 roundings of some 1300 outputs of size 1 over 2h, and h^2
        scale = float(got[n].double().norm() * d.double().norm())
        assert abs(num - ana) <= 2e-3 * scale + 1e-2, (n, num, ana)
