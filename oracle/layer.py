"""The operators that complete a block, token by token in NumPy fp64: gated linear
recurrence, norm and rotation of queries and keys, gated feed-forward product,
with their adjoints. Written from the definitions, nothing blocked or reordered;
the HIP path shares no code with it.

The adjoints return, beside every gradient, the sum of the absolute values of the
terms that make it: what a rounding error of the terms is measured against.
"""
import math

import numpy as np

from .mixer import _lengths, sigmoid

_erf = np.vectorize(math.erf, otypes=[float])
_erfc = np.vectorize(math.erfc, otypes=[float])


# ---------------------------------------------------------------------------
# Gated linear recurrence: x, r, i [B,T,C], A [C]
# ---------------------------------------------------------------------------

def glr_factors(r, A, normalize=True):
    """(rho, log a, a, m)."""
    rho = sigmoid(r)
    la = A * rho
    a = np.exp(la)
    m = np.sqrt(-np.expm1(2 * la)) if normalize else np.ones_like(a)
    return rho, la, a, m


def glr_ref(x, r, A, i=None, h0=None, lengths=None, normalize=True):
    """(y [B,T,C], h_T [B,C], h before every token [B,T,C])."""
    B, T, C = x.shape
    n = _lengths(lengths, B, T)
    y, before = np.zeros((B, T, C)), np.zeros((B, T, C))
    h_T = np.zeros((B, C))
    for b in range(B):
        h = np.zeros(C) if h0 is None else h0[b].copy()
        for t in range(T):
            before[b, t] = h
            if t < n[b]:
                _, _, a, m = glr_factors(r[b, t], A, normalize)
                u = x[b, t] * (1.0 if i is None else sigmoid(i[b, t]))
                h = a * h + m * u
                y[b, t] = h
        h_T[b] = h
    return y, h_T, before


def glr_backward_ref(x, r, A, dy, i=None, h0=None, dh_T=None, lengths=None,
                     normalize=True):
    """Two dicts x, r, i, A, h0: the gradients of sum <dy, y> + <dh_T, h_T>, and
    the magnitudes of their terms."""
    B, T, C = x.shape
    n = _lengths(lengths, B, T)
    before = glr_ref(x, r, A, i, h0, lengths, normalize)[2]
    big = glr_ref(np.abs(x), r, A, i, None if h0 is None else np.abs(h0), lengths,
                  normalize)[2]
    names = ("x", "r") + (() if i is None else ("i",))
    g = {k: np.zeros((B, T, C)) for k in names}
    mag = {k: np.zeros((B, T, C)) for k in names}
    for d in (g, mag):
        d.update(A=np.zeros(C), h0=np.zeros((B, C)))
    for b in range(B):
        c = np.zeros(C) if dh_T is None else dh_T[b].copy()
        cm = np.abs(c)
        for t in range(n[b] - 1, -1, -1):
            rho, la, a, m = glr_factors(r[b, t], A, normalize)
            # (1 - sigmoid(z) would lose its digits at an open gate)
            shut = sigmoid(-r[b, t])
            gi = np.ones(C) if i is None else sigmoid(i[b, t])
            u = gi * x[b, t]
            now, nowm = c + dy[b, t], cm + np.abs(dy[b, t])
            g["x"][b, t], mag["x"][b, t] = now * m * gi, nowm * m * gi
            if i is not None:
                less = u * sigmoid(-i[b, t])
                g["i"][b, t], mag["i"][b, t] = now * m * less, nowm * m * np.abs(less)
            w = np.zeros(C)
            if normalize:
                np.divide(a * a * u, m, out=w, where=m > 0)
            dla = now * (a * before[b, t] - w)
            dlam = nowm * (a * big[b, t] + np.abs(w))
            g["r"][b, t], mag["r"][b, t] = dla * la * shut, dlam * np.abs(la) * shut
            g["A"] += dla * rho
            mag["A"] += dlam * rho
            c, cm = a * now, a * nowm
        g["h0"][b], mag["h0"][b] = c, cm
    return g, mag


# ---------------------------------------------------------------------------
# Norm and rotation: x [B,T,H*D] -> y [B,H,T,D]
# ---------------------------------------------------------------------------

def _pairs(rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def _turn(v, positions, inv_freq, interleaved, sign):
    """v [B,T,H,D] turned by the positions [B,T]."""
    if inv_freq is None or not len(inv_freq):
        return v.copy(), np.abs(v)
    a, b = _pairs(2 * len(inv_freq), interleaved)
    w = positions[:, :, None, None] * inv_freq
    cs, sn = np.cos(w), sign * np.sin(w)
    y, mag = v.copy(), np.abs(v)
    y[..., a] = v[..., a] * cs - v[..., b] * sn
    y[..., b] = v[..., b] * cs + v[..., a] * sn
    mag[..., a] = mag[..., b] = np.abs(v[..., a]) + np.abs(v[..., b])
    return y, mag


def _root(x, norm, eps):
    if norm == "none":
        return np.ones_like(x[..., :1]), 0
    count = x.shape[-1] if norm == "rms" else 1
    s = (x * x).sum(-1, keepdims=True) / count + eps
    # (rows of zeros keep their zeros with eps = 0)
    return np.where(s == 0, 0.0, 1 / np.sqrt(np.where(s == 0, 1.0, s))), count


def _off(lengths, B, T):
    return np.arange(T)[None, :] >= _lengths(lengths, B, T)[:, None]


def _positions(positions, B, T):
    return (np.broadcast_to(np.arange(T, dtype=float), (B, T)) if positions is None
            else np.asarray(positions, dtype=float))


def qk_rotary_ref(x, head_dim, inv_freq=None, weight=None, positions=None,
                  lengths=None, norm="rms", interleaved=False, eps=1e-6):
    """(y [B,H,T,D], the magnitudes of its terms)."""
    B, T, C = x.shape
    h = x.reshape(B, T, C // head_dim, head_dim)
    off = _off(lengths, B, T)
    h = np.where(off[:, :, None, None], 0.0, h)
    r, _ = _root(h, norm, eps)
    v = h * r * (1.0 if weight is None else weight)
    y, mag = _turn(v, _positions(positions, B, T), inv_freq, interleaved, 1.0)
    y[off], mag[off] = 0.0, 0.0
    return y.transpose(0, 2, 1, 3), mag.transpose(0, 2, 1, 3)


def qk_rotary_backward_ref(x, dy, head_dim, inv_freq=None, weight=None,
                           positions=None, lengths=None, norm="rms",
                           interleaved=False, eps=1e-6):
    """Two dicts x [B,T,H*D], weight [D]: gradients and magnitudes."""
    B, T, C = x.shape
    off = _off(lengths, B, T)[:, :, None, None]
    h = np.where(off, 0.0, x.reshape(B, T, C // head_dim, head_dim))
    e = np.where(off, 0.0, dy.transpose(0, 2, 1, 3))
    e, em = _turn(e, _positions(positions, B, T), inv_freq, interleaved, -1.0)
    r, count = _root(h, norm, eps)
    n = h * r
    w = np.ones(head_dim) if weight is None else weight
    g = dict(weight=(e * n).sum((0, 1, 2)))
    mag = dict(weight=(em * np.abs(n)).sum((0, 1, 2)))
    f, fm = e * w, em * np.abs(w)
    dx, dm = f, fm
    if count:
        dx = f - n * (n * f).sum(-1, keepdims=True) / count
        dm = fm + np.abs(n) * (np.abs(n) * fm).sum(-1, keepdims=True) / count
    g["x"], mag["x"] = (r * dx).reshape(B, T, C), (r * dm).reshape(B, T, C)
    return g, mag


# ---------------------------------------------------------------------------
# Gated feed-forward product: x [R,C], w_gate, w_up [F,C]
# ---------------------------------------------------------------------------

def activation(g, act):
    """(act(g), its slope)."""
    if act == "silu":
        s = sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * _erfc(-g / math.sqrt(2))
        return g * p, p + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return (0.5 * g * (1 + t),
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g))


def gated_ffn_ref(x, w_gate, w_up, act="silu"):
    """(h, g, u)."""
    g, u = x @ w_gate.T, x @ w_up.T
    return activation(g, act)[0] * u, g, u


def gated_ffn_backward_ref(x, w_gate, w_up, gate, up, dh, act="silu"):
    """dict x, w_gate, w_up from the stored gate and up, and dg, du."""
    f, slope = activation(gate, act)
    dg, du = dh * up * slope, dh * f
    return dict(x=dg @ w_gate + du @ w_up, w_gate=dg.T @ x, w_up=du.T @ x), dg, du
