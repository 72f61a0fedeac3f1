"""The operators around the recurrences, token by token in NumPy fp64: short
causal convolution, selective state space scan, gated head norm and residual
norm, with their adjoints. Written from the definitions, nothing blocked or
reordered; the HIP path shares no code with it.

Every gradient is a sum of products, so the same functions called with the
absolute values of their inputs (``A`` keeps its sign inside the decay) give
the sum of the absolute values of the terms: what a rounding error of the
terms is measured against.
"""
import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))),
                    np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def softplus(x):
    return np.logaddexp(x, 0.0)


def silu(x):
    return x * sigmoid(x)


def _silu_slope(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def _lengths(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


# ---------------------------------------------------------------------------
# Short convolution: x [B,T,C] -> y [B,H,T,D]
# ---------------------------------------------------------------------------

def short_conv_ref(x, weight, bias=None, state=None, lengths=None, head_dim=None,
                   activation=True, l2norm=False, eps=1e-6):
    """(y, state_T, pre-activation u [B,T,C])."""
    B, T, C = x.shape
    W = weight.shape[1]
    D = C if head_dim is None else head_dim
    n = _lengths(lengths, B, T)
    state = np.zeros((B, W - 1, C)) if state is None else state
    y = np.zeros((B, C // D, T, D))
    u = np.zeros((B, T, C))
    tail = np.zeros((B, W - 1, C))
    for b in range(B):
        full = np.concatenate([state[b], x[b, :n[b]]])
        for t in range(n[b]):
            u[b, t] = (full[t:t + W] * weight.T).sum(0) + (0 if bias is None else bias)
            v = silu(u[b, t]) if activation else u[b, t]
            v = v.reshape(C // D, D)
            if l2norm:
                v = v / np.sqrt((v * v).sum(-1, keepdims=True) + eps)
            y[b, :, t] = v
        tail[b] = full[n[b]:n[b] + W - 1]
    return y, tail, u


def short_conv_backward_ref(x, weight, dy, bias=None, state=None, lengths=None,
                            head_dim=None, activation=True, l2norm=False,
                            eps=1e-6, dstate_T=None):
    """dict(x, weight, bias, state) of sum <dy, y> + <dstate_T, state_T>."""
    B, T, C = x.shape
    W = weight.shape[1]
    D = C if head_dim is None else head_dim
    n = _lengths(lengths, B, T)
    state = np.zeros((B, W - 1, C)) if state is None else state
    _, _, u = short_conv_ref(x, weight, bias, state, lengths, head_dim,
                             activation, l2norm, eps)
    g = dict(x=np.zeros((B, T, C)), weight=np.zeros((C, W)), bias=np.zeros(C),
             state=np.zeros((B, W - 1, C)))
    for b in range(B):
        full = np.concatenate([state[b], x[b, :n[b]]])
        dfull = np.zeros_like(full)
        if dstate_T is not None:
            dfull[n[b]:] += dstate_T[b]
        for t in range(n[b]):
            v = (silu(u[b, t]) if activation else u[b, t]).reshape(C // D, D)
            dv = dy[b, :, t]
            if l2norm:
                r = 1.0 / np.sqrt((v * v).sum(-1, keepdims=True) + eps)
                dv = r * dv - v * (v * dv).sum(-1, keepdims=True) * r ** 3
            du = dv.reshape(C) * (_silu_slope(u[b, t]) if activation else 1.0)
            dfull[t:t + W] += weight.T * du
            g["weight"] += (full[t:t + W] * du).T
            g["bias"] += du
        g["state"][b] = dfull[:W - 1]
        g["x"][b, :n[b]] = dfull[W - 1:]
    return g


# ---------------------------------------------------------------------------
# Selective scan
# ---------------------------------------------------------------------------

def _steps(dt, dt_bias, use_softplus):
    v = dt + (0.0 if dt_bias is None else dt_bias[None, :, None])
    return softplus(v) if use_softplus else v


def ssm_ref(x, dt, A, B, C, D=None, dt_bias=None, S0=None, lengths=None,
            use_softplus=True, states=False):
    """(y, S_T), and with ``states`` the list of S_0 .. S_T per batch entry and
    head as [B][H] -> [T + 1, P, N]."""
    nb, H, T, P = x.shape
    G, N = B.shape[1], B.shape[3]
    n = _lengths(lengths, nb, T)
    s = _steps(dt, dt_bias, use_softplus)
    y = np.zeros((nb, H, T, P))
    S_T = np.zeros((nb, H, P, N))
    kept = [[None] * H for _ in range(nb)]
    for b in range(nb):
        for h in range(H):
            g = h // (H // G)
            S = np.zeros((P, N)) if S0 is None else S0[b, h].copy()
            every = [S.copy()]
            for t in range(n[b]):
                S = np.exp(s[b, h, t] * A[h]) * S + s[b, h, t] * np.outer(x[b, h, t], B[b, g, t])
                y[b, h, t] = S @ C[b, g, t] + (0 if D is None else D[h] * x[b, h, t])
                if states:
                    every.append(S.copy())
            S_T[b, h] = S
            kept[b][h] = every
    return (y, S_T, kept) if states else (y, S_T)


def ssm_backward_ref(x, dt, A, B, C, dy, D=None, dt_bias=None, S0=None,
                     dS_T=None, lengths=None, use_softplus=True, bound=False):
    """Gradients of sum <dy, y> + <dS_T, S_T>: dict(x, dt, A, B, C, D,
    dt_bias, S0). ``bound``: with absolute inputs, the sums of the absolute
    terms (the decay's own factor A enters by its absolute value), and beside
    them ``own`` [B,H,T], the step's part of d dt_t times the step."""
    nb, H, T, P = x.shape
    G, N = B.shape[1], B.shape[3]
    n = _lengths(lengths, nb, T)
    s = _steps(dt, dt_bias, use_softplus)
    v = dt + (0.0 if dt_bias is None else dt_bias[None, :, None])
    slope = sigmoid(v) if use_softplus else np.ones_like(v)
    _, _, S = ssm_ref(x, dt, A, B, C, D, dt_bias, S0, lengths, use_softplus, True)
    g = dict(x=np.zeros_like(x), dt=np.zeros_like(dt), A=np.zeros(H),
             B=np.zeros_like(B), C=np.zeros_like(C), D=np.zeros(H),
             dt_bias=np.zeros(H), S0=np.zeros((nb, H, P, N)))
    for b in range(nb):
        for h in range(H):
            k = h // (H // G)
            dS = np.zeros((P, N)) if dS_T is None else dS_T[b, h].copy()
            for t in reversed(range(n[b])):
                st, a = s[b, h, t], np.exp(s[b, h, t] * A[h])
                xt, bt, ct, yt = x[b, h, t], B[b, k, t], C[b, k, t], dy[b, h, t]
                g["D"][h] += yt @ xt
                g["C"][b, k, t] += S[b][h][t + 1].T @ yt
                dS = dS + np.outer(yt, ct)
                g["x"][b, h, t] = st * (dS @ bt) + (0 if D is None else D[h] * yt)
                g["B"][b, k, t] += st * (dS.T @ xt)
                da = a * (dS * S[b][h][t]).sum()       # d / d(st A)
                if bound:
                    g.setdefault("own", np.zeros_like(dt))[b, h, t] = st * (xt @ dS @ bt)
                ds = xt @ dS @ bt + (abs(A[h]) if bound else A[h]) * da
                g["A"][h] += st * da
                g["dt"][b, h, t] = ds * slope[b, h, t]
                g["dt_bias"][h] += ds * slope[b, h, t]
                dS = a * dS
            g["S0"][b, h] = dS
    return g


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

def gated_norm_ref(x, z, weight, eps=1e-6, gate_first=False):
    """x [B,H,T,D], z [B,T,H*D] or None, weight [D] or [H,D] -> [B,T,H*D]."""
    B, H, T, D = x.shape
    xt = x.transpose(0, 2, 1, 3)
    gate = 1.0 if z is None else silu(z).reshape(B, T, H, D)
    v = xt * gate if gate_first else xt
    y = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * weight
    return (y if gate_first else y * gate).reshape(B, T, H * D)


def gated_norm_backward_ref(x, z, weight, dy, eps=1e-6, gate_first=False):
    B, H, T, D = x.shape
    xt = x.transpose(0, 2, 1, 3)
    dyt = dy.reshape(B, T, H, D)
    zt = None if z is None else z.reshape(B, T, H, D)
    gate = np.ones_like(xt) if z is None else silu(zt)
    v = xt * gate if gate_first else xt
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    up = dyt if gate_first else dyt * gate
    dn = up * weight
    dv = r * dn - v * (v * dn).mean(-1, keepdims=True) * r ** 3
    dgate = dv * xt if gate_first else dyt * v * r * weight
    dw = up * v * r
    return dict(
        x=(dv * gate if gate_first else dv).transpose(0, 2, 1, 3),
        z=None if z is None else (dgate * _silu_slope(zt)).reshape(B, T, H * D),
        weight=dw.sum((0, 1)) if weight.ndim == 2 else dw.sum((0, 1, 2)))


def residual_norm_ref(x, weight, residual=None, scale=1.0, eps=1e-6):
    h = scale * x + (0.0 if residual is None else residual)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight, h


def residual_norm_backward_ref(dy, h, weight, dh=None, scale=1.0, eps=1e-6):
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    dn = dy * weight
    g = r * dn - h * (h * dn).mean(-1, keepdims=True) * r ** 3
    g = g + (0.0 if dh is None else dh)
    return dict(x=scale * g, residual=g,
                weight=(dy * h * r).reshape(-1, h.shape[-1]).sum(0))
