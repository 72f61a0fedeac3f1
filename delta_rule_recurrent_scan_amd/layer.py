"""Operators that complete a block: gated linear recurrence, norm and rotation of
queries and keys, gated feed-forward product.

Argument marshalling only, as in the package's other calls: shapes, dtypes and
devices are checked, outputs and workspaces are allocated with PyTorch on the
inputs' device, and the C ABI (include/osdn.h) is called with raw pointers on
that device's current stream. Every call runs in the library's HIP kernels.
"""

import ctypes

import torch

from . import _DTYPE_CODE, load_library
from . import _check as _check_slow
from .mixer import _begin, _call, _check, _ptr, _required
from .mixer import _workspace as _any_workspace

__all__ = ["glr_forward", "glr_decode", "glr_backward",
           "glr_forward_workspace_bytes", "glr_backward_workspace_bytes",
           "qk_rotary_forward", "qk_rotary_backward",
           "qk_rotary_backward_workspace_bytes", "gated_ffn_forward",
           "gated_ffn_backward", "gated_ffn_forward_workspace_bytes",
           "gated_ffn_backward_workspace_bytes"]

_P, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_Z, _L = ctypes.c_size_t, ctypes.c_longlong
_GLR = [_I] * 4 + [_P, _L, _L] * 3
_QK = [_P, _L, _L, _P, _L, _L, _P, _P, _I, _F, _P, _I, _P, _P]

# name: (argument types, result type)
SIGNATURES = {
    "glr_forward_workspace_bytes": ([_I] * 3, _Z),
    "glr_forward": (_GLR + [_P, _P, _P, _I, _P, _P, _P, _P, _Z, _P], _I),
    "glr_decode": (_GLR + [_P, _P, _I, _P, _P, _P], _I),
    "glr_backward_workspace_bytes": ([_I] * 4, _Z),
    "glr_backward": (_GLR + [_P, _P, _P, _I] + [_P] * 9 + [_Z, _P], _I),
    "qk_rotary_forward": ([_I] * 7 + _QK + [_P, _P, _P], _I),
    "qk_rotary_backward_workspace_bytes": ([_I] * 3, _Z),
    "qk_rotary_backward": ([_I] * 8 + _QK + [_P] * 7 + [_Z, _P], _I),
    "gated_ffn_forward_workspace_bytes": ([_L, _I, _I, _I], _Z),
    "gated_ffn_forward": ([_L, _I, _I, _I, _P, _L, _P, _P, _I, _P, _P, _P, _P,
                           _Z, _P], _I),
    "gated_ffn_backward_workspace_bytes": ([_L, _I, _I, _I], _Z),
    "gated_ffn_backward": ([_L, _I, _I, _I, _P, _L, _P, _P, _P, _P, _I, _P, _P,
                            _P, _P, _P, _Z, _P], _I),
}

# OSDN_GLR_INTERVAL: tokens between the states that a forward leaves
GLR_INTERVAL = 16
_NORM = {"none": 0, "rms": 1, "l2": 2}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def bind(L):
    """Declare the C functions' argument types on the loaded library."""
    for name, (args, res) in SIGNATURES.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


def _workspace(ws, need, dev):
    """(pointer, bytes, tensor) of a call's workspace; none is made where none is
    needed (a single-token call would spend a fifth of its time on it)."""
    if ws is None and need == 0:
        return None, 0, None
    ws = _any_workspace(ws, need, dev)
    return ws.data_ptr(), ws.numel(), ws


def _rows(t, name, shape, dt, dev):
    """(pointer, batch stride, token stride) of token rows [B,T,C] with any strides over
    tokens and batch entries."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dt
            and t.device == dev):
        if t is None:
            raise ValueError("%s is required" % name)
        _check_slow(t, name, shape, dt, dev)
    bs, ts, cs = t.stride()
    if cs != 1 and shape[2] > 1 and t.numel():
        raise ValueError("%s must be contiguous along its channels" % name)
    # strides of dimensions of one entry are never used and may be anything
    return t.data_ptr(), bs if shape[0] > 1 else 0, ts if shape[1] > 1 else 0


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------

def _glr_checks(x, r, A, i):
    L, code, dev = _begin(x, "x")
    shape, dt = x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError("x must be [B, T, C]")
    if A is None:
        raise ValueError("A is required")
    _check(A, "A", shape[2:], torch.float32, dev)
    return L, dev, shape, (
        *shape, code, *_rows(x, "x", shape, dt, dev), *_rows(r, "r", shape, dt, dev),
        *((None, 0, 0) if i is None else _rows(i, "i", shape, dt, dev)), A.data_ptr())


def glr_forward_workspace_bytes(B, T, C):
    return int(load_library().glr_forward_workspace_bytes(B, T, C))


def glr_forward(x, r, A, i=None, h0=None, lengths=None, normalize=True,
                save=False, out=None, workspace=None):
    """Gated linear recurrence, one decay per channel: returns (y [B,T,C], h_T
    [B,C] fp32, states).

    x, r, i: [B,T,C] (one dtype, fp32 or bf16), contiguous along the channels
    (channel ranges of one wider projection are read in place; i None: no input
    gate); A: [C] fp32, finite, <= 0; h0: [B,C] fp32 (None: zeros); lengths: [B] int32 of
    a padded batch. With a = exp(A sigmoid(r)), h <- a h + m sigmoid(i) x and
    y = h, where m = sqrt(1 - a^2), or 1 with ``normalize=False``. With ``save``,
    states [B, ceil(T / 16), C] fp32 are h before tokens 0, 16, 32, ... for
    glr_backward; otherwise None. ``out`` may pass preallocated (y, h_T, states)
    (any of them None to skip it) and ``workspace`` a uint8 device buffer of
    glr_forward_workspace_bytes()."""
    L, dev, (B, T, C), args = _glr_checks(x, r, A, i)
    f32 = torch.float32
    _check(h0, "h0", (B, C), f32, dev)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    kept = (B, -(-T // GLR_INTERVAL), C)
    if out is None:
        y = torch.empty((B, T, C), dtype=x.dtype, device=dev)
        h_T = torch.empty((B, C), dtype=f32, device=dev)
        states = torch.empty(kept, dtype=f32, device=dev) if save else None
    else:
        y, h_T, states = out
        _check(y, "y", (B, T, C), x.dtype, dev)
        _check(h_T, "h_T", (B, C), f32, dev)
        _check(states, "states", kept, f32, dev)
    wp, wn, ws = _workspace(workspace, L.glr_forward_workspace_bytes(B, T, C), dev)
    _call(L.glr_forward, "glr_forward", dev, *args, _ptr(h0), _ptr(lengths),
          int(normalize), _ptr(y), _ptr(h_T), _ptr(states), wp, wn)
    return y, h_T, states


def glr_decode(x, r, A, h, i=None, normalize=True, out=None, h_out=None):
    """T tokens (usually 1) of glr_forward with the state h ([B,C] fp32) updated
    IN PLACE, or written to ``h_out`` with h left as it was: returns y [B,T,C]."""
    if h is None:
        raise ValueError("h is required")
    L, dev, (B, T, C), args = _glr_checks(x, r, A, i)
    _check(h, "h", (B, C), torch.float32, dev)
    ho, y = h, out
    if h_out is not None:
        ho = h_out
        _check(ho, "h_out", (B, C), torch.float32, dev)
    if out is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _check(y, "y", (B, T, C), x.dtype, dev)
    _call(L.glr_decode, "glr_decode", dev, *args, h.data_ptr(), int(normalize),
          y.data_ptr(), ho.data_ptr())
    return y


def glr_backward_workspace_bytes(B, T, C, have_states=True):
    return int(load_library().glr_backward_workspace_bytes(B, T, C,
                                                           int(have_states)))


def glr_backward(x, r, A, dy, i=None, h0=None, dh_T=None, lengths=None,
                 normalize=True, states=None, out=None, workspace=None):
    """Backward of glr_forward: the gradient of sum <dy, y> + <dh_T, h_T>, dy
    [B,T,C] in the dtype of x and dh_T [B,C] fp32 (None: zero). ``states`` are
    those of glr_forward(..., save=True); None forms them here from h0 (one more
    pass over x, r and i). Returns a dict x, r, i [B,T,C] in the dtype of x (i None
    without an input gate), A [C] and h0 [B,C] fp32; ``out`` may pass such a dict
    preallocated (h0 may be None to skip it) and ``workspace`` a uint8 device buffer
    of glr_backward_workspace_bytes()."""
    L, dev, (B, T, C), args = _glr_checks(x, r, A, i)
    f32 = torch.float32
    _check(h0, "h0", (B, C), f32, dev)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    _check(states, "states", (B, -(-T // GLR_INTERVAL), C), f32, dev)
    _check(dy, "dy", (B, T, C), x.dtype, dev)
    _check(dh_T, "dh_T", (B, C), f32, dev)

    def rows():
        return torch.empty((B, T, C), dtype=x.dtype, device=dev)
    g = out if out is not None else dict(
        x=rows(), r=rows(), i=None if i is None else rows(),
        A=torch.empty((C,), dtype=f32, device=dev),
        h0=torch.empty((B, C), dtype=f32, device=dev))
    _required(g, ("x", "r", "A") + (() if i is None else ("i",)))
    for n in ("x", "r") + (() if i is None else ("i",)):
        _check(g[n], "out[%s]" % n, (B, T, C), x.dtype, dev)
    _check(g["A"], "out[A]", (C,), f32, dev)
    _check(g.get("h0"), "out[h0]", (B, C), f32, dev)
    wp, wn, ws = _workspace(workspace, L.glr_backward_workspace_bytes(
        B, T, C, int(states is not None)), dev)
    _call(L.glr_backward, "glr_backward", dev, *args, _ptr(h0), _ptr(lengths),
          int(normalize), _ptr(states), _ptr(dy), _ptr(dh_T), _ptr(g["x"]),
          _ptr(g["r"]), _ptr(None if i is None else g["i"]), _ptr(g["A"]),
          _ptr(g.get("h0")), wp, wn)
    return g


# ---------------------------------------------------------------------------
# Norm and rotation of queries and keys
# ---------------------------------------------------------------------------

def _qk_checks(q, k, head_dim, inv_freq, q_weight, k_weight, positions, lengths,
               norm, interleaved, eps):
    lead = q if q is not None else k
    L, code, dev = _begin(lead, "q")
    if lead.dim() != 3:
        raise ValueError("q and k must be [B, T, H * head_dim]")
    B, T = lead.shape[:2]
    D = int(head_dim)
    if norm not in _NORM:
        raise ValueError("norm must be one of %s" % sorted(_NORM))
    dt, f32 = lead.dtype, torch.float32
    heads, rows = [], ()
    for t, name in ((q, "q"), (k, "k")):
        if t is None:
            heads.append(0)
            rows += (None, 0, 0)
            continue
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError("%s must be [B, T, H * head_dim]" % name)
        C = t.shape[2]
        if D < 1 or C % D:
            raise ValueError("head_dim %d does not divide the %d channels" % (D, C))
        heads.append(C // D)
        rows += _rows(t, name, (B, T, C), dt, dev)
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot / 2]")
        rot = 2 * inv_freq.shape[0]
        _check(inv_freq, "inv_freq", (rot // 2,), f32, dev)
    if q_weight is not None:
        _check(q_weight, "q_weight", (D,), f32, dev)
    if k_weight is not None:
        _check(k_weight, "k_weight", (D,), f32, dev)
    if positions is not None:
        _check(positions, "positions", (B, T), torch.int32, dev)
    if lengths is not None:
        _check(lengths, "lengths", (B,), torch.int32, dev)
    dims = (B, T, heads[0], heads[1], D)
    args = rows + (_ptr(q_weight), _ptr(k_weight), _NORM[norm], float(eps),
                   _ptr(inv_freq), int(interleaved), _ptr(positions),
                   _ptr(lengths))
    return L, code, dev, lead.dtype, dims, rot, args


def qk_rotary_forward(q, k, head_dim, inv_freq=None, q_weight=None, k_weight=None,
                      positions=None, lengths=None, norm="rms", interleaved=False,
                      eps=1e-6, out=None):
    """Norm of each query's and key's row and the rotation of its position, from
    token rows to the heads that the recurrences read: returns (q [B,Hq,T,D], k
    [B,Hk,T,D]).

    q: [B,T,Hq*D], k: [B,T,Hk*D] (one dtype, fp32 or bf16; either may be None),
    contiguous along the channels (channel ranges of one projection are read in
    place); head_dim: D in {32, 64, 128}; norm: "rms", "l2" or "none"; q_weight,
    k_weight: [D] fp32 (None: ones); inv_freq: [rot / 2] fp32 (None: no rotation),
    rot a multiple of 16 up to D: pair j turns by position * inv_freq[j]. Pairs are
    channels (j, j + rot / 2), or (2 j, 2 j + 1) with ``interleaved``. positions:
    [B,T] int32 (None: 0 .. T - 1); lengths: [B] int32 of a padded batch. ``out``
    may pass preallocated (q, k)."""
    L, code, dev, dt, (B, T, Hq, Hk, D), rot, args = _qk_checks(
        q, k, head_dim, inv_freq, q_weight, k_weight, positions, lengths, norm,
        interleaved, eps)
    if out is None:
        yq = None if q is None else q.new_empty((B, Hq, T, D))
        yk = None if k is None else k.new_empty((B, Hk, T, D))
    else:
        yq, yk = out
        _check(yq, "out[0]", (B, Hq, T, D), dt, dev)
        _check(yk, "out[1]", (B, Hk, T, D), dt, dev)
    _call(L.qk_rotary_forward, "qk_rotary_forward", dev, B, T, Hq, Hk, D, rot, code,
          *args, _ptr(yq), _ptr(yk))
    return yq, yk


def qk_rotary_backward_workspace_bytes(B, T, D):
    return int(load_library().qk_rotary_backward_workspace_bytes(B, T, D))


def qk_rotary_backward(q, k, dq, dk, head_dim, inv_freq=None, q_weight=None,
                       k_weight=None, positions=None, lengths=None, norm="rms",
                       interleaved=False, eps=1e-6, out=None, workspace=None):
    """Backward of qk_rotary_forward: dq [B,Hq,T,D], dk [B,Hk,T,D] in the dtype of
    q and k, or both fp32 (what the recurrences' backward returns). Returns a dict q
    [B,T,Hq*D], k [B,T,Hk*D] in the dtype of q and k (None for an input that is None)
    and q_weight, k_weight [D] fp32 (None without that weight); ``out`` may pass such
    a dict preallocated."""
    L, code, dev, dt, (B, T, Hq, Hk, D), rot, args = _qk_checks(
        q, k, head_dim, inv_freq, q_weight, k_weight, positions, lengths, norm,
        interleaved, eps)
    f32 = torch.float32
    lead = dq if q is not None else dk
    if not isinstance(lead, torch.Tensor) or lead.dtype not in (dt, f32):
        raise ValueError("dq and dk must have the dtype of q and k or float32")
    if q is not None:
        _check(dq, "dq", (B, Hq, T, D), lead.dtype, dev)
    if k is not None:
        if dk is None:
            raise ValueError("dk is required with k")
        _check(dk, "dk", (B, Hk, T, D), lead.dtype, dev)
    shapes = dict(q=((B, T, Hq * D), dt, q), k=((B, T, Hk * D), dt, k),
                  q_weight=((D,), f32, q_weight), k_weight=((D,), f32, k_weight))
    g = out if out is not None else {
        n: None if t is None else torch.empty(s, dtype=d, device=dev)
        for n, (s, d, t) in shapes.items()}
    _required(g, [n for n, (s, d, t) in shapes.items() if t is not None])
    for n, (s, d, t) in shapes.items():
        _check(g.get(n) if t is not None else None, "out[%s]" % n, s, d, dev)
    wp, wn, ws = _workspace(workspace, L.qk_rotary_backward_workspace_bytes(B, T, D), dev)

    def to(n):
        return _ptr(g[n]) if shapes[n][2] is not None else None
    _call(L.qk_rotary_backward, "qk_rotary_backward", dev, B, T, Hq, Hk, D, rot,
          code, _DTYPE_CODE[lead.dtype], *args,
          _ptr(dq) if q is not None else None, _ptr(dk) if k is not None else None,
          to("q"), to("k"), to("q_weight"), to("k_weight"), wp, wn)
    return g


# ---------------------------------------------------------------------------
# Gated feed-forward product
# ---------------------------------------------------------------------------

def _ffn_checks(x, w_gate, w_up, activation):
    L, code, dev = _begin(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have a channel dimension")
    if activation not in _ACT:
        raise ValueError("activation must be one of %s" % sorted(_ACT))
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise ValueError("w_gate must be [F, C]")
    C, F = x.shape[-1], w_gate.shape[0]
    R = 1
    for n in x.shape[:-1]:
        R *= n
    stride = C
    if R and C and not x.is_contiguous():
        # any rows whose leading dimensions lie one row stride apart
        want = None
        for n, s in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
            if n == 1:
                continue
            if want is None:
                stride = want = s
            if s != want:
                raise ValueError("x must have its rows one stride apart")
            want = s * n
        if C > 1 and x.stride(-1) != 1:
            raise ValueError("x must be contiguous along its channels")
    _check(w_gate, "w_gate", (F, C), x.dtype, dev)
    if w_up is None:
        raise ValueError("w_up is required")
    _check(w_up, "w_up", (F, C), x.dtype, dev)
    return L, code, dev, (R, C, F), (R, C, F, code, _ptr(x), stride, _ptr(w_gate),
                                     _ptr(w_up))


def gated_ffn_forward_workspace_bytes(R, C, F, dtype):
    return int(load_library().gated_ffn_forward_workspace_bytes(
        R, C, F, _DTYPE_CODE[dtype]))


def gated_ffn_forward(x, w_gate, w_up, activation="silu", save=False, out=None,
                      workspace=None):
    """Gated feed-forward product h = act(x w_gate^T) * (x w_up^T) in one kernel:
    returns (h [...,F], gate, up).

    x: [...,C], rows one stride apart (a channel range of wider rows is read in
    place); w_gate, w_up: [F,C], all of one dtype, fp32 or bf16; activation:
    "silu", "gelu" (error function) or "gelu_tanh". With ``save``, gate = x
    w_gate^T and up = x w_up^T [...,F] are kept for gated_ffn_backward; otherwise
    they are None. h is formed from the 32-bit sums. ``out`` may pass preallocated
    (h, gate, up) (gate and up both None to skip them) and ``workspace`` a uint8
    device buffer of gated_ffn_forward_workspace_bytes()."""
    L, code, dev, (R, C, F), args = _ffn_checks(x, w_gate, w_up, activation)
    shape = tuple(x.shape[:-1]) + (F,)
    if out is None:
        h = x.new_empty(shape)
        gate, up = ((torch.empty_like(h), torch.empty_like(h)) if save
                    else (None, None))
    else:
        h, gate, up = out
        for t, n in ((h, "h"), (gate, "gate"), (up, "up")):
            _check(t, n, shape, x.dtype, dev)
    wp, wn, ws = _workspace(workspace, L.gated_ffn_forward_workspace_bytes(R, C, F, code),
                    dev)
    _call(L.gated_ffn_forward, "gated_ffn_forward", dev, *args, _ACT[activation],
          _ptr(h), _ptr(gate), _ptr(up), wp, wn)
    return h, gate, up


def gated_ffn_backward_workspace_bytes(R, C, F, dtype):
    return int(load_library().gated_ffn_backward_workspace_bytes(
        R, C, F, _DTYPE_CODE[dtype]))


def gated_ffn_backward(x, w_gate, w_up, gate, up, dh, activation="silu", out=None,
                       workspace=None):
    """Backward of gated_ffn_forward from the gate and up it kept: dh [...,F] in
    the dtype of x. Returns a dict x [...,C], w_gate, w_up [F,C] in that dtype;
    ``out`` may pass such a dict preallocated and ``workspace`` a uint8 device
    buffer of gated_ffn_backward_workspace_bytes()."""
    L, code, dev, (R, C, F), args = _ffn_checks(x, w_gate, w_up, activation)
    dt, shape = x.dtype, tuple(x.shape[:-1]) + (F,)
    for t, n in ((gate, "gate"), (up, "up"), (dh, "dh")):
        if t is None:
            raise ValueError("%s is required" % n)
        _check(t, n, shape, dt, dev)
    g = out if out is not None else dict(
        x=torch.empty(x.shape, dtype=dt, device=dev),
        w_gate=torch.empty((F, C), dtype=dt, device=dev),
        w_up=torch.empty((F, C), dtype=dt, device=dev))
    _required(g, ("x", "w_gate", "w_up"))
    _check(g["x"], "out[x]", tuple(x.shape), dt, dev)
    _check(g["w_gate"], "out[w_gate]", (F, C), dt, dev)
    _check(g["w_up"], "out[w_up]", (F, C), dt, dev)
    wp, wn, ws = _workspace(workspace, L.gated_ffn_backward_workspace_bytes(R, C, F, code),
                    dev)
    _call(L.gated_ffn_backward, "gated_ffn_backward", dev, *args, _ptr(gate),
          _ptr(up), _ACT[activation], _ptr(dh), _ptr(g["x"]), _ptr(g["w_gate"]),
          _ptr(g["w_up"]), wp, wn)
    return g
