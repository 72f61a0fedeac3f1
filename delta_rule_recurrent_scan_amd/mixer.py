"""Operators around the recurrences: short causal convolution, selective state
space scan, gated head norm and residual norm.

Argument marshalling only, as in the package's other calls: shapes, dtypes and
devices are checked, outputs and workspaces are allocated with PyTorch on the
inputs' device, and the C ABI (include/osdn.h) is called with raw pointers on
that device's current stream. Every call runs in the library's HIP kernels.
"""

import ctypes

import torch

from . import _DTYPE_CODE, OsdnError, load_library
from . import _check as _check_slow

__all__ = ["short_conv_forward", "short_conv_decode", "short_conv_backward",
           "short_conv_backward_workspace_bytes", "ssm_forward", "ssm_decode",
           "ssm_backward", "ssm_forward_workspace_bytes",
           "ssm_backward_workspace_bytes", "gated_norm_forward",
           "gated_norm_backward", "gated_norm_backward_workspace_bytes",
           "residual_norm_forward", "residual_norm_backward",
           "residual_norm_backward_workspace_bytes"]

_P, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_Z, _L = ctypes.c_size_t, ctypes.c_longlong

# name: (argument types, result type)
SIGNATURES = {
    "short_conv_forward": ([_I] * 6 + [_P, _L, _L, _P, _P, _P, _P, _I, _I, _F,
                                       _P, _P, _P], _I),
    "short_conv_decode": ([_I] * 6 + [_P, _L, _L, _P, _P, _P, _I, _I, _F, _P,
                                      _P, _P], _I),
    "short_conv_backward_workspace_bytes": ([_I] * 5, _Z),
    "short_conv_backward": ([_I] * 7 + [_P, _L, _L, _P, _P, _P, _P, _I, _I, _F,
                                        _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "ssm_forward_workspace_bytes": ([_I] * 7, _Z),
    "ssm_forward": ([_I] * 7 + [_P] * 7 + [_I, _P, _P, _P, _P, _P, _Z, _P], _I),
    "ssm_decode": ([_I] * 7 + [_P] * 7 + [_I, _P, _P, _P, _P], _I),
    "ssm_backward_workspace_bytes": ([_I] * 7, _Z),
    "ssm_backward": ([_I] * 7 + [_P] * 7 + [_I] + [_P] * 13 + [_Z, _P], _I),
    "gated_norm_forward": ([_I] * 5 + [_P, _P, _L, _L, _P, _I, _F, _I, _P, _P],
                           _I),
    "gated_norm_backward_workspace_bytes": ([_I] * 4, _Z),
    "gated_norm_backward": ([_I] * 5 + [_P, _P, _L, _L, _P, _I, _F, _I, _P, _P,
                                        _P, _P, _P, _Z, _P], _I),
    "residual_norm_forward": ([_L, _I, _I, _I, _P, _P, _F, _P, _F, _P, _P, _P],
                              _I),
    "residual_norm_backward_workspace_bytes": ([_L, _I], _Z),
    "residual_norm_backward": ([_L, _I, _I, _I, _P, _P, _P, _F, _P, _F, _P, _P,
                                _P, _P, _Z, _P], _I),
}


def bind(L):
    """Declare the C functions' argument types on the loaded library."""
    for name, (args, res) in SIGNATURES.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# The current stream's handle without the Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _begin(t, name):
    """Library, dtype code and device of a call whose leading tensor is t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DTYPE_CODE:
        raise ValueError("%s must be float32 or bfloat16" % name)
    if t.device.type != "cuda":
        raise ValueError("inputs must be on a HIP device")
    return load_library(), _DTYPE_CODE[t.dtype], t.device


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, shape, dtype, device):
    """A tensor of this shape, dtype and device, contiguous (None passes). The
    attributes are read once here; what is wrong is found out only then (a
    single-token call spends as long on its checks as on its kernel)."""
    if t is None or (isinstance(t, torch.Tensor) and t.shape == shape
                     and t.dtype is dtype and t.device == device
                     and t.is_contiguous()):
        return
    _check_slow(t, name, shape, dtype, device)


def _call(fn, name, dev, *args):
    """The call on dev's current stream, with dev current while it is made (a
    launch goes to the current device)."""
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc != 0:
        raise OsdnError(rc, name)


def _rows(t, name, B, T, C, dtype, dev):
    """Token rows [B,T,C] with any strides over tokens and batch entries:
    checks them and returns (batch stride, token stride)."""
    if not (isinstance(t, torch.Tensor) and t.device == dev and t.dtype is dtype
            and t.shape == (B, T, C)):
        _check_slow(t, name, (B, T, C), dtype, dev)
    if C > 1 and t.numel() and t.stride(2) != 1:
        raise ValueError("%s must be contiguous along its channels" % name)
    # strides of dimensions of one entry are never used and may be anything
    return (t.stride(0) if B > 1 else 0), (t.stride(1) if T > 1 else 0)


def _workspace(ws, need, dev):
    if ws is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(ws, "workspace", (ws.numel(),), torch.uint8, dev)
    return ws


def _required(out, names):
    for n in names:
        if out.get(n) is None:
            raise ValueError("out must hold a tensor for %s" % n)
    return out


# ---------------------------------------------------------------------------
# Short causal convolution
# ---------------------------------------------------------------------------

def _conv_checks(x, weight, bias, state, head_dim):
    L, code, dev = _begin(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    D = C if head_dim is None else int(head_dim)
    if D < 1 or C % D:
        raise ValueError("head_dim %d does not divide the %d channels" % (D, C))
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    bs, ts = _rows(x, "x", B, T, C, x.dtype, dev)
    _check(weight, "weight", (C, W), torch.float32, dev)
    _check(bias, "bias", (C,), torch.float32, dev)
    _check(state, "state", (B, W - 1, C), x.dtype, dev)
    return L, code, dev, (B, T, C // D, D, W), (bs, ts)


def short_conv_forward(x, weight, bias=None, state=None, lengths=None,
                       head_dim=None, activation=True, l2norm=False, eps=1e-6,
                       out=None):
    """Short causal depthwise convolution with SiLU and an optional L2 norm of
    each head's row: returns (y [B,H,T,D], state_T [B,W-1,C]).

    x: [B,T,C] fp32 or bf16, contiguous along the channels (a channel slice of
    a wider tensor is read in place); weight: [C,W] fp32, W in {2, 3, 4};
    bias: [C] fp32 (None: zeros); state: [B,W-1,C], the inputs before the
    first (None: zeros); lengths: [B] int32 of a padded batch (None: T each);
    head_dim: D, with H = C / D (None: one head of all channels, i.e. token
    rows). y_t = silu(bias + sum_k weight[:,k] x_{t-W+1+k}), divided per head
    by sqrt(sum y^2 + eps) with ``l2norm`` (D in {32, 64, 128}). ``out`` may
    pass preallocated (y, state_T) (state_T may be None to skip it).
    """
    L, code, dev, (B, T, H, D, W), (bs, ts) = _conv_checks(x, weight, bias,
                                                           state, head_dim)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    if out is None:
        y = torch.empty((B, H, T, D), dtype=x.dtype, device=dev)
        state_T = torch.empty((B, W - 1, H * D), dtype=x.dtype, device=dev)
    else:
        y, state_T = out
    _check(y, "y", (B, H, T, D), x.dtype, dev)
    _check(state_T, "state_T", (B, W - 1, H * D), x.dtype, dev)
    _call(L.short_conv_forward, "short_conv_forward", dev, B, T, H, D, W, code,
          _ptr(x), bs, ts, _ptr(weight), _ptr(bias), _ptr(state),
          _ptr(lengths), int(activation), int(l2norm), float(eps), _ptr(y),
          _ptr(state_T))
    return y, state_T


def short_conv_decode(x, weight, state, bias=None, head_dim=None,
                      activation=True, l2norm=False, eps=1e-6, out=None,
                      state_out=None):
    """T tokens (usually 1) of short_conv_forward with the state updated IN
    PLACE, or written to ``state_out`` with ``state`` left as it was: returns
    y [B,H,T,D]."""
    if state is None:
        raise ValueError("state is required")
    L, code, dev, (B, T, H, D, W), (bs, ts) = _conv_checks(x, weight, bias,
                                                           state, head_dim)
    y = (torch.empty((B, H, T, D), dtype=x.dtype, device=dev) if out is None
         else out)
    so = state if state_out is None else state_out
    _check(y, "y", (B, H, T, D), x.dtype, dev)
    _check(so, "state_out", (B, W - 1, H * D), x.dtype, dev)
    _call(L.short_conv_decode, "short_conv_decode", dev, B, T, H, D, W, code,
          _ptr(x), bs, ts, _ptr(weight), _ptr(bias), _ptr(state),
          int(activation), int(l2norm), float(eps), _ptr(y), _ptr(so))
    return y


def short_conv_backward_workspace_bytes(B, T, H, D, W):
    return int(load_library().short_conv_backward_workspace_bytes(B, T, H, D, W))


def short_conv_backward(x, weight, dy, bias=None, state=None, lengths=None,
                        head_dim=None, activation=True, l2norm=False, eps=1e-6,
                        dstate_T=None, out=None, workspace=None):
    """Backward of short_conv_forward: the gradient of sum <dy, y> +
    <dstate_T, state_T>. dy: [B,H,T,D] in the dtype of x, or fp32 (what the
    recurrences' backward returns); dstate_T: [B,W-1,C] (None: zero). Returns
    a dict x [B,T,C], state [B,W-1,C] (dtype of x), weight [C,W], bias [C]
    (fp32); ``out`` may pass such a dict preallocated."""
    L, code, dev, (B, T, H, D, W), (bs, ts) = _conv_checks(x, weight, bias,
                                                           state, head_dim)
    C, dt, f32 = H * D, x.dtype, torch.float32
    _check(lengths, "lengths", (B,), torch.int32, dev)
    if dy.dtype not in (dt, f32):
        raise ValueError("dy must have the dtype of x or float32")
    _check(dy, "dy", (B, H, T, D), dy.dtype, dev)
    _check(dstate_T, "dstate_T", (B, W - 1, C), dt, dev)
    g = out if out is not None else dict(
        x=torch.empty((B, T, C), dtype=dt, device=dev),
        weight=torch.empty((C, W), dtype=f32, device=dev),
        bias=torch.empty((C,), dtype=f32, device=dev),
        state=torch.empty((B, W - 1, C), dtype=dt, device=dev))
    _required(g, ("x", "weight", "bias", "state"))
    _check(g["x"], "out[x]", (B, T, C), dt, dev)
    _check(g["weight"], "out[weight]", (C, W), f32, dev)
    _check(g["bias"], "out[bias]", (C,), f32, dev)
    _check(g["state"], "out[state]", (B, W - 1, C), dt, dev)
    ws = _workspace(workspace, L.short_conv_backward_workspace_bytes(
        B, T, H, D, W), dev)
    _call(L.short_conv_backward, "short_conv_backward", dev, B, T, H, D, W,
          code, _DTYPE_CODE[dy.dtype], _ptr(x), bs, ts, _ptr(weight),
          _ptr(bias), _ptr(state), _ptr(lengths), int(activation), int(l2norm),
          float(eps), _ptr(dy), _ptr(dstate_T), _ptr(g["x"]), _ptr(g["state"]),
          _ptr(g["weight"]), _ptr(g["bias"]), _ptr(ws), ws.numel())
    return g


# ---------------------------------------------------------------------------
# Selective scan
# ---------------------------------------------------------------------------

def _ssm_checks(x, dt, A, B, C, D, dt_bias):
    L, code, dev = _begin(x, "x")
    f32 = torch.float32
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [B, H, T, P] and B [B, G, T, N]")
    nb, H, T, P = x.shape
    G, N = B.shape[1], B.shape[3]
    if H and (G == 0 or H % G):
        raise ValueError("%d groups do not divide %d heads" % (G, H))
    _check(x, "x", (nb, H, T, P), x.dtype, dev)
    _check(dt, "dt", (nb, H, T), f32, dev)
    _check(A, "A", (H,), f32, dev)
    _check(B, "B", (nb, G, T, N), x.dtype, dev)
    _check(C, "C", (nb, G, T, N), x.dtype, dev)
    _check(D, "D", (H,), f32, dev)
    _check(dt_bias, "dt_bias", (H,), f32, dev)
    return L, code, dev, (nb, H, G, T, P, N)


def ssm_forward_workspace_bytes(B, H, G, T, P, N, dtype):
    return int(load_library().ssm_forward_workspace_bytes(
        B, H, G, T, P, N, _DTYPE_CODE[dtype]))


def ssm_forward(x, dt, A, B, C, D=None, dt_bias=None, S0=None, lengths=None,
                softplus=True, out=None, workspace=None):
    """Selective state space scan: returns (y [B,H,T,P], S_T [B,H,P,N] fp32).

    x: [B,H,T,P], B, C: [B,G,T,N] (one dtype, fp32 or bf16; G divides H, and
    H / G heads share a group's keys B and queries C); dt: [B,H,T] fp32; A
    [H] fp32 (negative: a decay), D, dt_bias [H] fp32 (None: zeros); S0
    [B,H,P,N] fp32 (None: zeros); lengths [B] int32 of a padded batch. With
    s = softplus(dt + dt_bias) (``softplus=False``: the sum itself),
    S <- exp(s A) S + s x B^T and y = S C + D x. P, N in {32, 64, 128}. A dt of
    -inf or the lowest fp32 value switches its token off.
    ``out`` may pass preallocated (y, S_T) (S_T may be None to skip it, or S0
    itself) and ``workspace`` a uint8 device buffer of
    ssm_forward_workspace_bytes().
    """
    L, code, dev, (nb, H, G, T, P, N) = _ssm_checks(x, dt, A, B, C, D, dt_bias)
    _check(S0, "S0", (nb, H, P, N), torch.float32, dev)
    _check(lengths, "lengths", (nb,), torch.int32, dev)
    if out is None:
        y = torch.empty((nb, H, T, P), dtype=x.dtype, device=dev)
        S_T = torch.empty((nb, H, P, N), dtype=torch.float32, device=dev)
    else:
        y, S_T = out
    _check(y, "y", (nb, H, T, P), x.dtype, dev)
    _check(S_T, "S_T", (nb, H, P, N), torch.float32, dev)
    ws = _workspace(workspace, L.ssm_forward_workspace_bytes(
        nb, H, G, T, P, N, code), dev)
    _call(L.ssm_forward, "ssm_forward", dev, nb, H, G, T, P, N, code, _ptr(x),
          _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
          int(softplus), _ptr(S0), _ptr(lengths), _ptr(y), _ptr(S_T), _ptr(ws),
          ws.numel())
    return y, S_T


def ssm_decode(x, dt, A, B, C, S, D=None, dt_bias=None, softplus=True, out=None,
               S_out=None):
    """T tokens (usually 1) of ssm_forward with the state S ([B,H,P,N] fp32)
    updated IN PLACE, or written to ``S_out`` with S left as it was: returns y
    [B,H,T,P]."""
    if S is None:
        raise ValueError("S is required")
    L, code, dev, (nb, H, G, T, P, N) = _ssm_checks(x, dt, A, B, C, D, dt_bias)
    so = S if S_out is None else S_out
    _check(S, "S", (nb, H, P, N), torch.float32, dev)
    _check(so, "S_out", (nb, H, P, N), torch.float32, dev)
    y = (torch.empty((nb, H, T, P), dtype=x.dtype, device=dev) if out is None
         else out)
    _check(y, "y", (nb, H, T, P), x.dtype, dev)
    _call(L.ssm_decode, "ssm_decode", dev, nb, H, G, T, P, N, code, _ptr(x),
          _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
          int(softplus), _ptr(S), _ptr(y), _ptr(so))
    return y


def ssm_backward_workspace_bytes(B, H, G, T, P, N, dtype):
    return int(load_library().ssm_backward_workspace_bytes(
        B, H, G, T, P, N, _DTYPE_CODE[dtype]))


def ssm_backward(x, dt, A, B, C, dy, D=None, dt_bias=None, S0=None, dS_T=None,
                 lengths=None, softplus=True, out=None, workspace=None):
    """Backward of ssm_forward: the gradient of sum <dy, y> + <dS_T, S_T>, dy
    [B,H,T,P] in the dtype of x and dS_T [B,H,P,N] fp32 (None: zero). Returns
    a dict x, B, C (in the dtype of x; B and C summed over their group's
    heads), dt [B,H,T] (of the raw dt), A, D, dt_bias [H] and S0 [B,H,P,N]
    (fp32). ``out`` may pass such a dict preallocated (D, dt_bias and S0 may be
    None to skip them) and ``workspace`` a uint8 device buffer of
    ssm_backward_workspace_bytes()."""
    L, code, dev, (nb, H, G, T, P, N) = _ssm_checks(x, dt, A, B, C, D, dt_bias)
    f32 = torch.float32
    _check(S0, "S0", (nb, H, P, N), f32, dev)
    _check(lengths, "lengths", (nb,), torch.int32, dev)
    _check(dy, "dy", (nb, H, T, P), x.dtype, dev)
    _check(dS_T, "dS_T", (nb, H, P, N), f32, dev)
    shapes = dict(x=((nb, H, T, P), x.dtype), dt=((nb, H, T), f32),
                  A=((H,), f32), B=((nb, G, T, N), x.dtype),
                  C=((nb, G, T, N), x.dtype), D=((H,), f32),
                  dt_bias=((H,), f32), S0=((nb, H, P, N), f32))
    g = out if out is not None else {
        n: torch.empty(s, dtype=d, device=dev) for n, (s, d) in shapes.items()}
    _required(g, ("x", "dt", "A", "B", "C"))
    for n, (s, d) in shapes.items():
        _check(g.get(n), "out[%s]" % n, s, d, dev)
    ws = _workspace(workspace, L.ssm_backward_workspace_bytes(
        nb, H, G, T, P, N, code), dev)
    _call(L.ssm_backward, "ssm_backward", dev, nb, H, G, T, P, N, code, _ptr(x),
          _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
          int(softplus), _ptr(S0), _ptr(lengths), _ptr(dy), _ptr(dS_T),
          _ptr(g["x"]), _ptr(g["dt"]), _ptr(g["A"]), _ptr(g["B"]), _ptr(g["C"]),
          _ptr(g.get("D")), _ptr(g.get("dt_bias")), _ptr(g.get("S0")),
          _ptr(ws), ws.numel())
    return g


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

def _gate_checks(x, z, weight):
    L, code, dev = _begin(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, H, T, D]")
    B, H, T, D = x.shape
    _check(x, "x", (B, H, T, D), x.dtype, dev)
    bs, ts = (0, 0) if z is None else _rows(z, "z", B, T, H * D, x.dtype, dev)
    per_head = isinstance(weight, torch.Tensor) and weight.dim() == 2
    _check(weight, "weight", (H, D) if per_head else (D,), torch.float32, dev)
    return L, code, dev, (B, H, T, D), (bs, ts), int(per_head)


def gated_norm_forward(x, z, weight, eps=1e-6, gate_first=False, out=None):
    """RMS norm of each head's row with a SiLU gate, from the heads x
    [B,H,T,D] to token rows: returns y [B,T,H*D].

    y = norm(x) * weight * silu(z), or norm(x * silu(z)) * weight with
    ``gate_first``. z: [B,T,H*D], contiguous along the channels (a slice of a
    wider projection is read in place; None: no gate); weight: [D] or [H,D]
    fp32. D in {32, 64, 128}."""
    L, code, dev, (B, H, T, D), (bs, ts), ph = _gate_checks(x, z, weight)
    y = (torch.empty((B, T, H * D), dtype=x.dtype, device=dev) if out is None
         else out)
    _check(y, "y", (B, T, H * D), x.dtype, dev)
    _call(L.gated_norm_forward, "gated_norm_forward", dev, B, H, T, D, code,
          _ptr(x), _ptr(z), bs, ts, _ptr(weight), ph, float(eps),
          int(gate_first), _ptr(y))
    return y


def gated_norm_backward_workspace_bytes(B, H, T, D):
    return int(load_library().gated_norm_backward_workspace_bytes(B, H, T, D))


def gated_norm_backward(x, z, weight, dy, eps=1e-6, gate_first=False, out=None,
                        workspace=None):
    """Backward of gated_norm_forward: dy [B,T,H*D] in the dtype of x. Returns
    a dict x [B,H,T,D], z [B,T,H*D] (None without a gate) in the dtype of x,
    and weight fp32; ``out`` may pass such a dict preallocated."""
    L, code, dev, (B, H, T, D), (bs, ts), ph = _gate_checks(x, z, weight)
    _check(dy, "dy", (B, T, H * D), x.dtype, dev)
    g = out if out is not None else dict(
        x=torch.empty_like(x),
        z=None if z is None else torch.empty((B, T, H * D), dtype=x.dtype,
                                             device=dev),
        weight=torch.empty_like(weight))
    _required(g, ("x", "weight") + (() if z is None else ("z",)))
    _check(g["x"], "out[x]", (B, H, T, D), x.dtype, dev)
    _check(g["z"] if z is not None else None, "out[z]", (B, T, H * D), x.dtype,
           dev)
    _check(g["weight"], "out[weight]", weight.shape, torch.float32, dev)
    ws = _workspace(workspace, L.gated_norm_backward_workspace_bytes(B, H, T, D),
                    dev)
    _call(L.gated_norm_backward, "gated_norm_backward", dev, B, H, T, D, code,
          _ptr(x), _ptr(z), bs, ts, _ptr(weight), ph, float(eps),
          int(gate_first), _ptr(dy), _ptr(g["x"]),
          _ptr(None if z is None else g["z"]), _ptr(g["weight"]), _ptr(ws),
          ws.numel())
    return g


def residual_norm_forward(x, weight, residual=None, scale=1.0, eps=1e-6,
                          out=None):
    """Residual add and RMS norm: h = residual + scale * x, y = norm(h) *
    weight; returns (y in the dtype of x, h in the dtype of the residual).

    x: [..., C]; residual: the same shape in the dtype of x or fp32 (None:
    h = scale * x, in the dtype of x); weight: [C] fp32. y is formed from the
    32-bit sum. ``out`` may pass preallocated (y, h); h may be None to skip it,
    or the residual itself."""
    L, code, dev = _begin(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have a channel dimension")
    C, f32 = x.shape[-1], torch.float32
    R = x.numel() // C if C else 0
    _check(x, "x", x.shape, x.dtype, dev)
    rt = x.dtype if residual is None else residual.dtype
    if rt not in (x.dtype, f32):
        raise ValueError("residual must have the dtype of x or float32")
    _check(residual, "residual", x.shape, rt, dev)
    _check(weight, "weight", (C,), f32, dev)
    if out is None:
        y, h = torch.empty_like(x), torch.empty(x.shape, dtype=rt, device=dev)
    else:
        y, h = out
    _check(y, "y", x.shape, x.dtype, dev)
    _check(h, "h", x.shape, rt, dev)
    _call(L.residual_norm_forward, "residual_norm_forward", dev, R, C, code,
          _DTYPE_CODE[rt], _ptr(x), _ptr(residual), float(scale), _ptr(weight),
          float(eps), _ptr(y), _ptr(h))
    return y, h


def residual_norm_backward_workspace_bytes(R, C):
    return int(load_library().residual_norm_backward_workspace_bytes(R, C))


def residual_norm_backward(dy, h, weight, dh=None, scale=1.0, eps=1e-6, out=None,
                           workspace=None):
    """Backward of residual_norm_forward from its h: dy [..., C] is the
    adjoint of y, dh (dtype of h; None: zero) the adjoint that reaches h from
    the blocks behind. Returns a dict residual (dtype of h: the whole gradient
    of h), x (dtype of dy: scale times it) and weight [C] fp32; ``out`` may
    pass such a dict preallocated (residual may be None to skip it)."""
    L, code, dev = _begin(dy, "dy")
    if dy.dim() < 1:
        raise ValueError("dy must have a channel dimension")
    C, f32 = dy.shape[-1], torch.float32
    R = dy.numel() // C if C else 0
    _check(dy, "dy", dy.shape, dy.dtype, dev)
    if h.dtype not in (dy.dtype, f32):
        raise ValueError("h must have the dtype of dy or float32")
    _check(h, "h", dy.shape, h.dtype, dev)
    _check(dh, "dh", dy.shape, h.dtype, dev)
    _check(weight, "weight", (C,), f32, dev)
    g = out if out is not None else dict(x=torch.empty_like(dy),
                                         residual=torch.empty_like(h),
                                         weight=torch.empty_like(weight))
    _required(g, ("x", "weight"))
    _check(g["x"], "out[x]", dy.shape, dy.dtype, dev)
    _check(g.get("residual"), "out[residual]", dy.shape, h.dtype, dev)
    _check(g["weight"], "out[weight]", (C,), f32, dev)
    ws = _workspace(workspace, L.residual_norm_backward_workspace_bytes(R, C),
                    dev)
    _call(L.residual_norm_backward, "residual_norm_backward", dev, R, C, code,
          _DTYPE_CODE[h.dtype], _ptr(dy), _ptr(h), _ptr(dh), float(scale),
          _ptr(weight), float(eps), _ptr(g["x"]), _ptr(g.get("residual")),
          _ptr(g["weight"]), _ptr(ws), ws.numel())
    return g
