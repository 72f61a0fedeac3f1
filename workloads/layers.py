"""Seeded synthetic inputs of one state space layer's operators: residual norm,
short convolutions over the channel slices of a projection, selective scan and
gated norm. Draws and the rounding to the storage dtype only, as in the
package's other generators.

Workloads (dims B, H, G, T, P, N; convolution of W taps; C model channels):

1. a prompt at the 1.3B-layer shape: 4, 16, 2, 4096, 128, 128, W=4, C=2048;
   bf16, the residual stream in fp32.
2. single tokens with a serving batch: 128, 16, 2, 1, 128, 128; bf16; drawn
   states.

The projection's rows hold x (H P channels), B and C (G N each) and the gate z
(H P). Decays A = -U(1, 16) and steps softplus(dt + dt_bias) with dt ~ N(0, 1)
and dt_bias the inverse softplus of log-uniform steps in (0.001, 0.1). Workload
i draws from torch generator seed 100 + i - 1.
"""

from dataclasses import dataclass, replace

import torch

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


@dataclass(frozen=True)
class Layer:
    name: str
    B: int
    H: int
    G: int
    T: int
    P: int
    N: int
    taps: int
    channels: int        # of the residual stream
    dtype: str           # "f32" or "bf16"
    seed: int
    decode: bool = False  # single tokens on drawn states

    def scaled(self, **kw):
        """Same recipe at other sizes."""
        return replace(self, **kw)

    @property
    def splits(self):
        """Channels of x, B, C and z in the projection's rows."""
        return (self.H * self.P, self.G * self.N, self.G * self.N,
                self.H * self.P)


LAYERS = [
    Layer("ssm-layer", 4, 16, 2, 4096, 128, 128, 4, 2048, "bf16", 100),
    Layer("ssm-layer-decode", 128, 16, 2, 1, 128, 128, 4, 2048, "bf16", 101,
          decode=True),
]

BY_NAME = {w.name: w for w in LAYERS}


def make_layer(w, device="cpu"):
    """dict of one layer's tensors: the residual stream `residual` (fp32) and
    the last block's output `block` [B,T,C]; `norm` [C]; the projection `proj`
    [B,T,sum(splits)]; `conv` (weight, bias) of the x, B and C channels; dt
    [B,H,T]; A, D, dt_bias [H]; `gate_norm` [H,P]; for decode workloads the
    convolutions' states `conv_state` and `S`; and the adjoints dy [B,T,H P],
    dnorm [B,T,C]."""
    g = torch.Generator().manual_seed(w.seed)
    t = _DTYPE[w.dtype]

    def draw(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)
    B, T, C, cx, cb = w.B, w.T, w.channels, w.splits[0], w.splits[1]
    a = dict(residual=draw(B, T, C), block=draw(B, T, C, dtype=t),
             norm=1 + draw(C, scale=0.1),
             proj=draw(B, T, sum(w.splits), dtype=t),
             conv_w=[draw(c, w.taps, scale=w.taps ** -0.5) for c in (cx, cb, cb)],
             conv_b=[draw(c, scale=0.1) for c in (cx, cb, cb)],
             dt=draw(B, w.H, T))
    a["A"] = -(1 + 15 * torch.rand(w.H, generator=g)).to(device)
    step = torch.exp(torch.rand(w.H, generator=g) * 4.6 - 6.9)
    a["dt_bias"] = torch.log(torch.expm1(step)).to(device)
    a["D"] = 1 + draw(w.H, scale=0.1)
    a["gate_norm"] = 1 + draw(w.H, w.P, scale=0.1)
    if w.decode:
        a["conv_state"] = [draw(B, w.taps - 1, c, dtype=t) for c in (cx, cb, cb)]
        a["S"] = draw(B, w.H, w.P, w.N, scale=w.N ** -0.5)
    else:
        a["dy"] = draw(B, T, cx, dtype=t)
        a["dnorm"] = draw(B, T, C, dtype=t)
    return a
