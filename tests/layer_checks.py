"""Inputs and error bounds shared by the tests of the operators that complete a
block (not a test module).

An element is held to |got - ref| <= U |ref| + sum of (units * magnitude), U half a
step of the output's type, magnitudes from the oracle (the sum of the absolute
values of the terms). Units of 2^-24 are counted along the path:

* recurrence: a decay exp2(A log2(e) sigmoid(r)) is off by 2 units for the exp2 and
  6 times its logarithm for the argument, |la| exp(-|la|) <= 1/e of a whole memory:
  under 3 together however long the memory is; each of the up to 16 tokens of a thread
  rounds once; every two threads (16 tokens or more) the carried state is rounded once
  more and its factor's distance from one is off by 4 units of itself (again under 2 over
  a memory). With the input factor (8), sigmoid(i) (4 and |i| <= 8 times its slope) and
  the products: 48 + T / 16. The gradients pass through two such chains and three
  more factors: 112 + T / 8.
* rotary: the sum of squares of a row is 8 additions a lane and 4 levels, its root 4
  units; cosine and sine are off by 6 units of one, the products 6: 40. Backward 64,
  and one unit for every term that a thread adds to a weight's gradient.
* feed-forward: one unit for each of the C (or 2 F, R) terms, and 24 for the
  activation, whose argument scales its error by 1 + |g|.
"""
import numpy as np
import torch

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = {F32: 2.0 ** -24, BF: 2.0 ** -8}
UNIT = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def held(got, ref, *terms, what=""):
    """terms: (units, magnitude), units as a multiple of 2^-24."""
    assert tuple(got.shape) == tuple(np.shape(ref)), what
    g = f64(got)
    assert np.all(np.isfinite(g)), "%s: not finite" % what
    bound = U[got.dtype] * np.abs(ref) + 1e-30
    for k, mag in terms:
        bound = bound + k * UNIT * np.abs(mag)
    if g.size == 0:
        return
    worst = float(np.max(np.abs(g - ref) / bound))
    print("%s: worst error %.3f of its bound" % (what, worst), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def split_rows(B, T, widths, dt, gen, extra=0):
    """[B,T,w] channel ranges of one wider tensor, as a projection's parts are."""
    t = torch.randn((B, T, sum(widths) + extra), generator=gen).to(dt).to(DEV)
    out, at = [], 0
    for w in widths:
        out.append(t[:, :, at:at + w])
        at += w
    return out


def spoil(t, lengths):
    """The rows behind each sequence's end made NaN, in place."""
    if lengths is not None and t is not None:
        for b, n in enumerate(lengths.tolist()):
            t[b, max(0, n):] = float("nan")
