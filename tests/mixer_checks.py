"""Error bounds shared by the tests of the operators around the recurrences
(not a test module).

Every output is held, element by element, to
    |got - ref| <= u_out |ref| + u_op mag + k 2^-24 mag
where mag is the sum of the absolute values of the terms that make the element
(the oracle run on absolute inputs, or written out), u_out = half a step of the
output's type (bf16 2^-8, fp32 2^-24), u_op the rounding of operands that the
kernel documents (bf16 matrix operands: 2^-8 once, or 2^-16 in two parts; none
elsewhere), and k the number of fp32 roundings on the path: one for every term
added and some for the functions (exp2, reciprocal and rsqrt are off by one to
two units).
"""
import numpy as np
import torch

DEV = "cuda:0"
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-30


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def held(got, ref, mag, k, u_op=0.0, what=""):
    """The bound above for a GPU tensor against fp64 arrays."""
    assert tuple(got.shape) == tuple(np.shape(ref)), what
    g = f64(got)
    assert np.all(np.isfinite(g)), "%s: not finite" % what
    bound = U[got.dtype] * np.abs(ref) + (u_op + k * 2.0 ** -24) * np.abs(mag) + TINY
    if g.size == 0:
        return
    worst = float(np.max(np.abs(g - ref) / bound))
    print("%s: worst error %.3f of its bound" % (what, worst), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def rows(shape, dtype, gen, extra=0, scale=1.0):
    """A [B,T,C] tensor that is a channel slice of a wider one when extra > 0."""
    B, T, C = shape
    t = (torch.randn((B, T, C + extra), generator=gen) * scale).to(dtype).to(DEV)
    return t[:, :, :C]
