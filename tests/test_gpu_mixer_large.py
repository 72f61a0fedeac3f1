"""Tensors past 2^31 elements and 2^32 bytes: the operators on the whole against
the same calls on its last rows, heads or batch entries, whose addresses lie
past the border. Row-wise operators give the same bits; the scan cuts sequences
by the number of heads, so there two correct results are compared (each within
three roundings of bf16, half a step each, of the exact one)."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from test_gpu_guard import _bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TOL = 6 * 2.0 ** -8


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def filled(*shape, dtype=BF, seed=0):
    """Values that repeat every 1e6 + 3 elements (drawing 2^31 takes long)."""
    g = torch.Generator().manual_seed(seed)
    tile = torch.randn(1000003, generator=g).to(dtype).to(DEV)
    n = 1
    for s in shape:
        n *= s
    t = torch.empty(n, dtype=dtype, device=DEV)
    whole = n // tile.numel() * tile.numel()
    t[:whole].view(-1, tile.numel()).copy_(tile.expand(whole // tile.numel(), -1))
    t[whole:] = tile[:n - whole]
    return t.view(*shape)


def near(a, b, what):
    a, b = a.double(), b.double()
    e = float((a - b).norm() / b.norm())
    print("%s: %.2e" % (what, e), flush=True)
    assert e <= TOL, what


def test_residual_norm():
    R, C = (1 << 20) + 5, 2048 + 24
    x, w = filled(R, C), filled(C, dtype=F32, seed=1)
    y, h = osdn.residual_norm_forward(x, w, scale=0.5)
    y2, h2 = osdn.residual_norm_forward(x[-9:].clone(), w, scale=0.5)
    assert torch.equal(_bits(y[-9:]), _bits(y2)) and torch.equal(_bits(h[-9:]), _bits(h2))
    g = osdn.residual_norm_backward(x, h, w, scale=0.5)
    g2 = osdn.residual_norm_backward(x[-9:].clone(), h2, w, scale=0.5)
    assert torch.equal(_bits(g["x"][-9:]), _bits(g2["x"]))


def test_convolution_and_gated_norm():
    B, T, H, D = 2, (1 << 17) + 3, 64, 128
    C = H * D
    x, w, b = filled(B, T, C), filled(C, 4, dtype=F32, seed=1), filled(C, dtype=F32, seed=2)
    y, tail = osdn.short_conv_forward(x, w, b, head_dim=D, l2norm=True)
    y2, tail2 = osdn.short_conv_forward(x[1:, -70:].clone(), w, b, x[1:, -73:-70].clone(),
                                        head_dim=D, l2norm=True)
    assert torch.equal(_bits(y[1, :, -70:]), _bits(y2[0]))
    assert torch.equal(_bits(tail[1]), _bits(tail2[0]))
    g = osdn.short_conv_backward(x, w, y, b, head_dim=D)
    g2 = osdn.short_conv_backward(x[1:, -70:].clone(), w, y[1:, :, -70:].contiguous(), b,
                                  x[1:, -73:-70].clone(), head_dim=D)
    assert torch.equal(_bits(g["x"][1, -70:]), _bits(g2["x"][0]))
    del g, g2
    o = osdn.gated_norm_forward(y, x, w[:D, 0].contiguous())
    o2 = osdn.gated_norm_forward(y[1:, :, -70:].contiguous(), x[1:, -70:].clone(),
                                 w[:D, 0].contiguous())
    assert torch.equal(_bits(o[1, -70:]), _bits(o2[0]))


def test_scan_and_its_backward():
    H, T, P, N = 32, (1 << 19) + 37, 128, 64
    x, dy = filled(1, H, T, P), filled(1, H, T, P, seed=1)
    B, C = filled(1, 1, T, N, seed=2), filled(1, 1, T, N, seed=3)
    dt = filled(1, H, T, dtype=F32, seed=4)
    A = -torch.linspace(1, 4, H, device=DEV)
    y, S = osdn.ssm_forward(x, dt, A, B, C)
    last = lambda t: t[:, -1:].clone()
    y2, S2 = osdn.ssm_forward(last(x), last(dt), A[-1:].clone(), B, C)
    near(y[:, -1:], y2, "y")
    near(S[:, -1:], S2, "S_T")
    g = osdn.ssm_backward(x, dt, A, B, C, dy)
    g2 = osdn.ssm_backward(last(x), last(dt), A[-1:].clone(), B, C, last(dy))
    near(g["x"][:, -1:], g2["x"], "dx")
    near(g["dt"][:, -1:], g2["dt"], "ddt")
    near(g["A"][-1:], g2["A"], "dA")


def test_single_tokens():
    B, H, P, N = 2100, 64, 128, 128
    S = filled(B, H, P, N, dtype=F32)
    x, dt = filled(B, H, 1, P, seed=1), filled(B, H, 1, dtype=F32, seed=2)
    Bm, Cm = filled(B, 2, 1, N, seed=3), filled(B, 2, 1, N, seed=4)
    A = -torch.linspace(1, 4, H, device=DEV)
    S2 = S[-2:].clone()
    y = osdn.ssm_decode(x, dt, A, Bm, Cm, S)
    y2 = osdn.ssm_decode(x[-2:].clone(), dt[-2:].clone(), A, Bm[-2:].clone(),
                         Cm[-2:].clone(), S2)
    assert torch.equal(_bits(y[-2:]), _bits(y2)) and torch.equal(S[-2:], S2)
