"""The sum of the parameters' gradients over workgroups is rounded once: with
integer terms whose partial sums fit fp32's 24 bits, the gradient is the exact sum
rounded to fp32, though the running sum passes 2^24."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32


def whole(shape, most, g):
    """Odd whole numbers up to `most`, mostly of one sign so that sums grow."""
    v = torch.randint(0, most // 2, shape, generator=g) * 2 + 1
    return torch.where(torch.rand(shape, generator=g) < 0.8, v, -v)


@pytest.mark.parametrize("R,C", [(4096, 40), (4000, 129), (2048, 1544)])
def test_residual_norm(R, C):
    """Rows of +-1 have a norm of one (eps 0): dweight = sum dy h."""
    g = torch.Generator().manual_seed(R)
    h = torch.randint(0, 2, (R, C), generator=g) * 2 - 1
    dy = whole((R, C), 1 << 20, g)
    got = osdn.residual_norm_backward(dy.to(F32).to(DEV), h.to(F32).to(DEV),
                                      torch.ones(C, device=DEV), eps=0.0)
    want = (dy.double() * h.double()).sum(0)
    assert want.abs().max() > 1 << 24
    assert torch.equal(got["weight"].cpu(), want.to(F32))


def test_convolution():
    """No activation and no norm: dweight_k = sum dy_t x_{t-W+1+k}, dbias = sum dy."""
    B, T, C, W = 4, 4096, 64, 3
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, 2, (B, T, C), generator=g) * 2 - 1
    dy = whole((B, 1, T, C), 1 << 15, g)
    got = osdn.short_conv_backward(x.to(F32).to(DEV), torch.ones(C, W, device=DEV),
                                   dy.to(F32).to(DEV), activation=False)
    full = torch.cat([torch.zeros(B, W - 1, C), x.double()], 1)
    d = dy.double()[:, 0]
    want = torch.stack([(d * full[:, k:k + T]).sum((0, 1)) for k in range(W)], 1)
    assert d.sum((0, 1)).max() > 1 << 24
    assert torch.equal(got["weight"].cpu(), want.to(F32))
    assert torch.equal(got["bias"].cpu(), d.sum((0, 1)).to(F32))
