"""The operators that complete a block on tensors whose offsets pass 32 bits: rows read
far apart give the bits of rows side by side, results far out those of a small call."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, dt=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dt)


def apart(t, row):
    """t [B,T,C] as rows `row` elements apart in a buffer of their own."""
    B, T, C = t.shape
    buf = torch.empty(B * T * row, dtype=t.dtype, device=DEV)
    far = buf.view(B, T, row)[:, :, :C]
    far.copy_(t)
    return far


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_rows_far_apart(dt):
    """Token strides at their limit of 2^22 elements, 5 GB (bf16) or 10 from end to end."""
    B, T, C = 2, 300, 64
    x, r, dy = (rand(B, T, C, seed=s, dt=dt) for s in range(3))
    A = -torch.rand(C, device=DEV)
    y, h_T, st = osdn.glr_forward(x, r, A, save=True)
    d = osdn.glr_backward(x, r, A, dy, states=st)
    fx = apart(x, 1 << 22)
    for a, b in zip(osdn.glr_forward(fx, r, A, save=True), (y, h_T, st)):
        assert torch.equal(a, b)
    e = osdn.glr_backward(fx, r, A, dy)
    assert all(torch.equal(e[n], d[n]) for n in d if d[n] is not None)
    h = torch.zeros(B, C, device=DEV)
    assert torch.equal(osdn.glr_decode(fx[:, -1:], r[:, -1:], A, h.clone())[0],
                       osdn.glr_decode(x[:, -1:], r[:, -1:], A, h)[0])

    q, f = rand(B, T, 64, seed=4, dt=dt), torch.rand(16, device=DEV)
    g = rand(B, 2, T, 32, seed=5, dt=dt)
    fq = fx
    fq.copy_(q)
    assert torch.equal(osdn.qk_rotary_forward(fq, None, 32, inv_freq=f)[0],
                       osdn.qk_rotary_forward(q, None, 32, inv_freq=f)[0])
    assert torch.equal(osdn.qk_rotary_backward(fq, None, g, None, 32, inv_freq=f)["q"],
                       osdn.qk_rotary_backward(q, None, g, None, 32, inv_freq=f)["q"])


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [64, 61])
def test_feed_forward_rows_far_apart(dt, C):
    """A row stride at its limit of 2^21 elements."""
    R, F = 1100, 72
    x, wg, wu, dh = (rand(*s, seed=k, dt=dt)
                     for k, s in enumerate(((R, C), (F, C), (F, C), (R, F))))
    fx = apart(x[None], 1 << 21)[0]
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    assert torch.equal(osdn.gated_ffn_forward(fx, wg, wu)[0], h)
    assert torch.equal(osdn.gated_ffn_forward(fx[-3:], wg, wu)[0],
                       osdn.gated_ffn_forward(x[-3:], wg, wu)[0])
    a, b = (osdn.gated_ffn_backward(t, wg, wu, g, u, dh) for t in (x, fx))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_results_past_32_bits():
    """More than 2^31 results of each operator: the last rows are those of a call of
    their own."""
    R, C, F = 140000, 64, 16384
    x, wg, wu = rand(R, C), rand(F, C, seed=1), rand(F, C, seed=2)
    h = osdn.gated_ffn_forward(x, wg, wu)[0]
    assert h.numel() > 1 << 31
    # (one tile of k: tiles of any shape form the same sums)
    at = R - 733
    assert torch.equal(h[at:], osdn.gated_ffn_forward(x[at:], wg, wu)[0])
    del h

    B, T, C = 3, 180000, 4096
    x = rand(1, T, C).expand(B, T, C)
    r, A = rand(1, T, C, seed=1).expand(B, T, C), -torch.rand(C, device=DEV)
    y, h_T, _ = osdn.glr_forward(x, r, A)
    assert y.numel() > 1 << 31
    assert torch.equal(y[2], y[0]) and torch.equal(h_T[2], h_T[0])
    tail = osdn.glr_forward(x[2:, -7:], r[2:, -7:], A, h0=y[2:, -8].float())[0]
    # half a step of the state that begins, under decays below one, and of both results
    first = float(y[2, -8].abs().max())
    assert torch.allclose(tail[0].float(), y[2, -7:].float(), rtol=2 ** -7,
                          atol=first * 2 ** -8)
    del y, tail

    f = 0.1 * torch.rand(64, device=DEV)
    yq = osdn.qk_rotary_forward(x, None, 128, inv_freq=f)[0]
    assert yq.numel() > 1 << 31
    pos = torch.arange(T - 5, T, dtype=torch.int32, device=DEV)[None]
    one = osdn.qk_rotary_forward(x[2:, -5:], None, 128, inv_freq=f, positions=pos)[0]
    assert torch.equal(yq[2, :, -5:], one[0]) and torch.equal(yq[2, 31], yq[0, 31])
