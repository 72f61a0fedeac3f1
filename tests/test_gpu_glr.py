"""Gated linear recurrence (forward, single tokens, backward) against the fp64
oracle, element by element: lengths from nothing to several tiles, odd widths,
channel ranges of wider rows, padded batches whose padding is NaN, decays from none
to total, segments, carried states, values at the ends of their ranges."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, UNIT, f64, held, spoil, split_rows
from oracle import layer as Y

pytestmark = pytest.mark.gpu


def inputs(B, T, C, dt, gate=True, lens=None, state=True, extra=0, seed=0, slow=False):
    g = torch.Generator().manual_seed(seed + 7 * T + C)
    x, r, i = split_rows(B, T, (C, C, C), dt, g, extra)
    low, high = (-9.0, -5.0) if slow else (-7.0, 1.0)
    A = -torch.exp(torch.rand(C, generator=g) * (high - low) + low).to(DEV)
    k = dict(i=i if gate else None,
             h0=torch.randn((B, C), generator=g).to(DEV) if state else None,
             lengths=None if lens is None else torch.tensor(lens, dtype=torch.int32,
                                                            device=DEV))
    for t in (x, r, i):
        spoil(t, k["lengths"])
    dy = torch.randn((B, T, C), generator=g).to(dt).to(DEV)
    spoil(dy, k["lengths"])
    dh = torch.randn((B, C), generator=g).to(DEV) if state else None
    return (x, r, A), k, dy, dh


def ref_kw(k):
    return {n: f64(t) if t is not None and t.is_floating_point() else
            (None if t is None else t.tolist()) for n, t in k.items()}


def check(B, T, C, dt, normalize=True, **kw):
    a, k, dy, dh = inputs(B, T, C, dt, **kw)
    print("case", B, T, C, dt, normalize, kw, flush=True)
    y, h_T, states = osdn.glr_forward(*a, normalize=normalize, save=True, **k)
    one = osdn.glr_backward(*a, dy, dh_T=dh, normalize=normalize, states=states, **k)
    two = osdn.glr_backward(*a, dy, dh_T=dh, normalize=normalize, **k)
    torch.cuda.synchronize()
    for n in one:        # the states formed there are the forward's
        assert (one[n] is None and two[n] is None) or torch.equal(one[n], two[n]), n
    ra, rk = [f64(t) for t in a], ref_kw(k)
    ry, rh, rb = Y.glr_ref(*ra, normalize=normalize, **rk)
    absk = dict(rk, h0=None if rk["h0"] is None else np.abs(rk["h0"]))
    my, mh, mb = Y.glr_ref(np.abs(ra[0]), ra[1], ra[2], normalize=normalize, **absk)
    u = 48 + T / 16
    held(y, ry, (u, my), what="y")
    held(h_T, rh, (u, mh), what="h_T")
    held(states, rb[:, ::16], (u, mb[:, ::16]), what="states")
    g, mag = Y.glr_backward_ref(*ra, f64(dy), dh_T=f64(dh), normalize=normalize, **rk)
    u = 112 + T / 8
    for n in g:
        # a gradient of A adds its terms in 32 bits over 8 tokens, then in 64
        held(one[n], g[n], (u, mag[n]), what="d" + n)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 15, 16, 17, 127, 128, 129, 300])
def test_lengths(T, dt):
    check(2, T, 70, dt, seed=1)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 3, 63, 64, 65, 130, 257])
def test_widths(C, dt):
    check(2, 37, C, dt, seed=2)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
def test_forms(normalize, gate, dt):
    check(2, 150, 66, dt, normalize=normalize, gate=gate, seed=3)
    check(2, 33, 65, dt, normalize=normalize, gate=gate, state=False, extra=3, seed=4)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("extra", [0, 1, 2, 5, 64])
def test_strides(extra, dt):
    check(3, 40, 64, dt, extra=extra, seed=5)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(200, [200, 0, 131, 1]), (130, [129, 128, 127, 5]),
                                    (16, [16, 15, 0, 20]), (700, [700, 260, 513, 0])])
def test_padded(T, lens, dt):
    check(4, T, 67, dt, lens=lens, seed=6)


def test_lengths_outside_are_clamped():
    a, k, dy, dh = inputs(3, 20, 10, F32)
    lens = torch.tensor([-5, 25, 20], dtype=torch.int32, device=DEV)
    y, h_T, _ = osdn.glr_forward(*a, **dict(k, lengths=lens))
    want, wh, _ = osdn.glr_forward(*a, **dict(k, lengths=lens.clamp(0, 20)))
    assert torch.equal(y, want) and torch.equal(h_T, wh)
    assert not y[0].any() and torch.equal(h_T[0], k["h0"][0])


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(1024, None), (1500, [1500, 1023]), (2100, [40, 2100])])
def test_segments(T, lens, dt):
    """Long sequences of few channels, cut into segments: some of them empty."""
    assert osdn.glr_forward_workspace_bytes(2, T, 64) > 0
    check(2, T, 64, dt, lens=lens, seed=7)


def test_long_memory():
    """Decays within 1e-4 of one over thousands of tokens."""
    check(1, 6000, 32, F32, slow=True, seed=8)


def test_many_workgroups_walk_whole_sequences():
    B, T, C = 3, 260, 64 * 66
    assert osdn.glr_forward_workspace_bytes(B, T, C) == 0
    check(B, T, C, BF, seed=9)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (5, 1, 130), (3, 4, 67), (2, 1, 4096)])
@pytest.mark.parametrize("gate", [True, False])
def test_decode(B, T, C, gate, dt):
    a, k, _, _ = inputs(B, T, C, dt, gate=gate, seed=10)
    h = k["h0"].clone()
    out = torch.empty_like(h)
    y2 = osdn.glr_decode(*a, h, i=k["i"], h_out=out)
    assert torch.equal(h, k["h0"])
    y = osdn.glr_decode(*a, h, i=k["i"])
    assert torch.equal(h, out) and torch.equal(y, y2)
    ra, rk = [f64(t) for t in a], ref_kw(k)
    ry, rh, _ = Y.glr_ref(*ra, **rk)
    my, mh, _ = Y.glr_ref(np.abs(ra[0]), ra[1], ra[2], **dict(rk, h0=np.abs(rk["h0"])))
    held(y, ry, (48, my), what="y")
    held(h, rh, (48, mh), what="h")


def test_prompt_then_tokens_is_the_whole():
    """A prompt, then single tokens from its state, against one call over all."""
    a, k, _, _ = inputs(2, 150, 96, F32, seed=11)
    y, h_T, _ = osdn.glr_forward(*a, **k)
    cut = lambda t, s: None if t is None else t[:, s]
    p = slice(0, 140)
    y0, h, _ = osdn.glr_forward(cut(a[0], p), cut(a[1], p), a[2],
                                **dict(k, i=cut(k["i"], p)))
    parts = [y0]
    for t in range(140, 150):
        s = slice(t, t + 1)
        parts.append(osdn.glr_decode(cut(a[0], s), cut(a[1], s), a[2], h,
                                     i=cut(k["i"], s)))
    got = torch.cat(parts, 1)
    big = Y.glr_ref(np.abs(f64(a[0])), f64(a[1]), f64(a[2]),
                    **dict(ref_kw(k), h0=np.abs(f64(k["h0"]))))
    held(got, f64(y), (2 * (48 + 150 / 16), big[0]), what="y")
    held(h, f64(h_T), (2 * (48 + 150 / 16), big[1]), what="h_T")


@pytest.mark.parametrize("normalize", [True, False])
def test_ends_of_the_gates(normalize):
    """Closed and open gates: a of exactly one keeps the state bit for bit and lets
    nothing in (normalize); a of zero forgets it. Gradients stay finite."""
    B, T, C = 1, 40, 64
    g = torch.Generator().manual_seed(12)
    x = torch.randn((B, T, C), generator=g).to(DEV)
    h0 = torch.randn((B, C), generator=g).to(DEV)
    A = torch.full((C,), -1.0, device=DEV)
    shut = torch.full_like(x, -200.0)
    y, h_T, st = osdn.glr_forward(x, shut, A, h0=h0, normalize=normalize, save=True)
    if normalize:
        assert torch.equal(y, h0[:, None].expand_as(y).contiguous())
        assert torch.equal(h_T, h0)
    big = torch.full((C,), -1e30, device=DEV)
    wide = torch.full_like(x, 30.0)
    y, _, _ = osdn.glr_forward(x, wide, big, h0=h0, normalize=normalize)
    assert torch.equal(y, x)        # m = 1, the decay is zero
    for r, a in ((shut, A), (wide, big), (shut, torch.zeros_like(A)), (wide, A)):
        d = osdn.glr_backward(x, r, a, x, h0=h0, dh_T=h0, normalize=normalize)
        for n in ("x", "r", "A", "h0"):
            assert torch.isfinite(d[n]).all(), n


def test_an_inf_or_nan_stays_in_its_channel_and_behind_its_token():
    a, k, dy, _ = inputs(2, 200, 66, F32, seed=13)
    y0, _, _ = osdn.glr_forward(*a, **k)
    for bad in (float("nan"), float("inf")):
        x = a[0].clone()
        x[1, 77, 5] = bad
        y, h_T, _ = osdn.glr_forward(x, a[1], a[2], **k)
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[1, 77:, 5] = False
        assert torch.equal(y[keep], y0[keep])
        assert not torch.isfinite(y[1, 77:, 5]).any()


def test_empty():
    for B, T, C in ((0, 5, 4), (2, 0, 4), (2, 5, 0)):
        a, k, dy, dh = inputs(B, T, C, F32)
        y, h_T, st = osdn.glr_forward(*a, save=True, **k)
        assert torch.equal(h_T, k["h0"]) and y.numel() == 0
        d = osdn.glr_backward(*a, dy, dh_T=dh, **k)
        torch.cuda.synchronize()
        assert not d["A"].any() and torch.equal(d["h0"], dh)
        osdn.glr_decode(*a, k["h0"], i=k["i"])
    a, k, dy, dh = inputs(2, 0, 4, F32)
    out = torch.full((2, 4), 9.0, device=DEV)
    osdn.glr_decode(*a, k["h0"], h_out=out)
    assert torch.equal(out, k["h0"])


def test_the_same_bits_again():
    a, k, dy, dh = inputs(2, 1500, 128, BF, seed=14)
    one = osdn.glr_backward(*a, dy, dh_T=dh, **k)
    for _ in range(3):
        two = osdn.glr_backward(*a, dy, dh_T=dh, **k)
        assert all(torch.equal(one[n], two[n]) for n in one)


def test_gradient_against_differences():
    """Differences of the fp32 forward along a direction."""
    a, k, dy, dh = inputs(1, 100, 64, F32, seed=15)
    d = osdn.glr_backward(*a, dy, dh_T=dh, **k)
    g = torch.Generator().manual_seed(16)
    for n, t in dict(x=a[0], r=a[1], i=k["i"], A=a[2], h0=k["h0"]).items():
        v = torch.randn(t.shape, generator=g).to(DEV)
        v = v * t.abs() if n == "A" else v
        e = 2e-3

        def loss(s):
            moved = dict(x=a[0], r=a[1], A=a[2], i=k["i"], h0=k["h0"])
            moved[n] = (t + s * v).contiguous()
            y, h, _ = osdn.glr_forward(**moved)
            return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())
        num = (loss(e) - loss(-e)) / (2 * e)
        want = float((d[n].double() * v.double()).sum())
        # the difference's own error: e^2 of the third derivative, and the outputs'
        # rounding (64 units of each of 6464 terms, at random) over 2 e
        scale = float((d[n].double() * v.double()).norm()) + 64 * UNIT * 100 / e
        print(n, num, want, scale, flush=True)
        assert abs(num - want) <= 2e-2 * scale


def test_wrong_tensors_are_refused():
    """What is missing, of another shape or type, or strided along its channels names
    itself in a ValueError or TypeError before the library is called."""
    x, A = torch.zeros(2, 3, 8, device=DEV), torch.zeros(8, device=DEV)
    h = torch.zeros(2, 8, device=DEV)
    for bad in (None, x[:1], x.double(), x.cpu(), x.transpose(0, 2).contiguous().transpose(0, 2),
                1.0):
        for call in (lambda: osdn.glr_forward(x, bad, A),
                     lambda: osdn.glr_backward(x, bad, A, x),
                     lambda: osdn.glr_decode(x, bad, A, h)):
            with pytest.raises((ValueError, TypeError)):
                call()
    for bad in (None, A[:7], A.double(), torch.zeros(16, device=DEV)[::2]):
        with pytest.raises((ValueError, TypeError)):
            osdn.glr_forward(x, x, bad)
    with pytest.raises(ValueError):
        osdn.glr_forward(x[0], x[0], A)
    for bad in (None, h[:1], h.double(), h.t().contiguous().t()):
        with pytest.raises((ValueError, TypeError)):
            osdn.glr_decode(x, x, A, bad)
