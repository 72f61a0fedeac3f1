"""Norm and rotation of queries and keys (forward and backward) against the fp64
oracle, element by element."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, f64, held, spoil, split_rows
from oracle import layer as Y

pytestmark = pytest.mark.gpu


def freqs(rot):
    return (None if rot == 0 else
            (10000.0 ** -(torch.arange(rot // 2) / (rot // 2))).float().to(DEV))


def inputs(B, T, Hq, Hk, D, dt, rot, weight=True, lens=None, pos=None, extra=0, seed=0,
           yt=None):
    g = torch.Generator().manual_seed(seed + T + D)
    q, k = split_rows(B, T, (Hq * D, Hk * D), dt, g, extra)
    w = lambda: (1 + 0.2 * torch.randn(D, generator=g)).to(DEV) if weight else None
    kw = dict(inv_freq=freqs(rot), q_weight=w(), k_weight=w(), positions=pos,
              lengths=None if lens is None else torch.tensor(lens, dtype=torch.int32,
                                                             device=DEV))
    n = lambda H: torch.randn((B, H, T, D), generator=g).to(yt or dt).to(DEV)
    dq, dk = n(Hq), n(Hk)
    for t in (q, k):
        spoil(t, kw["lengths"])
    for t in (dq, dk):
        spoil(t.transpose(1, 2), kw["lengths"])
    return q, k, dq, dk, kw


def check(B, T, Hq, Hk, D, dt, rot, norm="rms", interleaved=False, eps=1e-6, **make):
    print("case", B, T, Hq, Hk, D, dt, rot, norm, interleaved, make, flush=True)
    q, k, dq, dk, kw = inputs(B, T, Hq, Hk, D, dt, rot, **make)
    form = dict(norm=norm, interleaved=interleaved, eps=eps)
    yq, yk = osdn.qk_rotary_forward(q, k, D, **kw, **form)
    d = osdn.qk_rotary_backward(q, k, dq, dk, D, **kw, **form)
    torch.cuda.synchronize()
    rk = dict(inv_freq=f64(kw["inv_freq"]), positions=f64(kw["positions"]),
              lengths=None if kw["lengths"] is None else kw["lengths"].tolist(), **form)
    for x, dy, y, w, n in ((q, dq, yq, kw["q_weight"], "q"), (k, dk, yk, kw["k_weight"], "k")):
        ref, mag = Y.qk_rotary_ref(f64(x), D, weight=f64(w), **rk)
        held(y, ref, (40, mag), what=n)
        g, m = Y.qk_rotary_backward_ref(f64(x), f64(dy), D, weight=f64(w), **rk)
        held(d[n], g["x"], (64, m["x"]), what="d" + n)
        if w is None:
            assert d[n + "_weight"] is None
        else:
            rows = min(B * T * y.shape[1], 8 * y.shape[1] * (1 + B * T // 1024))
            held(d[n + "_weight"], g["weight"], (64 + rows, m["weight"]), what="dw" + n)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations(D, interleaved, dt):
    for rot in (0, 16, D // 2, D - 16, D):
        check(2, 9, 3, 2, D, dt, rot, interleaved=interleaved)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("weight", [True, False])
def test_norms(norm, weight, dt):
    check(2, 11, 4, 1, 64, dt, 64, norm=norm, weight=weight, seed=1)
    check(1, 5, 1, 3, 128, dt, 32, norm=norm, weight=weight, eps=0.5, seed=2)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (5, 1, 16, 2), (1, 2049, 2, 1),
                                       (3, 700, 5, 3), (2, 4100, 1, 1), (1, 17, 33, 7)])
def test_sizes(B, T, Hq, Hk, dt):
    check(B, T, Hq, Hk, 32, dt, 32, seed=3)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("extra", [1, 4, 8])
def test_strides(extra, dt):
    check(2, 13, 2, 2, 64, dt, 32, extra=extra, seed=4)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_padded(dt):
    check(4, 30, 3, 2, 64, dt, 64, lens=[30, 0, 11, 40], seed=5)


def test_adjoints_in_fp32():
    check(2, 19, 3, 1, 128, BF, 64, yt=F32, seed=6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles keep their digits at the largest positions, negative ones too."""
    top = 2 ** 31 - 1
    pos = torch.tensor([[0, 1, top, -top, 1 << 24], [12345678, 999999937, 5, -1, 7]],
                       dtype=torch.int32, device=DEV)
    check(2, 5, 2, 1, 64, F32, 64, pos=pos, interleaved=interleaved, norm="none",
          weight=False)


def test_one_input_alone():
    q, k, dq, dk, kw = inputs(2, 9, 3, 2, 64, BF, 64)
    both = osdn.qk_rotary_forward(q, k, 64, **kw)
    d = osdn.qk_rotary_backward(q, k, dq, dk, 64, **kw)
    one, none = osdn.qk_rotary_forward(q, None, 64, **kw)
    assert none is None and torch.equal(one, both[0])
    none, one = osdn.qk_rotary_forward(None, k, 64, **kw)
    assert none is None and torch.equal(one, both[1])
    a = osdn.qk_rotary_backward(q, None, dq, None, 64, **dict(kw, k_weight=None))
    b = osdn.qk_rotary_backward(None, k, None, dk, 64, **dict(kw, q_weight=None))
    assert torch.equal(a["q"], d["q"]) and torch.equal(a["q_weight"], d["q_weight"])
    assert torch.equal(b["k"], d["k"]) and torch.equal(b["k_weight"], d["k_weight"])
    assert a["k"] is None and b["q"] is None


def test_zero_rows():
    """A row of zeros stays one; its gradient is the weight over sqrt(eps)."""
    q, k, dq, dk, kw = inputs(1, 4, 2, 1, 32, F32, 0)
    q = torch.zeros_like(q)
    y, _ = osdn.qk_rotary_forward(q, k, 32, **kw)
    assert not y.any()
    d = osdn.qk_rotary_backward(q, k, dq, dk, 32, **kw)
    want = dq.transpose(1, 2).reshape(1, 4, -1) * kw["q_weight"].repeat(2) * 1e3
    assert torch.allclose(d["q"], want, rtol=1e-5)
    assert not d["q_weight"].any()


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_no_eps(dt, norm):
    """eps = 0: rows behind a sequence and rows of zeros give zeros, no NaN."""
    check(3, 9, 2, 1, 64, dt, 32, norm=norm, eps=0.0, lens=[9, 0, 4], seed=7)
    q, k, dq, dk, kw = inputs(1, 4, 2, 1, 64, dt, 32, seed=8)
    q = torch.zeros_like(q)
    y, _ = osdn.qk_rotary_forward(q, k, 64, norm=norm, eps=0.0, **kw)
    d = osdn.qk_rotary_backward(q, k, dq, dk, 64, norm=norm, eps=0.0, **kw)
    torch.cuda.synchronize()
    for t in (y, d["q"], d["q_weight"]):
        assert (t == 0).all()


def test_empty():
    for B, T in ((0, 4), (3, 0)):
        q, k, dq, dk, kw = inputs(B, T, 2, 1, 32, F32, 32)
        y, _ = osdn.qk_rotary_forward(q, k, 32, **kw)
        assert y.shape == (B, 2, T, 32)
        d = osdn.qk_rotary_backward(q, k, dq, dk, 32, **kw)
        torch.cuda.synchronize()
        assert not d["q_weight"].any() and not d["k_weight"].any()


def test_a_decode_step_is_the_prompts_row():
    """One token with its position gives the bits of the prompt's."""
    q, k, _, _, kw = inputs(3, 40, 4, 2, 64, BF, 32)
    yq, yk = osdn.qk_rotary_forward(q, k, 64, **kw)
    t = 37
    pos = torch.full((3, 1), t, dtype=torch.int32, device=DEV)
    oq, ok = osdn.qk_rotary_forward(q[:, t:t + 1], k[:, t:t + 1], 64,
                                    **dict(kw, positions=pos))
    assert torch.equal(oq[:, :, 0], yq[:, :, t]) and torch.equal(ok[:, :, 0], yk[:, :, t])
