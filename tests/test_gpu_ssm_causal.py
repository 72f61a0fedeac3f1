"""Selective scan: a token reaches itself and later tokens, also when it holds an
inf or a NaN. Against the same call on finite inputs, bit for bit: everything
before the token, the other channels of the state where only x is struck, and the
other heads; what the recurrence makes non-finite has to be non-finite."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from test_gpu_ssm import adjoints, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
# first and last of a block of 16, of a chunk of 32 and of 64, and the last token
AT = [0, 5, 15, 16, 40, 63, 64, 95, 149]


def same(a, b):
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("P,N", [(32, 32), (64, 128), (128, 64)])
def test_x(P, N, bad, dt):
    a, k = inputs(1, 2, 1, 150, P, N, dt, seed=1)
    y0, S0 = osdn.ssm_forward(**a, **k)
    for j in AT:
        p = 7 + 3 * j % (P - 8)
        keep = a["x"][0, 0, j, p].clone()
        a["x"][0, 0, j, p] = bad
        y, S = osdn.ssm_forward(**a, **k)
        a["x"][0, 0, j, p] = keep
        others = [c for c in range(P) if c != p]
        same(y[0, 1], y0[0, 1]), same(S[0, 1], S0[0, 1])
        same(y[0, 0, :j], y0[0, 0, :j])
        same(y[0, 0][:, others], y0[0, 0][:, others])
        same(S[0, 0, others], S0[0, 0, others])
        assert not torch.isfinite(y[0, 0, j:, p]).any()
        assert not torch.isfinite(S[0, 0, p]).any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_several_tokens_and_channels(bad, dt):
    """More than one struck token a chunk, in a sequence long enough for
    segments, and behind a length."""
    a, k = inputs(2, 2, 1, 900, 64, 64, dt, seed=2, lens=[900, 300])
    y0, S0 = osdn.ssm_forward(**a, **k)
    first = {}
    for b, h, j, p in ((0, 0, 130, 3), (0, 0, 135, 3), (0, 0, 133, 60), (0, 1, 640, 17),
                       (0, 1, 703, 18), (1, 0, 299, 5), (1, 1, 300, 6)):
        a["x"][b, h, j, p] = bad
        if j < (900, 300)[b]:
            first[b, h, p] = min(j, first.get((b, h, p), j))
    y, S = osdn.ssm_forward(**a, **k)
    for b in range(2):
        n = (900, 300)[b]
        for h in range(2):
            for p in range(64):
                j = first.get((b, h, p), n)
                same(y[b, h, :j, p], y0[b, h, :j, p])
                same(y[b, h, n:, p], y0[b, h, n:, p])
                assert not torch.isfinite(y[b, h, j:n, p]).any()
                if j == n:
                    same(S[b, h, p], S0[b, h, p])
                else:
                    assert not torch.isfinite(S[b, h, p]).any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_keys_and_queries(bad, dt):
    a, k = inputs(1, 4, 2, 150, 64, 32, dt, seed=3)
    y0, S0 = osdn.ssm_forward(**a, **k)
    for j in AT:
        for name in ("B", "C"):
            keep = a[name][0, 0, j, 9].clone()
            a[name][0, 0, j, 9] = bad
            y, S = osdn.ssm_forward(**a, **k)
            a[name][0, 0, j, 9] = keep
            same(y[0, 2:], y0[0, 2:]), same(S[0, 2:], S0[0, 2:])
            same(y[0, :2, :j], y0[0, :2, :j])
            if name == "B":
                assert not torch.isfinite(y[0, :2, j:]).any()
                assert not torch.isfinite(S[0, :2, :, 9]).any()
                others = [c for c in range(32) if c != 9]
                same(S[0, :2][:, :, others], S0[0, :2][:, :, others])
            else:
                assert not torch.isfinite(y[0, :2, j]).any()
                same(y[0, :2, j + 1:], y0[0, :2, j + 1:])
                same(S, S0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_steps(bad, dt):
    a, k = inputs(1, 2, 1, 150, 64, 64, dt, seed=4)
    y0, S0 = osdn.ssm_forward(**a, **k)
    for j in AT:
        keep = a["dt"][0, 0, j].clone()
        a["dt"][0, 0, j] = bad
        y, S = osdn.ssm_forward(**a, **k)
        a["dt"][0, 0, j] = keep
        same(y[0, 1], y0[0, 1]), same(S[0, 1], S0[0, 1])
        same(y[0, 0, :j], y0[0, 0, :j])
        assert not torch.isfinite(y[0, 0, j:]).any()
        assert not torch.isfinite(S[0, 0]).any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", ["x", "dy", "dt", "B", "C", "S0"])
def test_gradients_of_others_stay(name, dt):
    """Other heads, groups and batch entries keep their gradients' bits."""
    a, k = inputs(2, 6, 2, 150, 64, 32, dt, seed=6)
    dy, dS = adjoints(a, k)
    g0 = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    t = dict(a, **k, dy=dy)[name]
    t[(0, 0, 70) if name != "S0" else (0, 0)] = NAN
    g = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    one = name in ("x", "dy", "dt", "S0")        # a head's own, or its group's
    heads = list(range(1 if one else 3, 6))
    for n in ("x", "dt", "S0"):
        same(g[n][1], g0[n][1])
        same(g[n][0, heads], g0[n][0, heads])
    for n in ("B", "C"):
        same(g[n][1], g0[n][1])
        same(g[n][0, 1], g0[n][0, 1])
    for n in ("A", "D", "dt_bias"):
        same(g[n][heads], g0[n][heads])
    assert any(bool(v.isnan().any()) for v in g.values())
