"""The fp64 oracle of the operators around the recurrences: its gradients
against central differences of its forward, and its forward against closed
cases (no GPU)."""
import numpy as np
import pytest

from oracle import mixer as M

RNG = np.random.default_rng


def _diff(f, args, name, grad, rng, h=1e-6):
    """Directional central difference of f along a random direction of one
    argument against the gradient's inner product with it."""
    a = args[name]
    d = rng.standard_normal(a.shape)
    up, dn = dict(args), dict(args)
    up[name], dn[name] = a + h * d, a - h * d
    num = (f(up) - f(dn)) / (2 * h)
    ana = float((grad * d).sum())
    # the step's own error is h^2 f''' and cancellation 1e-16 |f| / h
    assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana), abs(num)), (name, num, ana)


@pytest.mark.parametrize("l2norm", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lengths", [None, [7, 0, 1]])
def test_short_conv_gradients(W, l2norm, lengths):
    r = RNG(W)
    B, T, H, D = 3, 7, 2, 5
    C = H * D
    a = dict(x=r.standard_normal((B, T, C)), weight=r.standard_normal((C, W)),
             bias=r.standard_normal(C), state=r.standard_normal((B, W - 1, C)))
    dy, dst = r.standard_normal((B, H, T, D)), r.standard_normal((B, W - 1, C))

    def f(p):
        y, tail, _ = M.short_conv_ref(p["x"], p["weight"], p["bias"], p["state"],
                                      lengths, D, True, l2norm, 1e-3)
        return float((y * dy).sum() + (tail * dst).sum())
    g = M.short_conv_backward_ref(a["x"], a["weight"], dy, a["bias"], a["state"],
                                  lengths, D, True, l2norm, 1e-3, dst)
    for n in a:
        _diff(f, a, n, g[n], r)


@pytest.mark.parametrize("use_softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [6, 0]])
def test_ssm_gradients(use_softplus, lengths):
    r = RNG(5)
    nb, H, G, T, P, N = 2, 4, 2, 6, 3, 5
    a = dict(x=r.standard_normal((nb, H, T, P)),
             dt=r.standard_normal((nb, H, T)) + (0 if use_softplus else 2),
             A=-r.uniform(0.2, 1.0, H), B=r.standard_normal((nb, G, T, N)),
             C=r.standard_normal((nb, G, T, N)), D=r.standard_normal(H),
             dt_bias=0.1 * r.standard_normal(H),
             S0=r.standard_normal((nb, H, P, N)))
    dy, dS = r.standard_normal((nb, H, T, P)), r.standard_normal((nb, H, P, N))

    def f(p):
        y, S = M.ssm_ref(p["x"], p["dt"], p["A"], p["B"], p["C"], p["D"],
                         p["dt_bias"], p["S0"], lengths, use_softplus)
        return float((y * dy).sum() + (S * dS).sum())
    g = M.ssm_backward_ref(a["x"], a["dt"], a["A"], a["B"], a["C"], dy, a["D"],
                           a["dt_bias"], a["S0"], dS, lengths, use_softplus)
    for n in a:
        _diff(f, a, n, g[n], r)


def test_ssm_closed_cases():
    r = RNG(6)
    x, B, C = (r.standard_normal(s) for s in ((1, 2, 5, 3), (1, 1, 5, 4), (1, 1, 5, 4)))
    # no decay, unit steps: a causal linear attention
    y, S = M.ssm_ref(x, np.ones((1, 2, 5)), np.zeros(2), B, C, use_softplus=False)
    scores = np.tril(C[0, 0] @ B[0, 0].T)
    assert np.allclose(y[0, 1], scores @ x[0, 1])
    assert np.allclose(S[0, 1], x[0, 1].T @ B[0, 0])
    # no step: the state stays and only D x leaves
    S0 = r.standard_normal((1, 2, 3, 4))
    y, S = M.ssm_ref(x, np.zeros((1, 2, 5)), -np.ones(2), B, C, np.full(2, 2.0),
                     S0=S0, use_softplus=False)
    assert np.allclose(S, S0)
    assert np.allclose(y[0, 0], 2 * x[0, 0] + C[0, 0] @ S0[0, 0].T)


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("gate", [True, False])
def test_gated_norm_gradients(gate_first, per_head, gate):
    r = RNG(7)
    B, H, T, D = 2, 3, 4, 5
    a = dict(x=r.standard_normal((B, H, T, D)),
             weight=r.standard_normal((H, D) if per_head else D))
    if gate:
        a["z"] = r.standard_normal((B, T, H * D))
    dy = r.standard_normal((B, T, H * D))

    def f(p):
        return float((M.gated_norm_ref(p["x"], p.get("z"), p["weight"], 1e-3,
                                       gate_first) * dy).sum())
    g = M.gated_norm_backward_ref(a["x"], a.get("z"), a["weight"], dy, 1e-3,
                                  gate_first)
    for n in a:
        _diff(f, a, n, g[n], r)


def test_residual_norm_gradients():
    r = RNG(8)
    a = dict(x=r.standard_normal((6, 9)), residual=r.standard_normal((6, 9)),
             weight=r.standard_normal(9))
    dy, dh = r.standard_normal((6, 9)), r.standard_normal((6, 9))

    def f(p):
        y, h = M.residual_norm_ref(p["x"], p["weight"], p["residual"], 0.3, 1e-3)
        return float((y * dy).sum() + (h * dh).sum())
    _, h = M.residual_norm_ref(a["x"], a["weight"], a["residual"], 0.3, 1e-3)
    g = M.residual_norm_backward_ref(dy, h, a["weight"], dh, 0.3, 1e-3)
    for n in a:
        _diff(f, a, n, g[n], r)
