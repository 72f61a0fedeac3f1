"""The fp64 oracle of the operators that complete a block: every gradient against
central differences, the forwards against closed forms, and planted mistakes that
the differences have to find."""
import numpy as np
import pytest

from oracle import layer as Y

H = 1e-6


def numeric(f, x):
    """Central differences of the scalar f at x."""
    g = np.zeros_like(x)
    for k in np.ndindex(x.shape):
        at = x[k]
        x[k] = at + H
        up = f()
        x[k] = at - H
        g[k] = (up - f()) / (2 * H)
        x[k] = at
    return g


def near(got, want):
    assert np.abs(got - want).max() <= 1e-6 * (1 + np.abs(want).max())


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_recurrence_gradients(normalize, gate):
    g = np.random.default_rng(0)
    B, T, C = 2, 5, 3
    x, r, dy = (g.standard_normal((B, T, C)) for _ in range(3))
    i = g.standard_normal((B, T, C)) if gate else None
    A = -np.exp(g.standard_normal(C))
    h0, dh = g.standard_normal((B, C)), g.standard_normal((B, C))
    lens = [5, 3]

    def loss():
        y, h_T, _ = Y.glr_ref(x, r, A, i, h0, lens, normalize)
        return (dy * y).sum() + (dh * h_T).sum()
    got, mag = Y.glr_backward_ref(x, r, A, dy, i, h0, dh, lens, normalize)
    for n, t in dict(x=x, r=r, i=i, A=A, h0=h0).items():
        if t is not None:
            near(got[n], numeric(loss, t))
            assert np.all(mag[n] >= np.abs(got[n]) - 1e-12), n


def test_recurrence_closed_forms():
    g = np.random.default_rng(1)
    x, r = g.standard_normal((1, 4, 2)), g.standard_normal((1, 4, 2))
    # no decay: a sum of the inputs; with the input factor, nothing comes in
    h0 = g.standard_normal((1, 2))
    y, h_T, _ = Y.glr_ref(x, r, np.zeros(2), None, h0, None, False)
    near(y, h0[:, None] + np.cumsum(x, 1))
    near(Y.glr_ref(x, r, np.zeros(2), None, h0)[1], h0)
    # a constant gate: a geometric series
    A = np.array([-0.3, -2.0])
    y, _, before = Y.glr_ref(x, np.full_like(r, 40.0), A)
    a = np.exp(A)
    m = np.sqrt(1 - a * a)
    want = sum(a ** (3 - t) * m * x[0, t] for t in range(4))
    near(y[0, 3], want)
    near(before[0, 3], y[0, 2])


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradients(norm, interleaved):
    g = np.random.default_rng(2)
    B, T, Hn, D = 2, 3, 2, 32
    x = g.standard_normal((B, T, Hn * D))
    dy = g.standard_normal((B, Hn, T, D))
    w = 1 + 0.1 * g.standard_normal(D)
    f = 10000.0 ** -(np.arange(8) / 8)
    pos = np.array([[3, 4, 100], [0, 7, 9]])
    k = dict(inv_freq=f, weight=w, positions=pos, lengths=[3, 2], norm=norm,
             interleaved=interleaved, eps=1e-3)

    def loss():
        return (dy * Y.qk_rotary_ref(x, D, **k)[0]).sum()
    got, mag = Y.qk_rotary_backward_ref(x, dy, D, **k)
    near(got["x"], numeric(loss, x))
    near(got["weight"], numeric(loss, w))
    assert np.all(mag["x"] >= np.abs(got["x"]) - 1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_distances(interleaved):
    g = np.random.default_rng(3)
    D, f = 32, 10000.0 ** -(np.arange(16) / 16)
    q, k = g.standard_normal((1, 1, D)), g.standard_normal((1, 1, D))

    def at(x, p):
        return Y.qk_rotary_ref(x, D, f, positions=[[p]], norm="none",
                               interleaved=interleaved)[0][0, 0, 0]
    near(np.linalg.norm(at(q, 17)), np.linalg.norm(q))
    near(at(q, 17) @ at(k, 12), at(q, 105) @ at(k, 100))
    near(at(q, 0), q[0, 0])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_feed_forward_gradients(act):
    g = np.random.default_rng(4)
    x, wg, wu = (g.standard_normal(s) for s in ((4, 3), (5, 3), (5, 3)))
    dh = g.standard_normal((4, 5))

    def loss():
        return (dh * Y.gated_ffn_ref(x, wg, wu, act)[0]).sum()
    _, gate, up = Y.gated_ffn_ref(x, wg, wu, act)
    got, dg, du = Y.gated_ffn_backward_ref(x, wg, wu, gate, up, dh, act)
    for n, t in dict(x=x, w_gate=wg, w_up=wu).items():
        near(got[n], numeric(loss, t))
    # the two forms of GELU are near each other
    if act != "silu":
        z = np.linspace(-4, 4, 50)
        a, b = Y.activation(z, "gelu"), Y.activation(z, "gelu_tanh")
        assert np.abs(a[0] - b[0]).max() < 5e-4 and np.abs(a[1] - b[1]).max() < 3e-3


@pytest.mark.parametrize("mistake", ["m", "rho", "before", "sign"])
def test_mistakes_are_found(mistake):
    """A term of the recurrence's adjoint dropped or taken wrong is further from the
    differences than the bound."""
    g = np.random.default_rng(5)
    x, r, dy = (g.standard_normal((1, 4, 2)) for _ in range(3))
    A = np.array([-0.5, -1.5])

    def loss():
        return (dy * Y.glr_ref(x, r, A)[0]).sum()
    want = numeric(loss, r)
    rho, la, a, m = Y.glr_factors(r, A)
    _, _, before = Y.glr_ref(x, r, A)
    c, out = np.zeros((1, 2)), np.zeros_like(r)
    for t in range(3, -1, -1):
        now = c + dy[:, t]
        b = Y.glr_ref(x, r, A)[0][:, t] if mistake == "before" else before[:, t]
        w = 0 if mistake == "m" else a[:, t] ** 2 / m[:, t] * x[:, t]
        dla = now * (a[:, t] * b + (w if mistake == "sign" else -w))
        out[:, t] = dla * la[:, t] * (1 if mistake == "rho" else 1 - rho[:, t])
        c = a[:, t] * now
    assert np.abs(out - want).max() > 1e-3 * np.abs(want).max()
