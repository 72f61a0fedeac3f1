"""GPU parity of the selective scan (forward, decode, backward) against the
fp64 token recurrence."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import DEV, U, f64, held
from oracle import mixer as M

BF, F32 = torch.bfloat16, torch.float32
# bf16 matrix operands: scores and states rounded once for the outputs; three
# parts (2^-24) where a sum leaves in fp32
OP1 = {BF: U[BF], F32: 0.0}
OP2 = {BF: U[BF] ** 3, F32: 0.0}
K = 320  # fp32 roundings: T terms in chunks, N or P products, decays, exps


def inputs(B, H, G, T, P, N, dt, seed=0, lens=None, A=(1.0, 16.0), state=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    a = dict(x=n(B, H, T, P).to(dt), dt=n(B, H, T),
             A=-(torch.rand(H, generator=g) * (A[1] - A[0]) + A[0]),
             B=n(B, G, T, N).to(dt), C=n(B, G, T, N).to(dt))
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    k = dict(D=1 + 0.1 * n(H), dt_bias=torch.log(torch.expm1(step)),
             S0=n(B, H, P, N) * N ** -0.5 if state else None,
             lengths=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    dev = lambda t: None if t is None else t.to(DEV)
    return {m: dev(t) for m, t in a.items()}, {m: dev(t) for m, t in k.items()}


def ref_args(a, k):
    r = {m: f64(t) for m, t in a.items()}
    q = {m: f64(t) for m, t in k.items()}
    q["lengths"] = None if k["lengths"] is None else k["lengths"].cpu().numpy()
    ab = dict(r, **{m: np.abs(r[m]) for m in ("x", "B", "C")})
    qb = dict(q, D=None if q["D"] is None else np.abs(q["D"]),
              S0=None if q["S0"] is None else np.abs(q["S0"]))
    return r, q, ab, qb


def check_forward(a, k, got, softplus=True, what=""):
    dt = a["x"].dtype
    r, q, ab, qb = ref_args(a, k)
    ry, rS = M.ssm_ref(**r, **q, use_softplus=softplus)
    my, mS = M.ssm_ref(**ab, **qb, use_softplus=softplus)
    held(got[0], ry, my, K, OP1[dt], what + "y")
    held(got[1], rS, mS, K, OP2[dt], what + "S_T")


# B, H, G, T, P, N, dtype, lengths
CASES = [
    (2, 4, 2, 130, 64, 128, BF, None),
    (1, 2, 1, 1, 128, 128, BF, None),
    (3, 6, 3, 65, 32, 32, BF, [65, 0, 17]),
    (1, 3, 1, 64, 64, 64, BF, None),
    (2, 2, 2, 63, 128, 32, BF, [63, 1]),
    (1, 5, 5, 17, 32, 128, BF, None),
    (1, 2, 1, 16, 128, 64, BF, None),
    (2, 4, 1, 100, 64, 128, F32, [100, 33]),
    (1, 2, 2, 31, 128, 128, F32, None),
    (2, 3, 1, 97, 32, 32, F32, None),
    (1, 4, 2, 48, 128, 32, F32, None),
    (1, 2, 1, 2, 32, 64, F32, None),
    # long enough for several segments
    (1, 2, 1, 1100, 64, 64, BF, None),
    (2, 1, 1, 777, 128, 128, BF, [777, 400]),
    (1, 2, 2, 700, 32, 32, F32, [650]),
]
IDS = ["-".join(map(str, c[:6])) + ("-f32" if c[6] is F32 else "-bf16")
       + ("-lens" if c[7] else "") for c in CASES]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    print("case:", case, flush=True)
    B, H, G, T, P, N, dt, lens = case
    a, k = inputs(B, H, G, T, P, N, dt, lens=lens)
    got = osdn.ssm_forward(**a, **k)
    torch.cuda.synchronize()
    check_forward(a, k, got)
    if lens:
        for b, n in enumerate(lens):
            assert not got[0][b, :, n:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [150, 900])
def test_forward_plain_options(T):
    """No D, bias, state or softplus; steps of zero among the tokens."""
    a, k = inputs(1, 2, 1, T, 64, 64, BF)
    a["dt"] = (a["dt"].abs() * 0.1)
    a["dt"][:, :, ::7] = 0
    k.update(D=None, dt_bias=None, S0=None)
    got = osdn.ssm_forward(**a, **k, softplus=False)
    check_forward(a, k, got, softplus=False)


@pytest.mark.gpu
@pytest.mark.parametrize("A", [(0.0, 0.0), (200.0, 2000.0), (-0.02, -0.01)],
                         ids=["none", "strong", "growth"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_forward_decay_range(A, dt):
    """No decay at all, decays that empty the state within a token, growth."""
    a, k = inputs(1, 2, 1, 200, 64, 64, dt, A=A)
    if A[0] < 0:
        a["dt"].clamp_(max=1.0)
    check_forward(a, k, osdn.ssm_forward(**a, **k))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [200, 900])
def test_padding_is_never_used(T):
    lens = [T, 70, 0]
    a, k = inputs(3, 2, 1, T, 64, 64, BF, lens=lens)
    y, S = osdn.ssm_forward(**a, **k)
    for b, n in enumerate(lens):
        for m in ("x", "B", "C"):
            a[m][b, :, n:] = float("nan")
        a["dt"][b, :, n:] = float("inf")
    y2, S2 = osdn.ssm_forward(**a, **k)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    assert torch.equal(S[2], k["S0"][2])


@pytest.mark.gpu
def test_forward_state_in_place_and_no_tokens():
    a, k = inputs(2, 2, 1, 600, 64, 64, BF)
    y, S = osdn.ssm_forward(**a, **k)
    S0 = k["S0"].clone()
    y2, S2 = osdn.ssm_forward(**a, **dict(k, S0=S0), out=(torch.empty_like(y), S0))
    assert S2 is S0 and torch.equal(S2, S) and torch.equal(y2, y)
    y3, S3 = osdn.ssm_forward(**a, **k, out=(torch.empty_like(y), None))
    assert S3 is None and torch.equal(y3, y)
    a, k = inputs(2, 2, 1, 0, 64, 64, BF)
    y, S = osdn.ssm_forward(**a, **k)
    assert y.shape == (2, 2, 0, 64) and torch.equal(S, k["S0"])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in CASES if c[7] is None and c[3] <= 130],
                         ids=lambda c: "-".join(map(str, c[:6])))
def test_decode(case):
    """The decode recurrence over all tokens: fp32 arithmetic throughout."""
    print("case:", case, flush=True)
    B, H, G, T, P, N, dt, _ = case
    a, k = inputs(B, H, G, T, P, N, dt)
    k.pop("lengths")
    S0 = k.pop("S0")
    S = torch.empty_like(S0)
    y = osdn.ssm_decode(**a, S=S0, S_out=S, **k)
    torch.cuda.synchronize()
    k.update(S0=S0, lengths=None)
    r, q, ab, qb = ref_args(a, k)
    ry, rS = M.ssm_ref(**r, **q)
    my, mS = M.ssm_ref(**ab, **qb)
    held(y, ry, my, K, what="y")
    held(S, rS, mS, K, what="S")


@pytest.mark.gpu
def test_decode_continues_forward():
    T, cut = 90, 83
    a, k = inputs(2, 4, 2, T, 64, 128, BF)
    k.pop("lengths")
    S0 = k.pop("S0")
    sl = lambda i, j: {m: (t if m == "A" else t[:, :, i:j].contiguous())
                       for m, t in a.items()}
    y, S = osdn.ssm_forward(**sl(0, cut), S0=S0, **k)
    out = [y]
    for t in range(cut, T):
        out.append(osdn.ssm_decode(**sl(t, t + 1), S=S, **k))
    k.update(S0=S0, lengths=None)
    check_forward(a, k, (torch.cat(out, 2), S), what="prompt then tokens ")


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------

def adjoints(a, k, seed=9):
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(a["x"].shape, generator=g).to(a["x"].dtype).to(DEV)
    nb, H, T, P = a["x"].shape
    N = a["B"].shape[-1]
    dS = (torch.randn((nb, H, P, N), generator=g) * N ** -0.5).to(DEV)
    return dy, dS


def check_backward(a, k, dy, dS, got, softplus=True):
    dt = a["x"].dtype
    r, q, ab, qb = ref_args(a, k)
    ref = M.ssm_backward_ref(**r, dy=f64(dy), dS_T=f64(dS), **q, use_softplus=softplus)
    ady, adS = np.abs(f64(dy)), None if dS is None else np.abs(f64(dS))
    mag = M.ssm_backward_ref(**ab, dy=ady, dS_T=adS, **qb, use_softplus=softplus,
                             bound=True)
    # inside a chunk the decay's gradient is a suffix sum of row minus column
    # sums: its rounding goes by the chunk's pairs, not by those crossing t
    own = mag.pop("own", np.zeros_like(r["dt"]))
    T = own.shape[2]
    pairs = np.zeros_like(own)
    for c in range(0, T, 64):
        pairs[:, :, c:c + 64] = 2 * own[:, :, c:c + 64].sum(2, keepdims=True)
    absA = np.abs(r["A"])
    mag["dt"] = mag["dt"] + absA[None, :, None] * pairs
    mag["dt_bias"] = mag["dt_bias"] + absA * pairs.sum((0, 2))
    step = M._steps(r["dt"], q["dt_bias"], softplus)
    mag["A"] = mag["A"] + (np.abs(step) * pairs).sum((0, 2))
    for n in ("x", "B", "C"):
        held(got[n], ref[n], mag[n], 2 * K, 2 * OP1[dt], "d" + n)
    for n in ("dt", "A", "D", "dt_bias", "S0"):
        held(got[n], ref[n], mag[n], 2 * K, OP2[dt], "d" + n)
    return ref


def check_l2(got, ref, names, tol):
    for n in names:
        e = np.linalg.norm(f64(got[n]) - ref[n]) / max(np.linalg.norm(ref[n]), 1e-30)
        print("d%s: rel L2 %.2e" % (n, e), flush=True)
        assert e <= tol, (n, e)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    print("case:", case, flush=True)
    B, H, G, T, P, N, dt, lens = case
    a, k = inputs(B, H, G, T, P, N, dt, lens=lens, seed=1)
    dy, dS = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    torch.cuda.synchronize()
    ref = check_backward(a, k, dy, dS, got)
    # and as a whole: 2 K independent fp32 roundings of terms some 6 times the
    # sums they cancel to (sqrt(640) 2^-24 6 = 9e-6)
    check_l2(got, ref, ("dt", "A", "D", "dt_bias", "S0"), 1e-5)
    # one rounding of the output and two of operands, half a step at most each
    check_l2(got, ref, ("x", "B", "C"), 3 * U[BF] if dt is BF else 1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [100, 600])
def test_backward_plain_options(dt, T):
    """No D, bias, states, adjoint of the state or softplus; zero steps."""
    a, k = inputs(2, 4, 1, T, 64, 64, dt, seed=2)
    a["dt"] = a["dt"].abs() * 0.1
    a["dt"][:, :, ::7] = 0
    k.update(D=None, dt_bias=None, S0=None)
    dy, _ = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, softplus=False, **k)
    check_backward(a, k, dy, None, got, softplus=False)


@pytest.mark.gpu
@pytest.mark.parametrize("A", [(0.0, 0.0), (200.0, 2000.0)], ids=["none", "strong"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_decay_range(A, dt):
    a, k = inputs(1, 2, 1, 200, 64, 64, dt, A=A, seed=3)
    dy, dS = adjoints(a, k)
    check_backward(a, k, dy, dS, osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [200, 900])
def test_backward_padding_is_never_used(T):
    lens = [T, 70, 0]
    a, k = inputs(3, 2, 1, T, 64, 64, BF, lens=lens, seed=4)
    dy, dS = adjoints(a, k)
    g1 = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    for b, n in enumerate(lens):
        for m in ("x", "B", "C"):
            a[m][b, :, n:] = float("nan")
        a["dt"][b, :, n:] = float("nan")
        dy[b, :, n:] = float("nan")
    g2 = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    for m in g1:
        assert torch.equal(g1[m], g2[m]), m
    for b, n in enumerate(lens):
        for m in ("x", "dt", "B", "C"):
            assert not g2[m][b, :, n:].any()
    assert torch.equal(g2["S0"][2], dS[2])


@pytest.mark.gpu
def test_backward_no_tokens_and_no_batch():
    a, k = inputs(2, 2, 1, 0, 64, 64, BF)
    dy, dS = adjoints(a, k)
    g = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    assert torch.equal(g["S0"], dS)
    assert not any(bool(g[m].any()) for m in ("A", "D", "dt_bias"))
    a, k = inputs(0, 2, 1, 5, 64, 64, BF)
    dy, dS = adjoints(a, k)
    g = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    assert not any(bool(g[m].any()) for m in ("A", "D", "dt_bias"))


@pytest.mark.gpu
def test_backward_against_differences():
    """The gradients against central differences of the forward, fp32."""
    a, k = inputs(1, 2, 1, 70, 32, 32, F32, seed=6)
    dy, dS = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    gen = torch.Generator().manual_seed(7)

    def loss(p, q):
        y, S = osdn.ssm_forward(**p, **q)
        return float((y.double() * dy.double()).sum() + (S.double() * dS.double()).sum())
    for n in ("x", "dt", "A", "B", "C", "D", "dt_bias", "S0"):
        src = a if n in a else k
        d = torch.randn(src[n].shape, generator=gen).to(DEV)
        h = 2.0 ** -9

        def at(s):
            moved = {n: src[n] + s * d}
            return loss(dict(a, **moved) if n in a else a, dict(k, **moved) if n in k else k)
        num = (at(h) - at(-h)) / (2 * h)
        ana = float((got[n].double() * d.double()).sum())
        # fp32 outputs of size up to 10, some 6600 of them: 2^-24 * 10 * 80 of
        # noise over 2h, and h^2 times a third derivative of the gradient's size
        scale = float(got[n].double().norm() * d.double().norm())
        assert abs(num - ana) <= 2e-3 * scale + 5e-2, (n, num, ana)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("A", [1e30, 3e38])
def test_decays_beyond_any_exponent(dt, A):
    """Products dt A up to the end of fp32's range and past it: every decay is
    zero, and nothing is NaN."""
    a, k = inputs(1, 2, 1, 150, 64, 32, dt, seed=11)
    a["A"] = torch.tensor([-A, -1.0], device=DEV)
    a["dt"][:, :, ::5] = 30.0
    got = osdn.ssm_forward(**a, **k)
    check_forward(a, k, got)
    dy, dS = adjoints(a, k)
    g = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    assert all(bool(torch.isfinite(t).all()) for t in g.values())
    assert float(g["A"][0]) == 0.0
    check_l2({n: g[n] for n in ("x", "B", "C")},
             M.ssm_backward_ref(**ref_args(a, k)[0], dy=f64(dy), dS_T=f64(dS),
                                **ref_args(a, k)[1]), ("x", "B", "C"),
             3 * U[BF] if dt is BF else 1e-5)
