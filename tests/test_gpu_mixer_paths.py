"""Paths that the operators around the recurrences take at sizes of their own: the
heads of a group in turn in one workgroup of the scan's backward, rows past one
pass of the norms' backward. Each test first asserts, from the size of the
workspace, that its size takes the path it is there for."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import DEV, U, f64, held, rows
from oracle import mixer as M
from test_gpu_ssm import adjoints, check_backward, check_l2, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def scan_workspace(B, H, G, T, P, N, dt, parts):
    """Bytes of the scan backward's workspace with one walk a stream and the
    heads of a group in `parts` parts."""
    Q = 64 if dt is BF else 32
    nch = -(-T // Q)
    up = lambda n, m: -(-n // m) * m
    decays = up(B * H * nch * (9 * Q + 20) * 4, 256)
    floats = 2 * B * H * nch * P * N + up(3 * B * nch * H, 4)
    floats += 2 * parts * B * G * T * N if parts > 1 else 0
    return up(decays + 4 * floats, 256)


# B, H, G, T, P, N, dtype, parts, heads of a part
HEADS = [
    (64, 4, 1, 70, 32, 32, BF, 2, 2),
    (48, 5, 1, 65, 64, 32, BF, 3, 2),       # the last part has one head
    (64, 4, 1, 66, 128, 64, BF, 2, 2),
    (128, 6, 2, 5, 128, 128, BF, 1, 3),     # one part: sums leave directly
    (64, 4, 2, 40, 64, 64, F32, 1, 2),
    (40, 7, 1, 35, 32, 128, F32, 4, 2),
    (128, 6, 2, 3, 128, 128, F32, 1, 3),
]


@pytest.mark.parametrize("lens", [False, True])
@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c[:6])) + "-%d" % c[7])
def test_scan_backward_heads_in_turn(case, lens):
    B, H, G, T, P, N, dt, parts, hper = case
    print("case:", case, lens, flush=True)
    assert hper > 1 and parts == -(-(H // G) // hper)
    assert (osdn.ssm_backward_workspace_bytes(B, H, G, T, P, N, dt)
            == scan_workspace(B, H, G, T, P, N, dt, parts))
    n = np.random.default_rng(B).integers(0, T + 1, B)
    n[0], n[1] = T, 0
    a, k = inputs(B, H, G, T, P, N, dt, lens=n.tolist() if lens else None, seed=B + T)
    dy, dS = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    torch.cuda.synchronize()
    ref = check_backward(a, k, dy, dS, got)
    check_l2(got, ref, ("dt", "A", "D", "dt_bias", "S0"), 1e-5)
    check_l2(got, ref, ("x", "B", "C"), 3 * U[BF] if dt is BF else 1e-5)


@pytest.mark.parametrize("dt,B,H,G,T", [(BF, 4, 16, 2, 2048), (F32, 2, 12, 3, 1500)])
def test_scan_backward_of_a_training_batch(dt, B, H, G, T):
    """Eight and four heads in turn, over whole sequences, against the same heads
    each in a group of its own, keys and queries repeated: one head a workgroup.
    fp32 results lie within 1e-5 of the exact ones on both sides, dx within three
    halves steps; dB and dC are off by one rounding of the sum on one side and one
    of every head's on the other."""
    P = N = 128
    a, k = inputs(B, H, G, T, P, N, dt, seed=21)
    dy, dS = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    one = dict(a, B=a["B"].repeat_interleave(H // G, 1), C=a["C"].repeat_interleave(H // G, 1))
    want = osdn.ssm_backward(**one, dy=dy, dS_T=dS, **k)
    torch.cuda.synchronize()

    def rel(x, y):
        return float((x.double() - y.double()).norm() / y.double().norm())
    for n in ("dt", "A", "D", "dt_bias", "S0"):
        print("d%s: %.2e" % (n, rel(got[n], want[n])), flush=True)
        assert rel(got[n], want[n]) <= 2e-5, n
    assert rel(got["x"], want["x"]) <= (6 * U[BF] if dt is BF else 2e-5)
    for n in ("B", "C"):
        heads = want[n].double().view(B, G, H // G, T, N)
        total, u = heads.sum(2), U[dt]
        bound = u * total.norm() + u * sum(heads[:, :, h].norm() for h in range(H // G))
        err = (got[n].double() - total).norm()
        print("d%s: %.2e of %.2e" % (n, err, bound), flush=True)
        assert err <= bound + (2e-5 * total.norm()), n


# rows B, heads, T, D, dtype, gate, weight per head
GATED = [
    (3, 16, 367, 128, BF, True, False),     # 1101 rows, 1024 a pass
    (2, 64, 150, 128, F32, True, True),     # 300 rows, 256 a pass
    (1, 8, 4301, 64, BF, True, True),       # 4096 a pass
    (1, 8, 4099, 64, F32, False, False),
]


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("case", GATED, ids=lambda c: "-".join(map(str, c)))
def test_gated_norm_backward_rows_in_turn(case, gate_first):
    B, H, T, D, dt, gated, ph = case
    print("case:", case, gate_first, flush=True)
    need = osdn.gated_norm_backward_workspace_bytes
    assert need(B, H, T, D) == need(B, H, T - 4, D) > 0      # no more partial rows
    g = torch.Generator().manual_seed(T)
    x = (torch.randn((B, H, T, D), generator=g) * 0.5).to(dt).to(DEV)
    z = rows((B, T, H * D), dt, g, 8) if gated else None
    w = (1 + 0.1 * torch.randn((H, D) if ph else D, generator=g)).to(DEV)
    dy = torch.randn((B, T, H * D), generator=g).to(dt).to(DEV)
    got = osdn.gated_norm_backward(x, z, w, dy, gate_first=gate_first)
    torch.cuda.synchronize()
    rx, rz, rw, rdy = f64(x), f64(z), f64(w), f64(dy)
    gr = M.gated_norm_backward_ref(rx, rz, rw, rdy, gate_first=gate_first)
    heads = lambda t: t.reshape(B, T, H, D)
    xt, zt = rx.transpose(0, 2, 1, 3), (None if z is None else heads(rz))
    gate = np.ones_like(xt) if z is None else np.abs(M.silu(zt))
    v = np.abs(xt) * gate if gate_first else np.abs(xt)
    r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6)
    up = np.abs(heads(rdy)) * (1 if gate_first else gate)
    dn = up * np.abs(rw)
    dv = r * dn + v * (v * dn).mean(-1, keepdims=True) * r ** 3
    f = 1 + (0 if z is None else np.abs(zt))
    held(got["x"], gr["x"], (dv * (gate if gate_first else 1) * f).transpose(0, 2, 1, 3),
         2 * D + 64, what="dx")
    mw = up * v * r * f
    held(got["weight"], gr["weight"], mw.sum((0, 1)) if ph else mw.sum((0, 1, 2)),
         2 * D + 128, what="dweight")
    if gated:
        dg = dv * np.abs(xt) if gate_first else np.abs(heads(rdy)) * v * r * np.abs(rw)
        slope = M.sigmoid(zt) * (1 + np.abs(zt))
        held(got["z"], gr["z"], (dg * slope * f).reshape(B, T, H * D), 2 * D + 64, what="dz")


# rows, width, dtype, dtype of h: rows of one wave, four a workgroup
RES = [
    (4097, 129, F32, F32),          # off 16 bytes
    (8201, 20, BF, F32),
    (8200, 24, BF, BF),
    (4101, 1000, BF, BF),           # two vectors a lane
    (4101, 1501, BF, F32),          # three, off 16 bytes
]


@pytest.mark.parametrize("case", RES, ids=lambda c: "-".join(map(str, c)))
def test_residual_norm_backward_rows_in_turn(case):
    R, C, dt, rt = case
    print("case:", case, flush=True)
    need = osdn.residual_norm_backward_workspace_bytes
    assert need(R, C) == need(R - 4, C) > 0
    g = torch.Generator().manual_seed(R + C)
    h = torch.randn((R, C), generator=g).to(rt).to(DEV)
    dy = torch.randn((R, C), generator=g).to(dt).to(DEV)
    dh = torch.randn((R, C), generator=g).to(rt).to(DEV)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(DEV)
    got = osdn.residual_norm_backward(dy, h, w, dh, scale=0.5)
    torch.cuda.synchronize()
    hh, dd, ww = f64(h), f64(dy), f64(w)
    gr = M.residual_norm_backward_ref(dd, hh, ww, f64(dh), 0.5)
    ar = 1 / np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-6)
    dn = np.abs(dd * ww)
    m = ar * dn + np.abs(hh) * (np.abs(hh) * dn).mean(-1, keepdims=True) * ar ** 3
    m = m + np.abs(f64(dh))
    k = C / 64 + 64
    held(got["residual"], gr["residual"], m, k, what="dh")
    held(got["x"], gr["x"], 0.5 * m, k, what="dx")
    held(got["weight"], gr["weight"], (np.abs(dd * hh) * ar).sum(0), k + R / 64 + 64,
         what="dweight")
