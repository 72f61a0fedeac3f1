"""Selective scan in segments: few (batch, head) pairs of long sequences, padded and
not, forward and backward, against the fp64 oracle and with NaN behind the lengths.
Each case first asserts, from the size of the workspaces, that it is cut."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import U
from test_gpu_ssm import (adjoints, check_backward, check_forward, check_l2, inputs)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def up(n, m):
    return -(-n // m) * m


def forward_segments(B, H, T, dt):
    Q = 64 if dt is BF else 32
    nch = -(-T // Q)
    want = min(-(-512 // (B * H)), nch // 2)
    per = -(-nch // (want if want >= 4 else 1))
    return -(-nch // per)


def forward_bytes(B, H, T, P, N, dt, nseg):
    Q = 64 if dt is BF else 32
    decays = up(B * H * -(-T // Q) * (9 * Q + 20) * 4, 256)
    return up(decays + (B * H * nseg * (P * N + 1) * 4 if nseg > 1 else 0), 256)


def walk_segments(B, H, T, P, dt):
    nch = -(-T // (64 if dt is BF else 32))
    streams = 2 * B * H * max(1, P // 64)
    want = min(-(-256 // streams), nch // 4)
    per = -(-nch // (want if want >= 4 else 1))
    return -(-nch // per)


def backward_bytes(B, H, G, T, P, N, dt, nseg, parts):
    Q = 64 if dt is BF else 32
    nch = -(-T // Q)
    decays = up(B * H * nch * (9 * Q + 20) * 4, 256)
    floats = 2 * B * H * (nch + nseg - 1) * P * N + up(2 * B * H * (nseg - 1), 4)
    floats += up(3 * B * nch * H, 4) + (2 * parts * B * G * T * N if parts > 1 else 0)
    return up(decays + 4 * floats, 256)


# B, H, G, T, P, N, dtype, lengths, head parts of the backward
CASES = [
    (1, 2, 1, 1100, 64, 64, BF, None, 2),
    (2, 2, 1, 1090, 128, 128, BF, [1090, 500], 2),
    (3, 2, 2, 1025, 32, 128, BF, [1025, 0, 64], 1),
    (1, 5, 1, 1500, 64, 32, BF, [1449], 5),
    (2, 3, 1, 600, 64, 64, F32, [600, 97], 3),
    (1, 2, 2, 530, 128, 128, F32, None, 1),
    (2, 2, 1, 700, 32, 32, F32, [33, 700], 2),
]
IDS = ["-".join(map(str, c[:6])) + ("-bf16" if c[6] is BF else "-f32") for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_segments(case):
    B, H, G, T, P, N, dt, lens, parts = case
    print("case:", case, flush=True)
    nf, nb = forward_segments(B, H, T, dt), walk_segments(B, H, T, P, dt)
    assert nf >= 4 and nb >= 4
    assert (osdn.ssm_forward_workspace_bytes(B, H, G, T, P, N, dt)
            == forward_bytes(B, H, T, P, N, dt, nf))
    assert (osdn.ssm_backward_workspace_bytes(B, H, G, T, P, N, dt)
            == backward_bytes(B, H, G, T, P, N, dt, nb, parts))
    a, k = inputs(B, H, G, T, P, N, dt, lens=lens, seed=T)
    dy, dS = adjoints(a, k)
    y, S = osdn.ssm_forward(**a, **k)
    check_forward(a, k, (y, S))
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    ref = check_backward(a, k, dy, dS, got)
    check_l2(got, ref, ("dt", "A", "D", "dt_bias", "S0"), 1e-5)
    check_l2(got, ref, ("x", "B", "C"), 3 * U[BF] if dt is BF else 1e-5)
    for b, n in enumerate(lens or []):
        for m in ("x", "B", "C", "dt"):
            a[m][b, :, n:] = float("nan")
        dy[b, :, n:] = float("nan")
    y2, S2 = osdn.ssm_forward(**a, **k)
    assert torch.equal(y2, y) and torch.equal(S2, S)
    g2 = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    for n in got:
        assert torch.equal(g2[n], got[n]), n
