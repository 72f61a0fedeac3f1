"""The recurrence's workgroups over several tiles in a row, against the fp64 oracle: what
is carried from tile to tile, the two join buffers in turn, the rows and states of later
tiles. In bf16 with an even number of channels, from 512 tokens on, a tile of the forward
is 256 tokens (16 a thread), else 128; the backward's is 128. Channels are independent, so
that the oracle walks a few of them: the first, the last and some between."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, f64, held, spoil, split_rows
from oracle import layer as Y

pytestmark = pytest.mark.gpu


def tiles_in_a_row(B, T, C, tile):
    """Tiles of one workgroup: the maps' workspace tells the number of segments."""
    need = osdn.glr_forward_workspace_bytes(B, T, C)
    segments = max(1, need // (B * 2 * C * 4))
    tiles = -(-T // tile)
    return -(-tiles // segments)


def check(B, T, C, dt, gate, normalize, lens, seed):
    g = torch.Generator().manual_seed(seed)
    x, r, i = split_rows(B, T, (C, C, C), dt, g, extra=2)
    A = -torch.exp(torch.rand(C, generator=g) * 8 - 7).to(DEV)
    L = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    dy = torch.randn((B, T, C), generator=g).to(dt).to(DEV)
    for t in (x, r, i, dy):
        spoil(t, L)
    h0, dh = (torch.randn((B, C), generator=g).to(DEV) for _ in range(2))
    k = dict(i=i if gate else None, h0=h0, lengths=L, normalize=normalize)
    y, h_T, states = osdn.glr_forward(x, r, A, save=True, **k)
    d = osdn.glr_backward(x, r, A, dy, dh_T=dh, states=states, **k)
    e = osdn.glr_backward(x, r, A, dy, dh_T=dh, **k)
    torch.cuda.synchronize()
    assert all(d[n] is None or torch.equal(d[n], e[n]) for n in d)

    pick = np.unique(np.r_[0:9, C - 9:C, np.random.default_rng(seed).integers(0, C, 14)])
    of = lambda t: None if t is None else f64(t[..., pick])
    rk = dict(i=of(k["i"]), h0=of(h0), lengths=lens, normalize=normalize)
    a = of(x), of(r), of(A)
    ry, rh, rb = Y.glr_ref(*a, **rk)
    my, mh, mb = Y.glr_ref(np.abs(a[0]), a[1], a[2], **dict(rk, h0=np.abs(rk["h0"])))
    u = 48 + T / 16
    held(y[..., pick], ry, (u, my), what="y")
    held(h_T[..., pick], rh, (u, mh), what="h_T")
    held(states[..., pick], rb[:, ::16], (u, mb[:, ::16]), what="states")
    ref, mag = Y.glr_backward_ref(*a, of(dy), dh_T=of(dh), **rk)
    u = 112 + T / 8
    for n in ref:
        held(d[n][..., pick], ref[n], (u, mag[n]), what="d" + n)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("B,T,C,lens", [
    (3, 777, 4098, [777, 300, 513]),       # whole sequences
    (3, 1024, 4096, None),                 # whole tiles and blocks of channels
    (2, 1900, 2050, [1900, 1281]),         # three segments
    (1, 3001, 2600, None)])
def test_tiles_in_a_row(B, T, C, lens, normalize, gate, dt):
    assert tiles_in_a_row(B, T, C, 256) >= 2
    check(B, T, C, dt, gate, normalize, lens, seed=T)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_tiles_in_a_row_of_odd_channels(dt):
    assert tiles_in_a_row(3, 777, 4097, 128) >= 2
    check(3, 777, 4097, dt, True, True, [640, 777, 0], seed=1)


@pytest.mark.parametrize("C", [64, 63])
def test_around_512_tokens(C):
    """Where the longer runs begin."""
    for T in (511, 512, 513):
        check(2, T, C, BF, True, True, None, seed=T)
