"""Host-side checks of the operators around the recurrences (no GPU): the C
entry points refuse bad arguments before anything is launched, and the Python
binding refuses tensors it cannot pass on. The pointers handed to the C calls
are never followed."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn

(OK, NULL_ARG, BAD_DIMS, UNSUPPORTED, WORKSPACE, ALIASING, HIP,
 MISALIGNED) = range(8)
F32, BF16 = 0, 1
needs_lib = pytest.mark.skipif(not os.path.exists(osdn.library_path()),
                               reason="libosdn.so not built")
X, Y, WT, BI, ST, SO, LEN, DY, DX, WS = (0x1000000 * i for i in range(1, 11))
Z, DZ, G1, G2, G3, G4, G5 = (0x1000000 * i for i in range(11, 18))


@needs_lib
def test_strerror_knows_alignment():
    assert b"aligned" in osdn.load_library().osdn_strerror(MISALIGNED)


@needs_lib
def test_short_conv_refusals():
    L = osdn.load_library()

    def fwd(B=2, T=8, H=2, D=32, W=4, dt=BF16, x=X, bs=512, ts=64, w=WT, b=BI,
            st=ST, le=None, l2=0, y=Y, so=SO):
        return L.short_conv_forward(B, T, H, D, W, dt, x, bs, ts, w, b, st, le, 1,
                                    l2, 1e-6, y, so, None)
    assert fwd(x=None) == NULL_ARG and fwd(w=None) == NULL_ARG
    assert fwd(y=None) == NULL_ARG
    for bad in (dict(B=-1), dict(T=-1), dict(H=-1), dict(D=0), dict(bs=-1),
                dict(ts=-64), dict(H=1 << 20, D=1 << 12)):
        assert fwd(**bad) == BAD_DIMS, bad
    for bad in (dict(W=1), dict(W=5), dict(dt=7), dict(D=48, l2=1)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(y=X + 64) == ALIASING                 # y over x
    assert fwd(y=X + 2 * (512 + 7 * 64 + 63)) == ALIASING   # x's last element
    assert fwd(so=ST) == ALIASING                    # in place: decode only
    assert fwd(so=Y + 8) == ALIASING
    assert fwd(le=Y) == ALIASING
    assert fwd(B=0, x=None, y=None, w=None) == OK
    assert fwd(H=0, x=None, y=None, w=None) == OK

    def dec(T=1, st=ST, so=ST, x=X, y=Y):
        return L.short_conv_decode(2, T, 2, 32, 4, BF16, x, 64, 64, WT, None, st, 1,
                                   0, 1e-6, y, so, None)
    assert dec(st=None) == NULL_ARG and dec(so=None) == NULL_ARG
    assert dec(so=ST + 4) == ALIASING                # partial overlap
    assert dec(T=0, x=None, y=None) == OK            # the state is already there

    need = L.short_conv_backward_workspace_bytes(2, 8, 2, 32, 4)
    assert need > 0 and need % 256 == 0
    assert L.short_conv_backward_workspace_bytes(2, 8, 2, 32, 9) == 0
    assert L.short_conv_backward_workspace_bytes(0, 8, 2, 32, 4) == 0

    def bwd(dt=BF16, dydt=BF16, x=X, dy=DY, dx=DX, ds=G1, dw=G2, db=G3, ws=WS,
            wsb=need):
        return L.short_conv_backward(2, 8, 2, 32, 4, dt, dydt, x, 512, 64, WT, BI,
                                     ST, None, 1, 0, 1e-6, dy, None, dx, ds, dw,
                                     db, ws, wsb, None)
    assert bwd(dy=None) == NULL_ARG and bwd(dx=None) == NULL_ARG
    assert bwd(dw=None) == NULL_ARG
    assert bwd(dt=F32, dydt=BF16) == UNSUPPORTED
    assert bwd(dydt=3) == UNSUPPORTED
    assert bwd(ws=None) == WORKSPACE and bwd(wsb=need - 1) == WORKSPACE
    assert bwd(ws=WS + 16) == WORKSPACE
    assert bwd(dx=X) == ALIASING and bwd(db=G2) == ALIASING
    assert bwd(ws=DY) == ALIASING


@needs_lib
def test_norm_refusals():
    L = osdn.load_library()

    def gf(B=2, H=2, T=4, D=32, dt=BF16, x=X, z=Z, bs=256, ts=64, w=WT, y=Y):
        return L.gated_norm_forward(B, H, T, D, dt, x, z, bs, ts, w, 0, 1e-6, 0, y,
                                    None)
    assert gf(x=None) == NULL_ARG and gf(w=None) == NULL_ARG
    assert gf(T=-1) == BAD_DIMS and gf(ts=-1) == BAD_DIMS
    assert gf(z=None, ts=-1, y=X) == ALIASING        # no gate: strides unread
    assert gf(D=48) == UNSUPPORTED and gf(dt=2) == UNSUPPORTED
    assert gf(x=X + 8) == MISALIGNED and gf(y=Y + 2) == MISALIGNED
    assert gf(y=Z) == ALIASING
    assert gf(T=0, x=None, y=None, w=None) == OK

    need = L.gated_norm_backward_workspace_bytes(2, 2, 4, 32)
    assert need > 0

    def gb(H=2, z=Z, dz=DZ, dy=DY, dx=DX, dw=G2, ws=WS, wsb=need, ph=0):
        return L.gated_norm_backward(2, H, 4, 32, BF16, X, z, 256, 64, WT, ph, 1e-6,
                                     0, dy, dx, dz, dw, ws, wsb, None)
    assert gb(dz=None) == NULL_ARG and gb(dw=None) == NULL_ARG
    assert gb(dx=DX + 4) == MISALIGNED
    assert gb(wsb=0) == WORKSPACE and gb(ws=None) == WORKSPACE
    assert gb(dx=X) == ALIASING and gb(dz=DX) == ALIASING
    assert gb(H=0, ph=1, dw=None) == OK

    def rf(R=4, C=64, dt=BF16, rt=F32, x=X, r=ST, w=WT, y=Y, h=SO):
        return L.residual_norm_forward(R, C, dt, rt, x, r, 1.0, w, 1e-6, y, h, None)
    assert rf(x=None) == NULL_ARG and rf(y=None) == NULL_ARG
    assert rf(R=-1) == BAD_DIMS and rf(C=-1) == BAD_DIMS
    assert rf(C=16385) == UNSUPPORTED and rf(dt=F32, rt=BF16) == UNSUPPORTED
    assert rf(h=ST + 16) == ALIASING and rf(y=X) == ALIASING
    assert rf(R=0, x=None, y=None, w=None) == OK
    need = L.residual_norm_backward_workspace_bytes(4, 64)

    def rb(C=64, dy=DY, h=X, dh=ST, dx=DX, dr=G1, dw=G2, ws=WS, wsb=need):
        return L.residual_norm_backward(4, C, BF16, F32, dy, h, dh, 1.0, WT, 1e-6,
                                        dx, dr, dw, ws, wsb, None)
    assert rb(dy=None) == NULL_ARG and rb(dw=None) == NULL_ARG
    assert rb(wsb=need - 1) == WORKSPACE
    assert rb(dr=ST) == ALIASING and rb(dx=DY) == ALIASING
    assert L.residual_norm_backward_workspace_bytes(4, 16385) == 0
    assert need >= 64 * 4


@needs_lib
def test_ssm_refusals():
    L = osdn.load_library()
    need = L.ssm_forward_workspace_bytes(1, 2, 1, 2048, 64, 64, BF16)
    assert need > 0 and need % 256 == 0
    assert L.ssm_forward_workspace_bytes(1, 2, 1, 0, 64, 64, BF16) == 0
    assert L.ssm_forward_workspace_bytes(1, 3, 2, 2048, 64, 64, BF16) == 0

    def fwd(B=1, H=2, G=1, T=2048, P=64, N=64, dt=BF16, x=X, d=DY, A=WT, Bm=Z,
            Cm=DZ, S0=None, y=Y, S=SO, ws=WS, wsb=need, le=None):
        return L.ssm_forward(B, H, G, T, P, N, dt, x, d, A, Bm, Cm, None, None, 1,
                             S0, le, y, S, ws, wsb, None)
    for bad in (dict(x=None), dict(d=None), dict(A=None), dict(Bm=None),
                dict(Cm=None), dict(y=None)):
        assert fwd(**bad) == NULL_ARG, bad
    for bad in (dict(B=-1), dict(G=0), dict(H=3, G=2), dict(T=-4), dict(G=-1)):
        assert fwd(**bad) == BAD_DIMS, bad
    for bad in (dict(P=48), dict(N=16), dict(dt=3)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(ws=None) == WORKSPACE and fwd(wsb=need - 1) == WORKSPACE
    assert fwd(ws=WS + 64) == WORKSPACE
    for bad in (dict(x=X + 2), dict(Bm=Z + 8), dict(y=Y + 4), dict(S=SO + 4)):
        assert fwd(**bad) == MISALIGNED, bad
    assert fwd(y=X) == ALIASING and fwd(S0=SO + 16) == ALIASING
    assert fwd(ws=Z) == ALIASING
    assert fwd(H=0, G=0, x=None, y=None) == OK and fwd(B=0, A=None) == OK

    def dec(T=1, S=ST, So=ST, x=X, y=Y):
        return L.ssm_decode(1, 2, 1, T, 64, 64, BF16, x, DY, WT, Z, DZ, None, None,
                            1, S, y, So, None)
    assert dec(S=None) == NULL_ARG and dec(So=None) == NULL_ARG
    assert dec(So=ST + 16) == ALIASING and dec(y=ST) == ALIASING
    assert dec(S=ST + 4, So=SO) == MISALIGNED
    assert dec(T=0, x=None, y=None) == OK


@needs_lib
def test_sizes_beyond_one_launch_are_refused():
    L = osdn.load_library()
    P = [i << 44 for i in range(1, 8)]
    r = lambda R: L.residual_norm_forward(R, 8, BF16, BF16, P[0], P[1], 1.0, P[2], 1e-6,
                                          P[3], P[4], None)
    assert r(1 << 26) == UNSUPPORTED and r(1 << 31) == UNSUPPORTED
    assert r((1 << 31) + 1) == BAD_DIMS
    big = (1 << 30) + 1
    assert L.ssm_forward_workspace_bytes(1, 1, 1, big, 32, 32, BF16) == 0
    assert L.ssm_forward_workspace_bytes(1, 1, 1, (1 << 31) - 1, 32, 32, BF16) == 0
    assert L.ssm_backward_workspace_bytes(1, 1, 1, big, 32, 32, F32) == 0
    assert L.short_conv_backward_workspace_bytes(1, (1 << 31) - 1, 1, 32, 4) == 0
    assert L.ssm_forward(1, 1, 1, big, 32, 32, BF16, P[0], P[1], P[2], P[3], P[4], None,
                         None, 1, None, None, P[5], None, P[6], 1 << 40, None) == BAD_DIMS
    assert L.short_conv_forward(1, big, 1, 32, 4, BF16, P[0], 0, 32, P[1], None, None, None,
                                1, 0, 1e-6, P[2], None, None) == BAD_DIMS
    assert L.ssm_decode(1 << 14, 1 << 10, 1, 1, 32, 32, BF16, P[0], P[1], P[2], P[3], P[4],
                        None, None, 1, P[5], P[6], P[5], None) == UNSUPPORTED


@needs_lib
def test_ssm_backward_refusals():
    L = osdn.load_library()
    assert L.ssm_backward_workspace_bytes(1, 3, 2, 256, 64, 64, BF16) == 0
    assert L.ssm_backward_workspace_bytes(1, 2, 1, 256, 48, 64, BF16) == 0
    need = L.ssm_backward_workspace_bytes(1, 2, 1, 256, 64, 64, BF16)
    assert need > 0 and need % 256 == 0
    at = {n: 0x1000000 * (i + 1) for i, n in enumerate(
        ("x", "dt", "A", "B", "C", "D", "bias", "S0", "dy", "dST", "gx", "gdt", "gA",
         "gB", "gC", "gD", "gbias", "gS0", "ws"))}

    def bwd(nb=1, H=2, G=1, T=256, P=64, N=64, code=BF16, wsb=need, le=None, **kw):
        p = dict(at, **kw)
        return L.ssm_backward(nb, H, G, T, P, N, code, p["x"], p["dt"], p["A"], p["B"],
                              p["C"], p["D"], p["bias"], 1, p["S0"], le, p["dy"],
                              p["dST"], p["gx"], p["gdt"], p["gA"], p["gB"], p["gC"],
                              p["gD"], p["gbias"], p["gS0"], p["ws"], wsb, None)
    for n in ("x", "dt", "A", "B", "C", "dy", "gx", "gdt", "gA", "gB", "gC"):
        assert bwd(**{n: None}) == NULL_ARG, n
    for bad in (dict(nb=-1), dict(G=0), dict(H=3, G=2), dict(T=-1)):
        assert bwd(**bad) == BAD_DIMS, bad
    for bad in (dict(P=16), dict(N=96), dict(code=2)):
        assert bwd(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=at["ws"] + 16)):
        assert bwd(**bad) == WORKSPACE, bad
    for n in ("x", "B", "C", "S0", "dy", "dST", "gx", "gB", "gC", "gS0"):
        assert bwd(**{n: at[n] + 4}) == MISALIGNED, n
    for a, b in (("gx", "x"), ("gx", "dy"), ("gdt", "dt"), ("gB", "B"), ("gC", "gB"),
                 ("gS0", "dST"), ("gS0", "S0"), ("gA", "A"), ("gD", "gA"),
                 ("ws", "gx"), ("ws", "C"), ("gbias", "bias")):
        assert bwd(**{a: at[b]}) == ALIASING, (a, b)
    assert bwd(le=at["gdt"]) == ALIASING
    assert bwd(H=0, G=0, x=None, gx=None) == OK


def test_binding_refuses_cpu_tensors_and_other_types():
    t = torch.zeros(1, 4, 64)
    w = torch.zeros(64, 4)
    with pytest.raises(ValueError, match="HIP device"):
        osdn.short_conv_forward(t, w)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        osdn.residual_norm_forward(t.half(), torch.zeros(64))
    with pytest.raises(TypeError):
        osdn.ssm_forward([1], t, t, t, t)
    x = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="HIP device"):
        osdn.gated_norm_forward(x, None, torch.zeros(64))
    with pytest.raises(ValueError, match="HIP device"):
        osdn.ssm_decode(x, x[..., 0], x[0, :, 0, 0], x, x, x)


@needs_lib
def test_calls_on_no_elements_need_no_gpu():
    """Nothing to launch: the C calls return before any HIP call, also in a
    process that sees no device."""
    code = ("import delta_rule_recurrent_scan_amd as o; L = o.load_library();"
            "assert L.ssm_forward(0,4,2,9,64,64,1,*[None]*7,1,*[None]*5,0,None)==0;"
            "assert L.residual_norm_forward(0,64,1,1,None,None,1.0,None,1e-6,"
            "None,None,None)==0")
    env = dict(os.environ, HIP_VISIBLE_DEVICES="")
    subprocess.run([sys.executable, "-c", code], check=True, env=env,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
