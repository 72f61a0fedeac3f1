"""Host-side checks of the operators that complete a block (no GPU): the C entry
points refuse bad arguments before anything is launched, and the Python binding
refuses tensors it cannot pass on. The pointers handed to the C calls are never
followed."""
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
P = [0x1000000 * k for k in range(1, 24)]
X, R, I, A, H0, LEN, Y, HT, ST, WS, DY, DH, DX, DR, DI, DA, D0 = P[:17]


@needs_lib
def test_recurrence_refusals():
    L = osdn.load_library()
    need = L.glr_forward_workspace_bytes(2, 1024, 64)
    assert need > 0 and need % 256 == 0
    assert L.glr_forward_workspace_bytes(2, 8, 64) == 0        # one segment
    assert L.glr_forward_workspace_bytes(-1, 8, 64) == 0

    def fwd(B=2, T=1024, C=64, dt=BF16, x=X, bs=1 << 17, ts=128, r=R, rts=64, i=I,
            its=64, a=A, h0=H0, le=None, y=Y, hT=HT, st=ST, ws=WS, wsb=need):
        return L.glr_forward(B, T, C, dt, x, bs, ts, r, 1 << 17, rts, i, 1 << 17, its,
                             a, h0, le, 1, y, hT, st, ws, wsb, None)
    for bad in (dict(x=None), dict(r=None), dict(a=None)):
        assert fwd(**bad) == NULL_ARG, bad
    for bad in (dict(B=-1), dict(T=-1), dict(C=-1), dict(bs=-1), dict(ts=-1),
                dict(rts=-64), dict(its=-1), dict(T=(1 << 30) + 1)):
        assert fwd(**bad) == BAD_DIMS, bad
    for bad in (dict(dt=5), dict(C=(1 << 22) + 1), dict(ts=(1 << 22) + 1),
                dict(its=(1 << 22) + 1)):
        assert fwd(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=WS + 64)):
        assert fwd(**bad) == WORKSPACE, bad
    for bad in (dict(y=X), dict(y=R + 64), dict(hT=H0), dict(st=I), dict(hT=Y + 8),
                dict(ws=X), dict(le=Y),
                dict(y=X + 2 * ((1 << 17) + 1023 * 128 + 63))):  # x's last element
        assert fwd(**bad) == ALIASING, bad
    assert fwd(B=0, x=None, r=None, a=None) == OK
    assert fwd(C=0, x=None, r=None, a=None) == OK

    def dec(T=1, x=X, h=H0, ho=H0, y=Y):
        return L.glr_decode(2, T, 64, BF16, x, 64, 64, R, 64, 64, None, 0, 0, A, h, 1, y,
                            ho, None)
    for bad in (dict(h=None), dict(ho=None), dict(x=None), dict(y=None)):
        assert dec(**bad) == NULL_ARG, bad
    assert dec(ho=H0 + 4) == ALIASING and dec(y=H0) == ALIASING
    assert dec(T=0, x=None, y=None) == OK                       # already there

    need1 = L.glr_backward_workspace_bytes(2, 1024, 64, 1)
    need0 = L.glr_backward_workspace_bytes(2, 1024, 64, 0)
    assert need0 >= need1 + 2 * 64 * 64 * 4

    def bwd(i=I, st=ST, dy=DY, dx=DX, dr=DR, di=DI, dA=DA, d0=D0, ws=WS, wsb=need1):
        return L.glr_backward(2, 1024, 64, BF16, X, 1 << 16, 64, R, 1 << 16, 64, i,
                              1 << 16, 64, A, H0, None, 1, st, dy, DH, dx, dr, di, dA,
                              d0, ws, wsb, None)
    for bad in (dict(dy=None), dict(dx=None), dict(dr=None), dict(di=None), dict(dA=None)):
        assert bwd(**bad) == NULL_ARG, bad
    for bad in (dict(ws=None), dict(wsb=need1 - 1), dict(st=None)):
        assert bwd(**bad) == WORKSPACE, bad
    for bad in (dict(dx=X), dict(dr=DX), dict(di=DY), dict(d0=DH), dict(ws=ST),
                dict(dA=A)):
        assert bwd(**bad) == ALIASING, bad


@needs_lib
def test_rotary_refusals():
    L = osdn.load_library()
    Q, K, WQ, WK, FR, PO, YQ, YK = P[:8]

    def fwd(B=2, T=8, Hq=2, Hk=1, D=64, rot=64, dt=BF16, q=Q, qts=128, k=K, kts=64,
            norm=1, fr=FR, po=PO, le=None, yq=YQ, yk=YK):
        return L.qk_rotary_forward(B, T, Hq, Hk, D, rot, dt, q, 1024, qts, k, 512, kts,
                                   WQ, WK, norm, 1e-6, fr, 0, po, le, yq, yk, None)
    for bad in (dict(q=None), dict(k=None), dict(yq=None), dict(yk=None), dict(fr=None)):
        assert fwd(**bad) == NULL_ARG, bad
    for bad in (dict(B=-1), dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(rot=-16),
                dict(qts=-1), dict(kts=-1), dict(Hq=1 << 23)):
        assert fwd(**bad) == BAD_DIMS, bad
    for bad in (dict(D=48), dict(rot=8), dict(rot=80), dict(dt=2), dict(norm=3),
                dict(norm=-1)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(yq=YQ + 8) == MISALIGNED and fwd(yk=YK + 2) == MISALIGNED
    for bad in (dict(yq=Q), dict(yk=YQ), dict(yk=Q + 128), dict(yq=PO), dict(yk=FR)):
        assert fwd(**bad) == ALIASING, bad
    assert fwd(B=0, q=None, k=None, yq=None, yk=None) == OK
    need = L.qk_rotary_backward_workspace_bytes(2, 8, 64)
    assert need > 0 and need % 256 == 0
    assert L.qk_rotary_backward_workspace_bytes(2, 8, 48) == 0

    def bwd(dt=BF16, dydt=BF16, q=Q, dyq=P[8], dyk=P[9], dq=P[10], dk=P[11], dwq=P[12],
            dwk=P[13], ws=P[14], wsb=need):
        return L.qk_rotary_backward(2, 8, 2, 1, 64, 64, dt, dydt, q, 1024, 128, K, 512,
                                    64, WQ, WK, 1, 1e-6, FR, 0, PO, None, dyq, dyk, dq,
                                    dk, dwq, dwk, ws, wsb, None)
    for bad in (dict(q=None), dict(dyq=None), dict(dyk=None), dict(dq=None), dict(dk=None)):
        assert bwd(**bad) == NULL_ARG, bad
    assert bwd(dt=F32, dydt=BF16) == UNSUPPORTED and bwd(dydt=9) == UNSUPPORTED
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=P[14] + 128)):
        assert bwd(**bad) == WORKSPACE, bad
    assert bwd(dq=P[10] + 4) == MISALIGNED and bwd(dyk=P[9] + 8) == MISALIGNED
    for bad in (dict(dq=P[8]), dict(dk=P[10]), dict(dwk=P[12]), dict(dwq=WQ), dict(ws=Q)):
        assert bwd(**bad) == ALIASING, bad


@needs_lib
def test_feed_forward_refusals():
    L = osdn.load_library()
    Xx, G, U, Hh, GA, UP, W, DHh, DXx, DG, DU = P[:11]
    need = L.gated_ffn_forward_workspace_bytes(96, 4096, 128, BF16)
    assert need > 0 and L.gated_ffn_forward_workspace_bytes(8, 4096, 128, BF16) == 0
    assert L.gated_ffn_forward_workspace_bytes(96, 4096, 128, 7) == 0

    def fwd(R=96, C=4096, F=128, dt=BF16, x=Xx, xs=4096, g=G, u=U, act=0, h=Hh, ga=None,
            up=None, ws=W, wsb=need):
        return L.gated_ffn_forward(R, C, F, dt, x, xs, g, u, act, h, ga, up, ws, wsb, None)
    for bad in (dict(x=None), dict(g=None), dict(u=None), dict(h=None), dict(ga=GA),
                dict(up=UP)):
        assert fwd(**bad) == NULL_ARG, bad
    for bad in (dict(R=-1), dict(C=-1), dict(F=-1), dict(xs=-1), dict(R=(1 << 31) + 1)):
        assert fwd(**bad) == BAD_DIMS, bad
    for bad in (dict(dt=3), dict(act=3), dict(act=-1), dict(C=(1 << 21) + 1),
                dict(F=(1 << 21) + 1), dict(xs=(1 << 21) + 1)):
        assert fwd(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=W + 2)):
        assert fwd(**bad) == WORKSPACE, bad
    for bad in (dict(h=Xx), dict(h=G + 64), dict(ga=Hh, up=UP), dict(ga=GA, up=GA),
                dict(ws=U)):
        assert fwd(**bad) == ALIASING, bad
    assert fwd(R=0, x=None, h=None) == OK and fwd(F=0, h=None) == OK
    need = L.gated_ffn_backward_workspace_bytes(96, 4096, 128, BF16)

    def bwd(x=Xx, g=G, ga=GA, up=UP, act=0, dh=DHh, dx=DXx, dg=DG, du=DU, ws=W, wsb=need):
        return L.gated_ffn_backward(96, 4096, 128, BF16, x, 4096, g, U, ga, up, act, dh, dx,
                                    dg, du, ws, wsb, None)
    for bad in (dict(x=None), dict(g=None), dict(ga=None), dict(up=None), dict(dh=None),
                dict(dx=None), dict(dg=None), dict(du=None)):
        assert bwd(**bad) == NULL_ARG, bad
    assert bwd(act=7) == UNSUPPORTED
    for bad in (dict(ws=None), dict(wsb=need - 256), dict(ws=W + 8)):
        assert bwd(**bad) == WORKSPACE, bad
    for bad in (dict(dx=Xx), dict(dg=G), dict(du=DG), dict(dx=DHh), dict(ws=GA)):
        assert bwd(**bad) == ALIASING, bad


def test_binding_refuses_host_tensors_and_types():
    t = torch.zeros(2, 4, 64)
    a = torch.zeros(64)
    calls = [lambda x: osdn.glr_forward(x, x, a), lambda x: osdn.glr_decode(x, x, a, a),
             lambda x: osdn.glr_backward(x, x, a, x),
             lambda x: osdn.qk_rotary_forward(x, x, 64),
             lambda x: osdn.qk_rotary_backward(x, x, x, x, 64),
             lambda x: osdn.gated_ffn_forward(x, a, a),
             lambda x: osdn.gated_ffn_backward(x, a, a, x, x, x)]
    for f in calls:
        with pytest.raises(ValueError, match="HIP device"):
            f(t)
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            f(t.half())
        with pytest.raises(TypeError):
            f([1.0])


def test_exported_names():
    for n in osdn.layer.__all__:
        assert n in osdn.__all__ and callable(getattr(osdn, n))
    assert osdn.layer.GLR_INTERVAL == 16


def test_import_needs_no_gpu():
    code = ("import delta_rule_recurrent_scan_amd as o;"
            "assert o.glr_forward and o.qk_rotary_forward and o.gated_ffn_forward")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
