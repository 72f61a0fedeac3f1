"""Calls of the operators that complete a block that their documentation allows and that
ordinary use seldom makes: one tensor in several places, rows and entries broadcast,
channels beside the range that hold NaN, workspaces made inside a capture, captures of
both passes while the eager ones live. Each gives the bits of the plain call."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])


def rand(*s, dt=F32, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(dt).to(DEV)


def flat(out):
    return (list(out.values()) if isinstance(out, dict) else
            list(out) if isinstance(out, tuple) else [out])


def same(a, b):
    torch.cuda.synchronize()
    a, b = flat(a), flat(b)
    assert len(a) == len(b)
    for s, t in zip(a, b):
        assert (s is None and t is None) or torch.equal(s, t)


@both
@pytest.mark.parametrize("R", [5, 40, 90, 300])
@pytest.mark.parametrize("C", [72, 61])
def test_one_row_for_all(R, C, dt):
    """A row broadcast over R: a stride of zero."""
    row, wg, wu = rand(C, dt=dt), rand(40, C, dt=dt, seed=1), rand(40, C, dt=dt, seed=2)
    x, dh = row.expand(R, C), rand(R, 40, dt=dt, seed=3)
    f = osdn.gated_ffn_forward(x, wg, wu, save=True)
    same(f, osdn.gated_ffn_forward(x.contiguous(), wg, wu, save=True))
    same(osdn.gated_ffn_backward(x, wg, wu, f[1], f[2], dh),
         osdn.gated_ffn_backward(x.contiguous(), wg, wu, f[1], f[2], dh))


@both
def test_one_tensor_in_several_places(dt):
    x, A, dy = rand(2, 150, 66, dt=dt), -rand(66).abs(), rand(2, 150, 66, dt=dt, seed=1)
    c = lambda: x.clone()
    same(osdn.glr_forward(x, x, A, i=x, save=True),
         osdn.glr_forward(c(), c(), A, i=c(), save=True))
    same(osdn.glr_backward(x, x, A, x, i=x), osdn.glr_backward(c(), c(), A, c(), i=c()))
    e = x[:1].expand(2, 150, 66)                        # entries a stride of zero apart
    same(osdn.glr_forward(e, x, A, i=e), osdn.glr_forward(e.contiguous(), x, A,
                                                          i=e.contiguous()))
    t = x[:, :1].expand(2, 150, 66)                     # and tokens
    same(osdn.glr_backward(t, x, A, dy), osdn.glr_backward(t.contiguous(), x, A, dy))
    q = rand(2, 9, 128, dt=dt)
    f, w = torch.rand(16, device=DEV), rand(64)
    k = dict(inv_freq=f, q_weight=w, k_weight=w)
    same(osdn.qk_rotary_forward(q, q, 64, **k),
         osdn.qk_rotary_forward(q.clone(), q.clone(), 64, **k))
    z = q[:1, :1].expand(2, 9, 128)
    same(osdn.qk_rotary_forward(z, q, 64, **k),
         osdn.qk_rotary_forward(z.contiguous(), q, 64, **k))
    wg, h = rand(48, 66, dt=dt), rand(300, 48, dt=dt)
    same(osdn.gated_ffn_backward(x.view(300, 66), wg, wg, h, h, h),
         osdn.gated_ffn_backward(x.view(300, 66), wg, wg.clone(), h, h.clone(), h.clone()))


@both
@pytest.mark.parametrize("C,extra", [(72, 8), (72, 3), (61, 3), (64, 64)])
def test_what_lies_beside_a_range_is_never_used(C, extra, dt):
    """Rows in the middle of wider ones that are NaN elsewhere."""
    def inside(t):
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 2 * extra), float("nan"), dtype=dt,
                          device=DEV)
        wide[..., extra:extra + t.shape[-1]] = t
        return wide[..., extra:extra + t.shape[-1]]
    wg, wu = rand(40, C, dt=dt, seed=1), rand(40, C, dt=dt, seed=2)
    for R in (7, 90):
        x, dh = rand(R, C, dt=dt), rand(R, 40, dt=dt, seed=3)
        f = osdn.gated_ffn_forward(x, wg, wu, save=True)
        same(osdn.gated_ffn_forward(inside(x), wg, wu, save=True), f)
        same(osdn.gated_ffn_backward(inside(x), wg, wu, f[1], f[2], dh),
             osdn.gated_ffn_backward(x, wg, wu, f[1], f[2], dh))
    x, r, i, dy = (rand(2, 300, C, dt=dt, seed=s) for s in range(4))
    A = -rand(C).abs()
    same(osdn.glr_forward(inside(x), inside(r), A, i=inside(i)),
         osdn.glr_forward(x, r, A, i=i))
    same(osdn.glr_backward(inside(x), inside(r), A, dy, i=inside(i)),
         osdn.glr_backward(x, r, A, dy, i=i))


@both
def test_capture_of_both_passes_beside_eager_ones(dt):
    """Results and workspaces from the capture's own pool, the eager results alive."""
    x, r, A, dy = rand(2, 1100, 64, dt=dt), rand(2, 1100, 64, dt=dt, seed=1), -rand(64).abs(), \
        rand(2, 1100, 64, dt=dt, seed=2)
    R, C, F = 130, 515, 72
    a, wg, wu, dh = (rand(*s, dt=dt, seed=k) for k, s in enumerate(
        ((R, C), (F, C), (F, C), (R, F))))
    q, dq, f = rand(2, 40, 128, dt=dt), rand(2, 2, 40, 64, dt=dt, seed=4), torch.rand(
        32, device=DEV)
    w = rand(64)

    def step():
        y, h_T, st = osdn.glr_forward(x, r, A, save=True)
        g = osdn.glr_backward(x, r, A, dy, dh_T=h_T, states=st)
        n = osdn.glr_backward(x, r, A, dy)
        h, gate, up = osdn.gated_ffn_forward(a, wg, wu, save=True)
        b = osdn.gated_ffn_backward(a, wg, wu, gate, up, dh)
        p = osdn.qk_rotary_forward(q, None, 64, inv_freq=f, q_weight=w)
        d = osdn.qk_rotary_backward(q, None, dq, None, 64, inv_freq=f, q_weight=w)
        return [t for o in ((y, h_T, st), g, n, (h, gate, up), b, p, d) for t in flat(o)]
    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            if t is not None:
                t.fill_(float("nan"))
        again = step()
        torch.cuda.synchronize()
        graph.replay()
        same(tuple(out), tuple(eager))
        same(tuple(again), tuple(eager))
