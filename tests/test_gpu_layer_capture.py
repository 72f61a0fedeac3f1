"""The operators that complete a block under HIP graph capture, on other streams,
beside other calls, and on buffers with guards (as the tests of the operators around
the recurrences do it): guards and inputs keep their bits, every replay gives the
eager call's bits, graphs that share a workspace run in turn and calls on
workspaces of their own at once."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32
from test_gpu_guard import Arena, _bits, _same

pytestmark = pytest.mark.gpu


def case(name, dt, seed=0, T=150):
    """(function, positional inputs, keyword inputs, workspace bytes or None, whether
    the last positional input is updated in place)."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)
    a = lambda *s: n(*s).to(dt)
    B, C, D = 3, 71, 64
    L = torch.tensor([T, 0, T // 2], dtype=torch.int32, device=DEV)
    A = -(0.1 + n(C).abs())
    scan = (a(B, T, C), a(B, T, C), A)
    long = T * 8
    P = torch.randint(0, 1 << 20, (B, T), generator=g, dtype=torch.int32).to(DEV)
    f = (10000.0 ** -(torch.arange(16) / 16)).float().to(DEV)
    qk = dict(inv_freq=f, q_weight=n(D), k_weight=n(D), positions=P, lengths=L)
    R, W, F = T, 131, 77
    x, wg, wu = a(R, W), a(F, W), a(F, W)
    wide = (a(R, 4096), a(64, 4096), a(64, 4096))       # split over k
    ffn = osdn.gated_ffn_backward_workspace_bytes
    cases = dict(
        glr_forward=(scan, dict(i=a(B, T, C), h0=n(B, C), lengths=L), 0, False),
        glr_forward_segments=((a(2, long, 64), a(2, long, 64), -n(64).abs()),
                              dict(i=a(2, long, 64)),
                              osdn.glr_forward_workspace_bytes(2, long, 64), False),
        glr_decode=((a(B, 1, C), a(B, 1, C), A, n(B, C)), dict(i=a(B, 1, C)), None, True),
        glr_backward=(scan + (a(B, T, C),),
                      dict(i=a(B, T, C), h0=n(B, C), dh_T=n(B, C), lengths=L),
                      osdn.glr_backward_workspace_bytes(B, T, C, False), False),
        glr_backward_segments=((a(2, long, 64), a(2, long, 64), -n(64).abs(),
                                a(2, long, 64)), dict(i=a(2, long, 64)),
                               osdn.glr_backward_workspace_bytes(2, long, 64, False),
                               False),
        qk_rotary_forward=((a(B, T, 3 * D), a(B, T, 2 * D), D), qk, None, False),
        qk_rotary_backward=((a(B, T, 3 * D), a(B, T, 2 * D), a(B, 3, T, D),
                             a(B, 2, T, D), D), qk,
                            osdn.qk_rotary_backward_workspace_bytes(B, T, D), False),
        gated_ffn_forward=((x, wg, wu), {}, osdn.gated_ffn_forward_workspace_bytes(
            R, W, F, dt), False),
        gated_ffn_forward_rows=((x[:9].contiguous(), wg, wu), {}, 0, False),
        gated_ffn_forward_parts=(wide, {}, osdn.gated_ffn_forward_workspace_bytes(
            R, 4096, 64, dt), False),
        gated_ffn_backward=((x, wg, wu, a(R, F), a(R, F), a(R, F)), {},
                            ffn(R, W, F, dt), False),
        gated_ffn_backward_parts=(wide + (a(R, 64), a(R, 64), a(R, 64)), {},
                                  ffn(R, 4096, 64, dt), False))
    fn = getattr(osdn, "_".join(p for p in name.split("_")
                                if p not in ("segments", "rows", "parts")))
    args, kw, need, moved = cases[name]
    if fn in (osdn.glr_forward, osdn.gated_ffn_forward):
        kw = dict(kw, save=True)
    return fn, args, kw, need, moved


NAMES = ["glr_forward", "glr_forward_segments", "glr_decode", "glr_backward",
         "glr_backward_segments", "qk_rotary_forward", "qk_rotary_backward",
         "gated_ffn_forward", "gated_ffn_forward_rows", "gated_ffn_forward_parts",
         "gated_ffn_backward", "gated_ffn_backward_parts"]
SHARED = [n for n in NAMES if "segments" in n or "parts" in n or "backward" in n]
both = pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])


def each(out, f):
    if isinstance(out, dict):
        return {k: f(t) for k, t in out.items()}
    if isinstance(out, tuple):
        return tuple(f(t) for t in out)
    return f(out)


def tensors(out):
    return (list(out.values()) if isinstance(out, dict) else
            list(out) if isinstance(out, tuple) else [out])


def prepared(name, dt, seed=0, ws=None, T=150):
    """(run, what it writes, the eager results, reset)."""
    fn, args, kw, need, moved = case(name, dt, seed, T)
    first = args[-1].clone() if moved else None

    def reset():
        if moved:
            args[-1].copy_(first)
    out = fn(*args, **kw)
    eager = [t.clone() for t in tensors(out) + ([args[-1]] if moved else [])]
    reset()
    out = each(out, torch.empty_like)
    kw = dict(kw, out=out)
    kw.pop("save", None)
    if need is not None:
        kw["workspace"] = (torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
                           if ws is None else ws[:max(need, 1)])
    return (lambda: fn(*args, **kw)), tensors(out) + ([args[-1]] if moved else []), eager, reset


def equal(outs, eager):
    torch.cuda.synchronize()
    for a, b in zip(outs, eager):
        assert torch.equal(_bits(a), _bits(b))


def blank(outs, name):
    for t in outs[:-1] if name == "glr_decode" else outs:
        t.fill_(float("nan"))


@both
@pytest.mark.parametrize("name", NAMES)
def test_guards(name, dt):
    fn, args, kw, need, moved = case(name, dt)
    last = args[-1].clone() if moved else None
    ref = fn(*args[:-1], last, **kw) if moved else fn(*args, **kw)
    a = Arena()
    gargs = [a.inp(t) for t in args]
    if moved:
        base, v, _ = a.bufs[-1]
        a.bufs[-1] = (base, v, None)
    gkw = {k: a.inp(t) for k, t in kw.items()}
    gkw.pop("save", None)
    gkw["out"] = each(ref, a.out)
    if need is not None:
        gkw["workspace"] = a.workspace(need)
    got = fn(*gargs, **gkw)
    a.check()
    _same(got, ref)
    if moved:
        _same(gargs[-1], last)


@both
@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name, dt):
    run, outs, eager, reset = prepared(name, dt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        blank(outs, name)
        reset()
        prepared(name, dt, seed=5)          # eager calls of the same operator
        torch.cuda.synchronize()
        g.replay()
        equal(outs, eager)


@pytest.mark.parametrize("name", SHARED)
def test_two_graphs_share_a_workspace_in_turn(name):
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    pair = [prepared(name, BF, seed, ws, T) for seed, T in ((0, 150), (1, 270))]
    graphs = []
    for run, *_ in pair:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1)):
        for _, outs, _, _ in pair:
            blank(outs, name)
        ws.fill_(0xA5)                       # nothing is kept in it between calls
        for i in order:
            graphs[i].replay()
        for _, outs, eager, _ in pair:
            equal(outs, eager)


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once_on_two_streams(name):
    pair = [prepared(name, BF, seed) for seed in (0, 1)]
    streams = [torch.cuda.Stream() for _ in pair]
    for _ in range(3):
        for _, outs, _, reset in pair:
            blank(outs, name)
            reset()
        torch.cuda.synchronize()
        for (run, *_), s in zip(pair, streams):
            with torch.cuda.stream(s):
                run()
        for _, outs, eager, _ in pair:
            equal(outs, eager)
