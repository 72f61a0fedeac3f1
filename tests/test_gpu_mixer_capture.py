"""The operators around the recurrences under HIP graph capture, on other
streams, beside other calls, and on buffers with guards.

Capture: every replay, with the program's own eager work and synchronisations
between, gives the eager call's bits. Two captured graphs that share a workspace
and run one after the other keep their results, and so do two that run at once
on workspaces of their own. Guards: each tensor is a view into the middle of an
allocation of its own, the workspace as long as the query says; 64 KiB of a
byte pattern on each side stay as they were, the inputs keep their bits and the
outputs are those of the call on ordinary buffers."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from test_gpu_guard import Arena, _bits, _same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def case(name, dt, seed=0, T=150):
    """(function, positional inputs, keyword inputs, workspace bytes or None,
    names of arguments that the call updates) of an entry point at ragged
    sizes."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)
    a = lambda *s: n(*s).to(dt)
    B, H, G, P, N, W, D = 3, 4, 2, 64, 32, 4, 64
    C = H * D
    L = torch.tensor([T, 0, T // 2], dtype=torch.int32, device=DEV)
    A = -(1 + n(H).abs())
    scan = (a(B, H, T, P), n(B, H, T), A, a(B, G, T, N), a(B, G, T, N))
    extra = dict(D=n(H), dt_bias=n(H))
    one = (a(B, H, 1, P), n(B, H, 1), A, a(B, G, 1, N), a(B, G, 1, N))
    rows = 71
    cases = dict(
        short_conv_forward=((a(B, T, C), n(C, W), n(C), a(B, W - 1, C), L),
                            dict(head_dim=D, l2norm=True), None, ()),
        short_conv_decode=((a(B, 1, C), n(C, W), a(B, W - 1, C), n(C)),
                           dict(head_dim=D), None, (2,)),
        short_conv_backward=((a(B, T, C), n(C, W), a(B, H, T, D), n(C),
                              a(B, W - 1, C), L),
                             dict(head_dim=D, l2norm=True, dstate_T=a(B, W - 1, C)),
                             osdn.short_conv_backward_workspace_bytes(B, T, H, D, W), ()),
        ssm_forward=(scan, dict(extra, S0=n(B, H, P, N), lengths=L),
                     osdn.ssm_forward_workspace_bytes(B, H, G, T, P, N, dt), ()),
        ssm_decode=(one + (n(B, H, P, N),), extra, None, (5,)),
        ssm_backward=(scan + (a(B, H, T, P),),
                      dict(extra, S0=n(B, H, P, N), dS_T=n(B, H, P, N), lengths=L),
                      osdn.ssm_backward_workspace_bytes(B, H, G, T, P, N, dt), ()),
        gated_norm_forward=((a(B, H, T, D), a(B, T, C), n(H, D)), {}, None, ()),
        gated_norm_backward=((a(B, H, T, D), a(B, T, C), n(H, D), a(B, T, C)), {},
                             osdn.gated_norm_backward_workspace_bytes(B, H, T, D), ()),
        residual_norm_forward=((a(rows, 515), n(515), n(rows, 515)),
                               dict(scale=0.5), None, ()),
        residual_norm_backward=((a(rows, 515), n(rows, 515), n(515), n(rows, 515)),
                                dict(scale=0.5),
                                osdn.residual_norm_backward_workspace_bytes(rows, 515),
                                ()))
    return (getattr(osdn, name),) + cases[name]


NAMES = ["short_conv_forward", "short_conv_decode", "short_conv_backward",
         "ssm_forward", "ssm_decode", "ssm_backward", "gated_norm_forward",
         "gated_norm_backward", "residual_norm_forward", "residual_norm_backward"]


def tensors(out):
    if isinstance(out, dict):
        return [t for t in out.values() if t is not None]
    return list(out) if isinstance(out, tuple) else [out]


def like(out):
    if isinstance(out, dict):
        return {k: None if t is None else torch.empty_like(t) for k, t in out.items()}
    if isinstance(out, tuple):
        return tuple(torch.empty_like(t) for t in out)
    return torch.empty_like(out)


def prepared(name, dt, seed=0, ws=None, T=150):
    """(run, outputs that run writes, eager results, reset): an entry point on
    preallocated outputs and workspace; reset restores what it updates."""
    fn, args, kw, need, moved = case(name, dt, seed, T)
    first = [args[i].clone() for i in moved]

    def reset():
        for i, t in zip(moved, first):
            args[i].copy_(t)
    eager = tensors(fn(*args, **kw)) + [args[i] for i in moved]
    eager = [t.clone() for t in eager]
    reset()
    out = like(fn(*args, **kw))
    reset()
    kw = dict(kw, out=out)
    if need is not None:
        kw["workspace"] = (torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
                           if ws is None else ws[:max(need, 1)])
    return (lambda: fn(*args, **kw)), tensors(out), eager, reset, [args[i] for i in moved]


def equal(outs, eager):
    torch.cuda.synchronize()
    for a, b in zip(outs, eager):
        assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", NAMES)
def test_guards(name, dt):
    fn, args, kw, need, moved = case(name, dt)
    ref_args = [t.clone() if i in moved else t for i, t in enumerate(args)]
    ref = fn(*ref_args, **kw)
    a = Arena()
    gargs = [a.inp(t) for t in args]
    gkw = {k: a.inp(t) for k, t in kw.items()}
    for i in moved:       # updated in place: not held to its old bits
        for j, (base, v, orig) in enumerate(a.bufs):
            if v is gargs[i]:
                a.bufs[j] = (base, v, None)
    if isinstance(ref, dict):
        gkw["out"] = {k: a.out(t) for k, t in ref.items()}
    elif isinstance(ref, tuple):
        gkw["out"] = tuple(a.out(t) for t in ref)
    else:
        gkw["out"] = a.out(ref)
    if need is not None:
        gkw["workspace"] = a.workspace(need)
    got = fn(*gargs, **gkw)
    a.check()
    _same(got, ref)
    for i in moved:
        _same(gargs[i], ref_args[i])


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name, dt):
    run, outs, eager, reset, moved = prepared(name, dt)
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
        reset()
        for t in outs:
            t.fill_(float("nan"))
        prepared(name, dt, seed=5)          # eager calls of the same operator
        torch.cuda.synchronize()
        g.replay()
        equal(outs + moved, eager)


@pytest.mark.parametrize("name", ["ssm_forward", "ssm_backward", "short_conv_backward",
                                  "gated_norm_backward", "residual_norm_backward"])
def test_two_graphs_share_a_workspace_in_turn(name):
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    one, two = (prepared(name, BF, seed, ws, T) for seed, T in ((0, 150), (1, 270)))
    graphs = []
    for run, *_ in (one, two):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1)):
        for t in one[1] + two[1]:
            t.fill_(float("nan"))
        ws.fill_(0xA5)                       # nothing is kept in it between calls
        for i in order:
            graphs[i].replay()
        equal(one[1], one[2])
        equal(two[1], two[2])


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once_on_two_streams(name):
    """Calls on streams other than the default one, on workspaces of their own,
    with nothing between them."""
    pair = [prepared(name, BF, seed) for seed in (0, 1)]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(3):
        for _, outs, _, reset, _ in pair:
            reset()
            for t in outs:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for (run, *_), s in zip(pair, streams):
            with torch.cuda.stream(s):
                run()
        for _, outs, eager, _, moved in pair:
            equal(outs + moved, eager)


def test_layer_captured_whole():
    """A layer's forward and backward in one graph."""
    import bench
    from workloads import layers as WL
    w = WL.BY_NAME["ssm-layer"].scaled(B=2, H=4, G=2, T=150, P=64, N=64, channels=96)
    a = WL.make_layer(w, DEV)
    fwd, o = bench.layer_forward(w, a)
    bwd, g = bench.layer_backward(w, a, o)

    def flat():
        return ([o["norm"], o["h"], o["y"], o["S"], o["out"]] + o["conv"]
                + tensors(g["gate"]) + tensors(g["scan"]) + tensors(g["norm"])
                + [t for c in g["conv"] for t in tensors(c)])
    fwd()
    bwd()
    torch.cuda.synchronize()
    eager = [t.clone() for t in flat()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd()
        bwd()
    for _ in range(3):
        for t in flat():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        equal(flat(), eager)


def test_refusals_of_tensors():
    """Shapes, types, strides and devices that a call cannot take raise before
    anything is launched."""
    z = lambda *s, d=F32: torch.zeros(s, dtype=d, device=DEV)
    x, w = z(2, 8, 64), z(64, 4)
    bad = [
        (ValueError, lambda: osdn.short_conv_forward(x, w, head_dim=48)),
        (ValueError, lambda: osdn.short_conv_forward(x, z(32, 4))),
        (ValueError, lambda: osdn.short_conv_forward(x, w.to(BF))),
        (ValueError, lambda: osdn.short_conv_forward(z(2, 64, 8).transpose(1, 2), w)),
        (ValueError, lambda: osdn.short_conv_forward(x, w, lengths=z(2))),
        (ValueError, lambda: osdn.short_conv_forward(x, w.cpu())),
        (ValueError, lambda: osdn.short_conv_decode(x, w, None)),
        (ValueError, lambda: osdn.short_conv_backward(x, w, z(2, 1, 8, 64, d=BF))),
        (ValueError, lambda: osdn.residual_norm_forward(x, z(64), z(2, 8, 64, d=BF))),
        (ValueError, lambda: osdn.residual_norm_forward(x, z(32))),
        (ValueError, lambda: osdn.gated_norm_forward(z(2, 3, 8, 64), z(2, 8, 64), z(64))),
        (ValueError, lambda: osdn.gated_norm_backward(z(2, 1, 8, 64), None, z(64),
                                                      z(2, 8, 64), out={})),
        (ValueError, lambda: osdn.ssm_forward(z(1, 3, 4, 64), z(1, 3, 4), z(3),
                                              z(1, 2, 4, 64), z(1, 2, 4, 64))),
        (ValueError, lambda: osdn.ssm_forward(z(1, 2, 4, 64), z(1, 2, 4, d=BF), z(2),
                                              z(1, 2, 4, 64), z(1, 2, 4, 64))),
        (ValueError, lambda: osdn.ssm_forward(z(1, 4, 2, 64).transpose(1, 2), z(1, 2, 4),
                                              z(2), z(1, 2, 4, 64), z(1, 2, 4, 64))),
        (osdn.OsdnError, lambda: osdn.ssm_forward(z(1, 2, 4, 48), z(1, 2, 4), z(2),
                                                  z(1, 2, 4, 64), z(1, 2, 4, 64))),
        (osdn.OsdnError, lambda: osdn.ssm_forward(
            z(1, 2, 4, 64), z(1, 2, 4), z(2), z(1, 2, 4, 64), z(1, 2, 4, 64),
            workspace=z(1, d=torch.uint8))),
        (osdn.OsdnError, lambda: osdn.residual_norm_forward(x, z(64), out=(x, None))),
    ]
    # rows that begin off a 16-byte boundary: taken in place where the call reads
    # rows, refused where it reads whole pieces
    off = z(1 * 2 * 4 * 64 + 1)[1:].view(1, 2, 4, 64)
    bad.append((osdn.OsdnError, lambda: osdn.ssm_forward(
        off, z(1, 2, 4), z(2), z(1, 2, 4, 64), z(1, 2, 4, 64))))
    for i, (err, call) in enumerate(bad):
        print("call", i, flush=True)
        with pytest.raises(err):
            call()
