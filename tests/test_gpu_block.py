"""The operators of a hybrid stack's block in a row, as a model runs them, forward and
backward, against the fp64 oracle of the whole row:

    y1, h1 = residual norm;  projections;
    recurrent mixer: short convolution -> gated linear recurrence, or
    delta rule: queries and keys normed and rotated -> OSDN;
    projection back;  y2, h2 = residual norm;  gated feed-forward;  projection back.

The projections are plain products of the caller. In fp32, so that every operator is
fed what the oracle's is up to 32-bit rounding: relative errors of the results and
gradients under 1e-4 (the operators' own are 1e-6 and less, the delta rule's 1e-5; a
chain of eight that each add theirs to what they pass on, twice for the way back)."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import DEV, F32, f64
from oracle import backward as OB, layer as Y, mixer as M, recurrence as R

pytestmark = pytest.mark.gpu
B, T, C, F, H, D = 2, 70, 64, 96, 2, 32
TOL = 1e-4


def rel(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


def weights(kind):
    g = torch.Generator().manual_seed(3)
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(DEV)
    c = C ** -0.5
    w = dict(x=n(B, T, C), res=n(B, T, C), n1=1 + n(C, scale=0.1), n2=1 + n(C, scale=0.1),
             proj=n(3 * C, C, scale=c), back=n(C, C, scale=c), wg=n(F, C, scale=c),
             wu=n(F, C, scale=c), down=n(C, F, scale=F ** -0.5), dy=n(B, T, C),
             lengths=torch.tensor([T, T - 21], dtype=torch.int32, device=DEV))
    if kind == "recurrence":
        w.update(conv=n(C, 4, scale=0.5), A=-torch.exp(n(C)))
    else:
        w.update(qw=1 + n(D, scale=0.1), kw=1 + n(D, scale=0.1),
                 f=(100.0 ** -(torch.arange(D // 2) / (D // 2))).float().to(DEV),
                 beta=torch.sigmoid(n(B, H, T)))
    return w


def mixer_forward(w, p, kind):
    """From the projection's rows [B,T,3C] to token rows, and what the backward keeps."""
    if kind == "recurrence":
        x, r, i = p[:, :, :C], p[:, :, C:2 * C], p[:, :, 2 * C:]
        cx, _ = osdn.short_conv_forward(x, w["conv"], lengths=w["lengths"])
        cx = cx[:, 0]
        y, _, states = osdn.glr_forward(cx, r, w["A"], i=i, lengths=w["lengths"],
                                        save=True)
        return y, (x, cx, r, i, states)
    q, k = osdn.qk_rotary_forward(p[:, :, :C], p[:, :, C:2 * C], D, inv_freq=w["f"],
                                  q_weight=w["qw"], k_weight=w["kw"], norm="l2")
    v = p[:, :, 2 * C:].reshape(B, T, H, D).transpose(1, 2).contiguous()
    o = osdn.osdn_forward(q, k, v, w["beta"], None, 0.1)[0]
    return o.transpose(1, 2).reshape(B, T, C), (q, k, v)


def mixer_backward(w, p, kept, dy, kind):
    if kind == "recurrence":
        x, cx, r, i, states = kept
        d = osdn.glr_backward(cx, r, w["A"], dy, i=i, lengths=w["lengths"], states=states)
        dc = osdn.short_conv_backward(x, w["conv"], d["x"][:, None].contiguous(),
                                      lengths=w["lengths"])
        return (torch.cat([dc["x"], d["r"], d["i"]], -1),
                dict(A=d["A"], conv=dc["weight"]))
    q, k, v = kept
    do = dy.reshape(B, T, H, D).transpose(1, 2).contiguous()
    d = osdn.osdn_backward(q, k, v, w["beta"], do, eta=0.1)
    e = osdn.qk_rotary_backward(p[:, :, :C], p[:, :, C:2 * C], d["q"], d["k"], D,
                                inv_freq=w["f"], q_weight=w["qw"], k_weight=w["kw"],
                                norm="l2")
    dv = d["v"].transpose(1, 2).reshape(B, T, C)
    return (torch.cat([e["q"], e["k"], dv], -1),
            dict(qw=e["q_weight"], kw=e["k_weight"], beta=d["beta"]))


def block(w, kind):
    y1, h1 = osdn.residual_norm_forward(w["x"], w["n1"], w["res"])
    p = y1 @ w["proj"].t()
    y, kept = mixer_forward(w, p, kind)
    m = y @ w["back"].t()
    y2, h2 = osdn.residual_norm_forward(m, w["n2"], h1)
    h, gate, up = osdn.gated_ffn_forward(y2, w["wg"], w["wu"], save=True)
    out = h @ w["down"].t()
    dh = w["dy"] @ w["down"]
    g = osdn.gated_ffn_backward(y2, w["wg"], w["wu"], gate, up, dh)
    n2 = osdn.residual_norm_backward(g["x"], h2, w["n2"])
    dm, dh1 = n2["x"], n2["residual"]
    dp, dmix = mixer_backward(w, p, kept, (dm @ w["back"]).contiguous(), kind)
    n1 = osdn.residual_norm_backward((dp @ w["proj"]).contiguous(), h1, w["n1"], dh=dh1)
    return dict(out=out, h2=h2, w_gate=g["w_gate"], w_up=g["w_up"], n2=n2["weight"],
                n1=n1["weight"], res=n1["residual"], x=n1["x"], **dmix)


def oracle_mixer(w, p, kind, lens):
    if kind == "recurrence":
        cx = M.short_conv_ref(p[:, :, :C], w["conv"], lengths=lens)[0][:, 0]
        return Y.glr_ref(cx, p[:, :, C:2 * C], w["A"], p[:, :, 2 * C:], None, lens)[0], cx
    q = Y.qk_rotary_ref(p[:, :, :C], D, w["f"], w["qw"], norm="l2")[0]
    k = Y.qk_rotary_ref(p[:, :, C:2 * C], D, w["f"], w["kw"], norm="l2")[0]
    v = p[:, :, 2 * C:].reshape(B, T, H, D).transpose(0, 2, 1, 3)
    o = R.osdn_ref(q, k, v, w["beta"], None, 0.1)[0]
    return o.transpose(0, 2, 1, 3).reshape(B, T, C), (q, k, v)


def oracle_mixer_backward(w, p, kept, dy, kind, lens):
    if kind == "recurrence":
        d, _ = Y.glr_backward_ref(kept, p[:, :, C:2 * C], w["A"], dy, p[:, :, 2 * C:], None,
                                  None, lens)
        dc = M.short_conv_backward_ref(p[:, :, :C], w["conv"], d["x"][:, None], lengths=lens)
        return (np.concatenate([dc["x"], d["r"], d["i"]], -1),
                dict(A=d["A"], conv=dc["weight"]))
    q, k, v = kept
    do = dy.reshape(B, T, H, D).transpose(0, 2, 1, 3)
    d = OB.osdn_backward_ref(q, k, v, w["beta"], None, 0.1, None, None, do)
    eq, _ = Y.qk_rotary_backward_ref(p[:, :, :C], d["q"], D, w["f"], w["qw"], norm="l2")
    ek, _ = Y.qk_rotary_backward_ref(p[:, :, C:2 * C], d["k"], D, w["f"], w["kw"], norm="l2")
    dv = d["v"].transpose(0, 2, 1, 3).reshape(B, T, C)
    return (np.concatenate([eq["x"], ek["x"], dv], -1),
            dict(qw=eq["weight"], kw=ek["weight"], beta=d["beta"]))


def oracle_block(w, kind):
    lens = w["lengths"].tolist()
    w = {n: f64(t) for n, t in w.items()}
    y1, h1 = M.residual_norm_ref(w["x"].reshape(-1, C), w["n1"], w["res"].reshape(-1, C))
    p = (y1 @ w["proj"].T).reshape(B, T, 3 * C)
    y, kept = oracle_mixer(w, p, kind, lens)
    m = y.reshape(-1, C) @ w["back"].T
    y2, h2 = M.residual_norm_ref(m, w["n2"], h1)
    h, gate, up = Y.gated_ffn_ref(y2, w["wg"], w["wu"])
    dh = w["dy"].reshape(-1, C) @ w["down"]
    g, _, _ = Y.gated_ffn_backward_ref(y2, w["wg"], w["wu"], gate, up, dh)
    n2 = M.residual_norm_backward_ref(g["x"], h2, w["n2"])
    dp, dmix = oracle_mixer_backward(w, p, kept, (n2["x"] @ w["back"]).reshape(B, T, C), kind,
                                     lens)
    n1 = M.residual_norm_backward_ref(dp.reshape(-1, 3 * C) @ w["proj"], h1, w["n1"],
                                      dh=n2["residual"])
    shape = lambda t: t.reshape(B, T, C)
    return dict(out=shape(h @ w["down"].T), h2=shape(h2), w_gate=g["w_gate"],
                w_up=g["w_up"], n2=n2["weight"], n1=n1["weight"],
                res=shape(n1["residual"]), x=shape(n1["x"]), **dmix)


@pytest.mark.parametrize("kind", ["recurrence", "delta"])
def test_block(kind):
    w = weights(kind)
    got = block(w, kind)
    torch.cuda.synchronize()
    want = oracle_block(w, kind)
    assert set(got) == set(want)
    for n in got:
        e = rel(got[n], want[n])
        print("%s: %.2e" % (n, e), flush=True)
        assert e <= TOL, n


@pytest.mark.parametrize("kind", ["recurrence", "delta"])
def test_block_in_a_graph(kind):
    """The whole step captured, while an eager result of the same weights lives:
    every replay gives the eager bits."""
    w = weights(kind)
    eager = block(w, kind)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(w, kind)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block(w, kind)
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        again = block(w, kind)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], eager[n]) and torch.equal(again[n], eager[n]), n


def test_tokens_after_a_prompt():
    """The recurrence block's mixer a token at a time, after a prompt: convolution and
    recurrence carry their states in place."""
    w = weights("recurrence")
    g = torch.Generator().manual_seed(4)
    p = torch.randn((B, T, 3 * C), generator=g).to(DEV)
    x, r, i = p[:, :, :C], p[:, :, C:2 * C], p[:, :, 2 * C:]
    cx, _ = osdn.short_conv_forward(x, w["conv"])
    y, h_T, _ = osdn.glr_forward(cx[:, 0], r, w["A"], i=i)
    n = T - 5
    cut = lambda t, a, b: t[:, a:b]
    c0, cs = osdn.short_conv_forward(cut(x, 0, n), w["conv"])
    _, h, _ = osdn.glr_forward(c0[:, 0], cut(r, 0, n), w["A"], i=cut(i, 0, n))
    for t in range(n, T):
        ct = osdn.short_conv_decode(cut(x, t, t + 1), w["conv"], cs)
        yt = osdn.glr_decode(ct[:, 0], cut(r, t, t + 1), w["A"], h, i=cut(i, t, t + 1))
        assert rel(yt, f64(cut(y, t, t + 1))) <= 1e-5
    assert rel(h, f64(h_T)) <= 1e-5


def test_kernel_times_of_both_blocks():
    """Every kernel of the two blocks is reported, more than 16 of them."""
    osdn.kernel_timing(True)
    try:
        for kind in ("recurrence", "delta"):
            block(weights(kind), kind)
        seen = osdn.kernel_times()
    finally:
        osdn.kernel_timing(False)
    print(sorted(seen))
    assert len(seen) > 16
    assert {"glr", "glr_bwd", "qk_rotary", "qk_rotary_bwd", "ffn_grad", "residual_norm",
            "short_conv_bwd"} <= set(seen)
