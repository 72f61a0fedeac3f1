"""The layer workloads' draws and the bytes that their roofline divides by."""
import torch

import bench
from workloads import layers as WL


def test_draws_are_seeded_and_shaped():
    w = WL.BY_NAME["ssm-layer"].scaled(B=2, H=4, G=2, T=9, P=32, N=64, channels=40)
    a, b = WL.make_layer(w), WL.make_layer(w)
    assert w.splits == (128, 128, 128, 128)
    assert a["proj"].shape == (2, 9, 512) and a["proj"].dtype == torch.bfloat16
    assert a["residual"].dtype == torch.float32 and a["block"].shape == (2, 9, 40)
    assert [t.shape for t in a["conv_w"]] == [(128, 4)] * 3
    assert torch.all(a["A"] <= -1) and torch.all(a["A"] >= -16)
    assert torch.equal(a["proj"], b["proj"]) and torch.equal(a["dy"], b["dy"])
    d = WL.make_layer(WL.BY_NAME["ssm-layer-decode"].scaled(B=2, channels=8))
    assert d["S"].shape == (2, 16, 128, 128) and d["S"].dtype == torch.float32
    assert [t.shape for t in d["conv_state"]] == [(2, 3, 2048), (2, 3, 256), (2, 3, 256)]


def test_layer_bytes_at_the_layer_shape():
    w = WL.BY_NAME["ssm-layer"]
    rows = 4 * 4096
    norm = 2048 * (2 + 4 + 4 + 2)          # block, residual, h, y
    conv = 2 * (2048 + 2 * 256) * 2        # read and written
    scan = (2 * 2048 + 2 * 256) * 2 + 16 * 4
    gate = 3 * 2048 * 2                    # y, z, out
    assert bench.layer_bytes(w) == (rows * (norm + conv + scan + gate)
                                    + 4 * 16 * 128 * 128 * 4)
    back = (norm                           # dy, h, d residual, d block
            + 3 * (2048 + 2 * 256) * 2     # x, dy, dx
            + 5 * 2048 * 2                 # y, z, d out; dy, dz
            + (3 * 2048 + 4 * 256) * 2 + 2 * 16 * 4)
    assert bench.layer_bytes(w, True) == rows * back
    d = WL.BY_NAME["ssm-layer-decode"]
    assert bench.layer_bytes(d) == (128 * (norm + conv + scan + gate)
                                    + 2 * 128 * 16 * 128 * 128 * 4
                                    + 2 * 128 * 3 * (2048 + 512) * 2)
