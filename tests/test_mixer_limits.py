"""Host-side limits of the operators' backward calls (no GPU): a call whose sum of
the parameters' gradients would need 2^32 threads is refused before its first
launch. The pointers are never followed."""
import os

import pytest

import delta_rule_recurrent_scan_amd as osdn

UNSUPPORTED, F32, BF16 = 3, 0, 1
P = [i << 44 for i in range(1, 14)]
BIG = 1 << 60

pytestmark = pytest.mark.skipif(not os.path.exists(osdn.library_path()),
                                reason="libosdn.so not built")


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [0, 1])
def test_convolution_columns(W, T):
    L = osdn.load_library()
    H = (1 << 27) // (W + 1) // 128 + 1        # (W + 1) 128 H >= 2^27 columns
    assert L.short_conv_backward(1, T, H, 128, W, BF16, BF16, P[0], 0, 0, P[1], P[2],
                                 P[3], None, 1, 0, 1e-6, P[4], None, P[5], P[6], P[7],
                                 P[8], P[9], BIG, None) == UNSUPPORTED


def test_weights_of_every_head():
    L = osdn.load_library()
    assert L.gated_norm_backward(1, 1 << 20, 1, 128, BF16, P[0], None, 0, 0, P[1], 1, 1e-6,
                                 0, P[2], P[3], None, P[4], P[5], BIG, None) == UNSUPPORTED


def test_heads_of_an_empty_batch():
    """The parameters' gradients are zeros then, of as many heads as there are."""
    L = osdn.load_library()
    for H in ((1 << 27) // 3 + 1, (1 << 31) - 1):
        assert L.ssm_backward(0, H, 1, 4, 64, 64, BF16, *[P[0]] * 7, 1, P[1], None, P[2],
                              P[3], P[4], P[5], P[6], P[7], P[8], P[9], P[10], P[11], P[12],
                              BIG, None) == UNSUPPORTED
