"""The launches that a feed-forward product is cut into, asked of the library's own
planner (not a test module): sizes in a test name the path they are there for, and a
planner that takes another one fails the test in place of leaving the path out."""
import ctypes

import delta_rule_recurrent_scan_amd as osdn

LARGE, MIDDLE, SMALL = 0, 1, 2
ONE, TWO, FORWARDS = 0, 1, 2
LAUNCH = 4.5                       # microseconds between two launches


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("shape", "tm", "tn", "nt", "whole", "splits",
                                            "per", "area")] + [("parts_at", ctypes.c_longlong)]

    @property
    def rest(self):
        return self.tm * self.tn - self.whole


_L, _I, _D, _P = ctypes.c_longlong, ctypes.c_int, ctypes.c_double, ctypes.POINTER


def _plan(kind, M, N, K, bf16):
    f = osdn.load_library()._ZN4osdn3ffn9make_planERNS0_4PlanENS0_4KindExxxiPd
    f.argtypes, f.restype = [_P(Plan), _I, _L, _L, _L, _I, _P(_D)], ctypes.c_bool
    p, us = Plan(), _D()
    assert f(ctypes.byref(p), kind, M, N, K, int(bf16), ctypes.byref(us))
    return p, us.value


def tile_of_k(bf16):
    return 64 if bf16 else 32


def forward(R, C, F, bf16):
    """The plan of a forward of more rows than the kernel for few takes."""
    return _plan(FORWARDS, R, 2 * F, (C + 7) // 8 * 8, bf16)[0]


def backward(R, C, F, bf16):
    """(dx's plan, the weights' gradients' plan, whether they share a launch)."""
    kt = tile_of_k(bf16)
    x, w = (R, C, 2 * -(-F // kt) * kt), (F, C, R)
    p, tx = _plan(ONE, *x, bf16)
    q, tw = _plan(TWO, *w, bf16)
    f = osdn.load_library()._ZN4osdn3ffn9make_pairERNS0_4PlanES2_RA3_KxS5_id
    f.argtypes = [_P(Plan), _P(Plan), _P(_L), _P(_L), _I, _D]
    f.restype = ctypes.c_bool
    pair = f(ctypes.byref(p), ctypes.byref(q), (_L * 3)(*x), (_L * 3)(*w), int(bf16),
             tx + tw + LAUNCH)
    return p, q, pair
