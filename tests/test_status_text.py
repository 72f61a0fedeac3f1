"""Texts of the status codes: the older entry points' arguments are named (no GPU)."""
import os

import pytest

import delta_rule_recurrent_scan_amd as osdn


@pytest.mark.skipif(not os.path.exists(osdn.library_path()), reason="libosdn.so not built")
@pytest.mark.parametrize("code,words", [
    (0, "ok"), (1, "a required pointer argument is NULL"),
    (2, "bad dimensions: B, H and T must be >= 0"),
    (3, "unsupported combination of Dk, Dv, chunk and dtype"),
    (4, "workspace missing or too small"),
    (5, "an output overlaps an input or another output"),
    (6, "the HIP runtime rejected a kernel launch"),
    (7, "not 16-byte aligned"), (99, "unknown status")])
def test_text(code, words):
    assert words in osdn.load_library().osdn_strerror(code).decode()
