"""Overlapping rows of a rotation are refused for every number of tokens and every stride."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest

import looped_transformer_decode_b200 as lla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rope(n, xs, ys, y, dtype=0):
    cfg = lla.Cfg(4, 2, 64, 16, 32)
    p = ctypes.c_void_p(0x10000)
    return lla.lib.lla_rope_apply(ctypes.byref(cfg.c()), p, 8, 0, 0, dtype, n, 2, p, p, xs,
                                  ctypes.c_void_p(y), ys, None, None)


def test_one_row_with_a_stride_of_zero():
    """In a process of its own: the refusal once divided by the stride."""
    code = ("import sys; sys.path.insert(0, 'tests'); import test_rope_overlap as t; "
            "print(t.rope(1, 0, 0, 0x10010))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.returncode
    assert int(r.stdout) == lla.ERR_INVALID


@pytest.mark.parametrize("n,xs,ys,y", [
    (1, 128, 128, 0x10010), (1, 0, 128, 0x10010), (1, 256, 256, 0x101f0), (1, 4096, 4096, 0xfe10),
    (1, 0, 0, 0xfff0), (2, 128, 128, 0x10200 - 16), (2, 256, 256, 0x10400 - 16)])
def test_overlapping_rows_are_refused(n, xs, ys, y):
    """Rows of 512 bytes at 0x10000: shifted by less than a row, whatever the stride says."""
    assert rope(n, xs, ys, y) == lla.ERR_INVALID
    assert "overlap" in lla.last_error()
