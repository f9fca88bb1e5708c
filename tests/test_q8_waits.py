"""The waits of the 8-bit decode attention end alike for all lanes of a warp.

After a wait the warp runs full-mask shuffles and votes.  A lane's own result depends on when it
read the barrier, the abort flag and the timer, so a branch on it may part the warp near a timeout.
That cannot be brought about on purpose; the source is checked instead.
"""
from __future__ import annotations

import os
import re

import looped_transformer_decode_b200 as lla

CSRC = os.path.join(os.path.dirname(lla.__file__), "csrc")


def test_every_wait_is_agreed_on_by_the_warp():
    with open(os.path.join(CSRC, "lla_q8_decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    waits = [m.start() for m in re.finditer(r"\bmbar_wait\w*\(", text)]
    assert waits
    for at in waits:
        assert re.search(r"__all_sync\(0xffffffffu,\s*sm100::$", text[:at]), text[at - 60:at + 60]
