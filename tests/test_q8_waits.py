"""The waits of the 8-bit and full-memory decode attention end alike for all lanes of a warp.

After a wait the warp runs full-mask shuffles and votes.  A lane's own result depends on when it
read the barrier, the abort flag and the timer, so a branch on it may part the warp near a timeout.
That cannot be brought about on purpose; the source is checked instead.
"""
from __future__ import annotations

import os
import re

import looped_transformer_decode_b200 as lla

CSRC = os.path.join(os.path.dirname(lla.__file__), "csrc")


def agreed(name, wait):
    """How many of the waits matching ``wait`` the file has; each is inside a vote."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = [m.start() for m in re.finditer(wait, text)]
    for at in found:
        assert re.search(r"__all_sync\(0xffffffffu,\s*(sm100::)?$", text[:at]), text[at - 60:at + 60]
    return len(found)


def test_every_wait_is_agreed_on_by_the_warp():
    assert agreed("lla_q8_decode.cu", r"\bmbar_wait\w*\(") >= 1


def test_full_memory_consumers_agree():
    """Its consumers wait for `full` barriers as whole warps; one producer thread waits for `empty`."""
    assert agreed("lla_full.cu", r"\bmbar_wait\(&full\[") >= 1
