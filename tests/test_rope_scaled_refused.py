"""Decode over latents refuses tables of scaled frequencies: it turns the history by rope_base.

The Python call raises; the library's status has LLA_STATUS_ROPE_TABLE on every decode path.
"""
from __future__ import annotations

import pytest
import torch

import oracle as O
import looped_transformer_decode_b200 as lla

SCALED = [("linear", 2.0), ("ntk", 8.0), ("yarn", 4.0)]
PLAIN = [("none", 5.0), ("linear", 1.0), ("ntk", 1.0), ("yarn", 1.0)]
PATHS = [(O.Cfg(4, 2, 128, 96, 160), ""), (O.Cfg(4, 4, 128, 16, 32), ""),      # per head, phase operands
         (O.Cfg(4, 4, 128, 16, 32), "u"), (O.Cfg(2, 4, 64, 32, 48, O.MODE_2D), ""),
         (O.Cfg(4, 2, 128, 96, 160), "cuda_core")]


def test_python_call_refuses_a_marked_table():
    cfg = lla.Cfg(4, 2, 64, 16, 32)
    table = torch.zeros((8, 32, 2))
    table.scaled_frequencies = True
    x, one = torch.zeros((1, 2, 64)), torch.zeros((1, 4), dtype=torch.int32)
    for t in (table, table[:4]):
        with pytest.raises(ValueError, match="scaled frequencies"):
            lla.decode_attn(cfg, None, t, 0, one[0], x, x, x, one, one[0], None, None)
    part = table[:4]
    part.scaled_frequencies = False              # as after rope_table(out=part)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lla.decode_attn(cfg, x.byte(), part, 0, one[0], x, x, x, one, one[0], None, None,
                        ws=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(TypeError, match="rope must be|packed must be"):
        lla.decode_attn(cfg, None, None, 0, one[0], x, x, x, one, one[0], None, None,
                        ws=torch.zeros(8, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_rope", [(128, 0), (96, 0), (64, 32), (32, 0)])
def test_only_the_sign_of_a_zero_marks_a_table(d, d_rope):
    cfg = lla.Cfg(4, 2, d, 16, 32, d_rope=d_rope)
    plain = lla.rope_table(cfg, 300)
    for kind, factor in SCALED + PLAIN:
        got = lla.rope_table(cfg, 300, scaling=lla.RopeScaling(kind, factor, 64))
        scaled = (kind, factor) in SCALED
        assert bool(torch.signbit(got[0, 0, 1])) == got.scaled_frequencies == scaled
        assert torch.equal(got[0], plain[0]) and not torch.signbit(got[0, 1:, 1]).any()
        assert scaled or torch.equal(got, plain)
        # a buffer filled again with plain frequencies is a plain table
        lla.rope_table(cfg, 300, out=got)
        assert not got.scaled_frequencies and not torch.signbit(got[0, 0, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("cfg,path", PATHS)
def test_every_decode_path_tells(cfg, path, monkeypatch):
    from cases import decode_case
    from gpu_util import DeviceCase
    if path == "cuda_core":
        monkeypatch.setenv("LLA_DECODE_PATH", path)
    elif path:
        monkeypatch.setenv("LLA_TC_FORM", path)
    case = decode_case(cfg, 2, 300, seed=5, ctx_len=[300, 190])
    dev = DeviceCase(case)
    plain = dev.rope
    want = dev.decode(1)
    assert lla.decode_status(dev.ws) == 0
    for kind, factor in SCALED + PLAIN:
        table = lla.rope_table(dev.cfg, plain.shape[0], scaling=lla.RopeScaling(kind, factor, 64))
        scaled = (kind, factor) in SCALED
        if scaled:
            dev.rope = table
            with pytest.raises(ValueError, match="scaled frequencies"):
                dev.decode(1)
        dev.rope = table.clone()                    # as another caller of the library hands it over
        got = dev.decode(1)
        assert lla.decode_status(dev.ws) == (lla.STATUS_ROPE_TABLE if scaled else 0)
        assert scaled or (got == want).all()
    dev.rope = plain
    assert (dev.decode(1) == want).all() and lla.decode_status(dev.ws) == 0
