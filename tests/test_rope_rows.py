"""Rotary positions as operators: scaled tables, and the rotation of rows of heads with its
gradient.

CPU: the oracle's frequencies against their closed forms, the refusals.  GPU: tables and
rotated rows against the oracle.  Tolerances count roundings: half a step of the result's
type, and three fp32 roundings of each product of a pair.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as P

import looped_transformer_decode_b200 as lla

SCALINGS = [("none", 1.0, 1), ("linear", 4.0, 1), ("ntk", 8.0, 1), ("yarn", 32.0, 4096),
            ("yarn", 1.5, 300), ("ntk", 1.0, 1)]


def cfg_of(d, d_rope=0, base=10000.0, H=2):
    return lla.Cfg(4, H, d, 16, 32, rope_base=base, d_rope=d_rope)


# ----------------------------------------------------------------------------- oracle

def test_scaled_frequencies_closed_forms():
    plain = P.rope_angles(64, 10000.0)
    assert np.allclose(plain, 10000.0 ** (-np.arange(32) / 32))
    assert np.allclose(P.rope_angles(64, 10000.0, "linear", 4.0), plain / 4)
    # the last pair of NTK turns exactly factor times slower, the first one not at all
    ntk = P.rope_angles(64, 10000.0, "ntk", 8.0)
    assert np.isclose(ntk[0], 1.0) and np.isclose(ntk[-1], plain[-1] / 8)
    yarn = P.rope_angles(64, 10000.0, "yarn", 16.0, 4096)
    turns = 4096 * plain / (2 * np.pi)
    assert np.array_equal(yarn[turns > 60], plain[turns > 60])
    assert np.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 16)
    assert (np.diff(plain / yarn) >= -1e-12).all()


def test_rotation_back_is_the_transpose():
    g = np.random.default_rng(0)
    x, dy = g.standard_normal((2, 3, 2, 64))
    ang = g.uniform(0, 100, (3, 16))
    for layout in ("half", "interleaved"):
        y = P.rope_rows(x, np.cos(ang), np.sin(ang), layout)
        dx = P.rope_rows(dy, np.cos(ang), np.sin(ang), layout, inverse=True)
        assert np.isclose((y * dy).sum(), (x * dx).sum())
        assert np.allclose(P.rope_rows(y, np.cos(ang), np.sin(ang), layout, True), x)


# ----------------------------------------------------------------------------- refusals

def test_rope_apply_refusals():
    f, p = lla.lib.lla_rope_apply, ctypes.c_void_p(0x10000)

    def call(cfg=cfg_of(64), rope=p, mp=8, layout=0, dtype=0, n=4, heads=2, pos=p, x=p, xs=128,
             y=ctypes.c_void_p(0x20000), ys=128, status=None):
        return f(ctypes.byref(cfg.c()), rope, mp, layout, 0, dtype, n, heads, pos, x, xs, y, ys,
                 status, None)

    bad, no = lla.ERR_INVALID, lla.ERR_UNSUPPORTED
    assert call(n=0) == lla.OK
    for kw, code in ((dict(rope=None), bad), (dict(pos=None), bad), (dict(x=None), bad),
                     (dict(y=None), bad), (dict(mp=0), bad), (dict(layout=2), bad),
                     (dict(layout=-1), bad), (dict(dtype=2), no), (dict(heads=0), no),
                     (dict(heads=4097), no), (dict(n=-1), bad), (dict(n=1 << 60), no),
                     (dict(xs=127), bad), (dict(xs=124), bad), (dict(xs=130), bad),
                     (dict(xs=1 << 62), bad), (dict(dtype=1, ys=132), bad), (dict(xs=-128), bad),
                     (dict(x=ctypes.c_void_p(0x10008)), bad), (dict(status=ctypes.c_void_p(2)), bad),
                     (dict(pos=ctypes.c_void_p(0x10002)), bad), (dict(cfg=cfg_of(80)), no),
                     # overlapping rows: shifted by less than a row, or different strides
                     (dict(y=ctypes.c_void_p(0x10010)), bad),
                     (dict(y=p, ys=256), bad),
                     (dict(xs=256, ys=256, y=ctypes.c_void_p(0x10000 + 256)), bad)):
        assert call(**kw) == code, kw
        assert lla.last_error()


def test_rope_table_scaled_refusals():
    f, p = lla.lib.lla_rope_table_scaled, ctypes.c_void_p(0x10000)

    def call(kind="yarn", factor=2.0, orig=4096, fast=0.0, slow=0.0, mp=8, table=p, nbytes=None,
             cfg=cfg_of(64), raw_kind=None):
        s = lla.RopeScaling(kind, factor, orig, fast, slow).c()
        if raw_kind is not None:
            s.kind = raw_kind
        return f(ctypes.byref(cfg.c()), ctypes.byref(s), mp, table,
                 mp * 32 * 8 if nbytes is None else nbytes, None)

    bad = lla.ERR_INVALID
    for kw in (dict(factor=0.5), dict(factor=float("nan")), dict(factor=float("inf")),
               dict(orig=0), dict(fast=1.0, slow=1.0), dict(slow=-1.0), dict(mp=0),
               dict(fast=float("nan")), dict(table=None), dict(raw_kind=4), dict(raw_kind=-1)):
        assert call(**kw) == bad, kw
    assert call(nbytes=8 * 32 * 8 - 1) == lla.ERR_TOO_SMALL
    assert f(ctypes.byref(cfg_of(64).c()), None, 8, p, 1 << 20, None) == bad
    with pytest.raises(ValueError):
        lla.RopeScaling("dynamic").c()


# ----------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("kind,factor,orig", SCALINGS)
@pytest.mark.parametrize("d,d_rope,base", [(128, 0, 10000.0), (96, 0, 500000.0), (64, 32, 10000.0)])
def test_scaled_table_matches_oracle(kind, factor, orig, d, d_rope, base):
    n = 5003
    got = lla.rope_table(cfg_of(d, d_rope, base), n, scaling=lla.RopeScaling(kind, factor, orig))
    ang = np.arange(n)[:, None] * P.rope_angles(d_rope or d, base, kind, factor, orig)
    want = np.stack([np.cos(ang), np.sin(ang)], -1)
    # one rounding to fp32 of values up to 1, and fp64 angles up to 5003 rad
    assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -25 + 5003 * 2.0 ** -50
    if kind == "none":
        assert torch.equal(got, lla.rope_table(cfg_of(d, d_rope, base), n))


def pair_bound(x, table, pos, layout, y, dtype):
    """Half a step of the result, and three fp32 roundings of the pair's products."""
    rd = 2 * table.shape[1]
    big = np.zeros_like(y)
    a = np.abs(x[..., :rd])
    big[..., :rd] = a + (np.roll(a, rd // 2, -1) if layout == "half"
                         else a.reshape(*a.shape[:-1], -1, 2)[..., ::-1].reshape(a.shape))
    return torch.finfo(dtype).eps / 2 * np.abs(y) + 3 * 2.0 ** -24 * big


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,d_rope,H,n", [(32, 0, 1, 1), (64, 32, 3, 17), (96, 0, 8, 130),
                                          (96, 64, 5, 33), (128, 0, 16, 257), (128, 64, 2, 1000),
                                          (128, 32, 1, 4)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotated_rows_match_oracle(dtype, layout, d, d_rope, H, n, inverse):
    g = torch.Generator().manual_seed(n + d)
    table = lla.rope_table(cfg_of(d, d_rope, H=H), 700)
    pos = torch.randint(0, 700, (n,), generator=g).int().cuda()
    x = torch.randn((n, H, d), generator=g).to(dtype).cuda()
    got = lla.rope_apply(cfg_of(d, d_rope, H=H), table, pos, x, layout=layout, inverse=inverse)
    t = table.double().cpu().numpy()[pos.cpu().numpy()]
    xs = x.double().cpu().numpy()
    want = P.rope_rows(xs, t[..., 0], t[..., 1], layout, inverse)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= pair_bound(xs, t, pos, layout, want, dtype)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 15, 17, 129])
def test_scaled_table_of_few_positions(n):
    got = lla.rope_table(cfg_of(96), n, scaling=lla.RopeScaling("linear", 3.0))
    ang = np.arange(n)[:, None] * P.rope_angles(96, 10000.0, "linear", 3.0)
    want = np.stack([np.cos(ang), np.sin(ang)], -1)
    assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -25 + n * 2.0 ** -50


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,layout,d,d_rope,H,n", [
    (torch.bfloat16, "half", 96, 0, 7, 12001), (torch.float32, "interleaved", 128, 64, 5, 5003),
    (torch.bfloat16, "interleaved", 32, 0, 1, 300001), (torch.float32, "half", 64, 32, 130, 301)])
def test_many_rows_match_oracle(dtype, layout, d, d_rope, H, n):
    """Calls large enough for a thread to take several heads, whose number is no multiple."""
    cfg = cfg_of(d, d_rope, H=min(H, 128))
    g = torch.Generator(device="cuda").manual_seed(n)
    table = lla.rope_table(cfg, 900)
    pos = torch.randint(0, 900, (n,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((n, H, d), generator=g, device="cuda").to(dtype)
    got = lla.rope_apply(cfg, table, pos, x, layout=layout)
    pick = torch.randint(0, n, (400,), generator=g, device="cuda")
    pick[0], pick[1] = 0, n - 1
    t = table.double()[pos[pick].long()].cpu().numpy()
    xs = x[pick].double().cpu().numpy()
    want = P.rope_rows(xs, t[..., 0], t[..., 1], layout, False)
    err = np.abs(got[pick].double().cpu().numpy() - want)
    assert (err <= pair_bound(xs, t, None, layout, want, dtype)).all()
    # every row against the same rows in calls of a few, which a thread a head takes
    few = torch.cat([lla.rope_apply(cfg, table, pos[i:i + 97], x[i:i + 97], layout=layout)
                     for i in range(0, min(n, 970), 97)])
    assert torch.equal(got[:few.shape[0]], few)
    lla.rope_apply(cfg, table, pos, x, layout=layout, out=x)
    assert torch.equal(x, got)


@pytest.mark.gpu
def test_strided_and_in_place_rows():
    """Slices of a fused projection, rows alternating in one buffer, and y = x."""
    cfg, n, H, d = cfg_of(64, H=4), 37, 4, 64
    table = lla.rope_table(cfg, 100)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    wide = torch.randn((n, 3, H, d), device="cuda")
    want = lla.rope_apply(cfg, table, pos, wide[:, 1].contiguous())
    before = wide.clone()
    assert torch.equal(lla.rope_apply(cfg, table, pos, wide[:, 1]), want)
    lla.rope_apply(cfg, table, pos, wide[:, 1], out=wide[:, 2])       # alternate rows
    assert torch.equal(wide[:, 2], want) and torch.equal(wide[:, :2], before[:, :2])
    lla.rope_apply(cfg, table, pos, wide[:, 1], out=wide[:, 1])       # in place
    assert torch.equal(wide[:, 1], want) and torch.equal(wide[:, 0], before[:, 0])
    lla.rope_apply(cfg, table, pos, wide[:, 1], inverse=True, out=wide[:, 1])
    assert (wide[:, 1] - before[:, 1]).abs().max() < 1e-5
    with pytest.raises(lla.LLAError):
        flat = torch.zeros((n + 1) * H * d, device="cuda")
        lla.rope_apply(cfg, table, pos, flat[:-H * d].view(n, H, d), out=flat[H * d:].view(n, H, d))


@pytest.mark.gpu
def test_gradient_against_differences():
    """dL/dx by the inverse rotation against central differences of L = sum(w y)."""
    cfg, n, H, d = cfg_of(96, 32, H=2), 3, 2, 96
    table = lla.rope_table(cfg, 50)
    pos = torch.tensor([0, 7, 49], dtype=torch.int32, device="cuda")
    x = torch.randn((n, H, d), device="cuda")
    w = torch.randn_like(x)
    for layout in ("half", "interleaved"):
        dx = lla.rope_apply(cfg, table, pos, w, layout=layout, inverse=True).double()
        v = torch.randn_like(x)
        eps = 0.5                                        # the map is linear: any step serves
        up = lla.rope_apply(cfg, table, pos, x + eps * v, layout=layout).double()
        dn = lla.rope_apply(cfg, table, pos, x - eps * v, layout=layout).double()
        diff = float((w.double() * (up - dn)).sum()) / (2 * eps)
        want = float((dx * v.double()).sum())
        # 576 terms of a few units, each side rounded in fp32 a few times
        assert abs(diff - want) <= 576 * 10 * 4 * 2.0 ** -24


@pytest.mark.gpu
def test_positions_out_of_range_are_clamped_and_told():
    cfg = cfg_of(64, H=1)
    table = lla.rope_table(cfg, 10)
    x = torch.randn((4, 1, 64), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lla.rope_apply(cfg, table, torch.tensor([-1, 0, 9, 10], dtype=torch.int32, device="cuda"),
                         x, status=status)
    same = lla.rope_apply(cfg, table, torch.tensor([0, 0, 9, 9], dtype=torch.int32, device="cuda"), x)
    assert torch.equal(got, same)
    assert int(status) == lla.STATUS_POSITION_RANGE
