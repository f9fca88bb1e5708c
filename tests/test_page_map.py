"""Block tables and slot maps on the GPU against a sequence-by-sequence reference: every
output is a whole number and has to be equal."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as P

import looped_transformer_decode_b200 as lla


def state(g, lens, page, max_pages, n_pages):
    """Sequences holding shuffled pages, -1 behind them, the rest of the pool free."""
    perm = g.permutation(n_pages)
    bt = np.full((len(lens), max_pages), -1, np.int64)
    at = 0
    for b, n in enumerate(lens):
        m = -(-int(n) // page)
        bt[b, :m] = perm[at:at + m]
        at += m
    assert at <= n_pages
    fl = np.full(n_pages, -7, np.int64)             # entries past n_free are never read
    fl[:n_pages - at] = perm[at:]
    return dict(ctx_len=np.array(lens, np.int64), block_table=bt, free_list=fl, n_free=n_pages - at)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


class Device:
    def __init__(self, s):
        self.ctx, self.bt = dev(s["ctx_len"]), dev(s["block_table"])
        self.fl, self.nf = dev(s["free_list"]), dev([s["n_free"]])

    def call(self, page, n_new, cap):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        t, slot, pos = lla.page_map(page, self.ctx, dev(n_new), self.bt, self.fl, self.nf, cap,
                                    status=st)
        return dict(tok_start=t, slot=slot, positions=pos, ctx_len=self.ctx, block_table=self.bt,
                    free_list=self.fl, n_free=self.nf, status=st)


def same(got, want):
    for k, w in want.items():
        g = got[k].cpu().numpy().astype(np.int64)
        np.testing.assert_array_equal(g, np.asarray(w, np.int64).reshape(g.shape), err_msg=k)


def step(s, d, page, n_new, cap):
    want = P.page_map(page, s["ctx_len"], n_new, s["block_table"], s["free_list"], s["n_free"], cap)
    same(d.call(page, n_new, cap), want)
    return {k: want[k] for k in s}, want["status"]


# ----------------------------------------------------------------------------- reference, refusals

def test_reference_rollback_restores():
    g = np.random.default_rng(1)
    s = state(g, [5, 0, 33, 16], 16, 8, 20)
    a = P.page_map(16, s["ctx_len"], [20, 1, 0, 1], s["block_table"], s["free_list"], s["n_free"], 64)
    back = a["tok_start"][:-1] - a["tok_start"][1:]
    b = P.page_map(16, a["ctx_len"], back, a["block_table"], a["free_list"], a["n_free"], 0)
    for k in s:
        np.testing.assert_array_equal(b[k], s[k])
    assert a["status"] == b["status"] == 0 and a["tok_start"][-1] == 22


def test_refusals():
    f, p, q = lla.lib.lla_page_map, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)

    def call(B=2, page=16, mp=4, n=8, ctx=p, new=p, bt=p, fl=p, nf=p, cap=4, ts=p, slot=p, pos=p,
             st=None):
        return f(B, page, mp, n, ctx, new, bt, fl, nf, cap, ts, slot, pos, st, None)

    bad, no = lla.ERR_INVALID, lla.ERR_UNSUPPORTED
    for kw, code in ((dict(B=-1), bad), (dict(mp=-1), bad), (dict(n=-1), bad), (dict(cap=-1), bad),
                     (dict(page=8), no), (dict(page=48), no), (dict(page=256), no),
                     (dict(B=65536), no), (dict(mp=1 << 27), no), (dict(cap=1 << 31), no),
                     (dict(ctx=None), bad), (dict(new=None), bad), (dict(bt=None), bad),
                     (dict(fl=None), bad), (dict(nf=None), bad), (dict(ts=None), bad),
                     (dict(slot=None), bad), (dict(pos=None), bad), (dict(slot=q), bad),
                     (dict(ctx=ctypes.c_void_p(0x10001)), bad),
                     (dict(st=ctypes.c_void_p(0x10002)), bad)):
        assert call(**kw) == code, kw


# ----------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_steps_match_reference(page):
    g = np.random.default_rng(page)
    lens = list(g.integers(0, 300, 61)) + [0, page - 1, page, page + 1]
    s = state(g, lens, page, 400 // page + 2, 65 * (400 // page + 2))
    d = Device(s)
    for _ in range(2 * 16 + 3):
        s, status = step(s, d, page, np.ones(len(lens)), len(lens) + 3)
        assert status == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,cap", [(1, 70000), (7, 5000), (37, 20000), (1025, 4097), (3000, 9000)])
def test_growth_and_release_match_reference(B, cap):
    """Prompts admitted, steps, sequences finished and cut back, in one batch each."""
    page, mp = 16, max(64, 70000 // 16 + 1 if B == 1 else 0)
    g = np.random.default_rng(B)
    s = state(g, [0] * B, page, mp, min(B * mp, 30000))
    d = Device(s)
    for turn in range(5):
        room = mp * page - s["ctx_len"]
        n_new = np.minimum(g.integers(0, max(2, 2 * cap // B), B), room)
        n_new = np.where(g.random(B) < 0.3, -g.integers(0, 2 * page * 3, B), n_new)
        n_new = np.where(g.random(B) < 0.1, -2**31, n_new)          # finished
        if turn == 0:
            n_new = np.minimum(np.abs(n_new), cap // B)
        s, _ = step(s, d, page, n_new, cap)


@pytest.mark.gpu
def test_refused_growth_leaves_the_sequence():
    g = np.random.default_rng(3)
    s = state(g, [10, 30, 16, 0, 64], 16, 5, 12)                    # 4 pages free
    d = Device(s)
    # 1 + 1 + 3 pages: they run out at the third sequence; the fourth comes after it
    s, status = step(s, d, 16, [7, 3, 40, 1, 0], 100)
    assert status & lla.STATUS_PAGES_SHORT
    # too many tokens for the list; past the table; the whole batch idle
    s, status = step(s, d, 16, [3, 3, 0, 0, 0], 4)
    assert status == lla.STATUS_PAGES_SHORT
    s, status = step(s, d, 16, [0, 0, 0, 0, 100], 200)
    assert status == lla.STATUS_CTX_RANGE
    s, status = step(s, d, 16, [0] * 5, 0)
    assert status == 0


@pytest.mark.gpu
def test_freed_pages_serve_the_same_call_and_rollback():
    g = np.random.default_rng(4)
    s = state(g, [64, 64, 0, 0], 16, 4, 8)                          # nothing free
    d = Device(s)
    s, status = step(s, d, 16, [-64, -20, 50, 10], 80)
    assert status == 0 and s["n_free"] == 0
    kept = {k: np.array(v, copy=True) for k, v in s.items()}
    s, _ = step(s, d, 16, [0, 0, 3, 1], 80)
    s, _ = step(s, d, 16, [0, 0, -3, -1], 0)
    for k in kept:
        np.testing.assert_array_equal(s[k], kept[k])


@pytest.mark.gpu
def test_damaged_tables_are_told_and_stay_in_bounds():
    page, mp, n_pages = 16, 4, 8
    s = state(np.random.default_rng(5), [20, 16, 0], page, mp, n_pages)
    s["block_table"][0, 1] = 99                                     # the page being written
    s["block_table"][1, 0] = -5
    d = Device(s)
    s, status = step(s, d, page, [2, 0, 3], 8)
    assert status == lla.STATUS_PAGE_RANGE
    s, status = step(s, d, page, [-22, -16, 0], 0)                  # given back as -1
    assert status == lla.STATUS_PAGE_RANGE
    s, status = step(s, d, page, [20, 20, 20], 60)                  # and handed out as -1
    assert status & lla.STATUS_PAGE_RANGE
    bad = state(np.random.default_rng(6), [20, 16], page, mp, n_pages)
    bad["ctx_len"][1] = 65                                          # past the table
    s, status = step(bad, Device(bad), page, [1, 1], 8)
    assert status == lla.STATUS_CTX_RANGE
    for nf in (-3, 100):
        bad = state(np.random.default_rng(7), [3, 0], page, mp, n_pages)
        bad["free_list"] = np.arange(n_pages)
        bad["n_free"] = nf
        step(bad, Device(bad), page, [1, 1], 8)
    full = state(np.random.default_rng(8), [64], page, mp, 4)
    full["n_free"] = 2                                              # pages freed twice
    full["free_list"][:2] = [0, 1]
    d = Device(full)
    got = d.call(page, [-64], 0)
    assert int(got["status"]) == lla.STATUS_PAGE_RANGE and int(got["n_free"]) == 4


@pytest.mark.gpu
def test_empty_batch_and_unaligned_lists():
    d = Device(dict(ctx_len=[], block_table=np.zeros((0, 3)), free_list=[1, 0], n_free=2))
    got = d.call(16, [], 5)
    assert got["tok_start"].tolist() == [0] and got["slot"].tolist() == [-1] * 5
    # every list may start on any element of a larger buffer
    s = state(np.random.default_rng(9), [5, 40], 16, 4, 12)
    d = Device(s)
    for name in ("ctx", "bt", "fl", "nf"):
        t = getattr(d, name)
        wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        wide[1:] = t.reshape(-1)
        setattr(d, name, wide[1:].view(t.shape))
    step(s, d, 16, [30, 1], 40)
