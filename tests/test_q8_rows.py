"""Appending the rows of a batch of which page_map refused some sequences: the others keep their
own keys and values.  Codes go by the float64 reference of the served sequences' tokens.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as P

import looped_transformer_decode_b200 as lla


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def test_refusals():
    from looped_transformer_decode_b200._lib import CQ8Cache
    cfg, p = lla.Cfg(4, 2, 64, 16, 32), ctypes.c_void_p(0x10000)
    cache = CQ8Cache(0x10000, 0x10000, 0x10000, 0x10000, 8, 16)

    def call(B=2, n=4, rows=p, ks=128, k=p):
        return lla.lib.lla_q8_append_rows(ctypes.byref(cfg.c()), ctypes.byref(cache), p, 8, 0, 0, B, 4,
                                          p, p, n, p, p, rows, k, ks, p, 128, None, None)

    assert call(B=0) == call(n=0) == call(B=0, rows=None) == lla.OK
    assert call(rows=ctypes.c_void_p(0x10002)) == call(ks=126) == call(k=None) == lla.ERR_INVALID


class Batch:
    """Sequences over a pool with too few pages."""

    def __init__(self, lens, page, width, n_pages, H=3, d=64, seed=0):
        self.g = np.random.default_rng(seed)
        self.page, self.H, self.d, self.B = page, H, d, len(lens)
        self.cfg = lla.Cfg(4, H, d, 16, 32)
        used = [-(-n // page) for n in lens]
        bt = np.full((len(lens), width), -1, np.int64)
        perm, at = self.g.permutation(n_pages), 0
        for b, m in enumerate(used):
            bt[b, :m] = perm[at:at + m]
            at += m
        self.ctx, self.bt, self.nf = i32(lens), i32(bt), i32([n_pages - at])
        self.free = i32(np.concatenate([perm[at:], np.zeros(at, int)]))
        self.cache = lla.q8_cache_alloc(self.cfg, n_pages, page)
        self.table = lla.rope_table(self.cfg, width * page + 1)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.codes = [np.zeros(self.cache.k.shape) for _ in "kv"]
        self.scale = [np.zeros(self.cache.k_scale.shape) for _ in "kv"]

    def expect(self, ctx, asked, x):
        """The reference after this step: which sequences were served, and their tokens packed."""
        before = ctx
        after = self.ctx.cpu().numpy().astype(int)
        got = after - before
        assert all(n in (0, m) for n, m in zip(got, asked))
        first = np.concatenate([[0], np.cumsum(asked)])
        at = np.concatenate([np.arange(first[b], first[b] + got[b]) for b in range(self.B)]).astype(int)
        pos = np.concatenate([np.arange(before[b], after[b]) for b in range(self.B)]).astype(int)
        start = np.concatenate([[0], np.cumsum(got)])
        t = self.table.double().cpu().numpy()[pos]
        rows = [x[0][at].double().cpu().numpy(), x[1][at].double().cpu().numpy()]
        rows[0] = P.rope_rows(rows[0], t[..., 0], t[..., 1], "half")
        for i in range(2):
            self.codes[i], self.scale[i], kind = P.q8_append(
                self.codes[i], self.scale[i], self.bt.cpu().numpy(), after, start, rows[i])
            want = (self.cache.k, self.cache.v)[i].cpu().numpy().astype(float)
            scale = (self.cache.k_scale, self.cache.v_scale)[i].double().cpu().numpy()
            np.testing.assert_allclose(scale, self.scale[i], rtol=16 * 2.0 ** -24)
            # half a step, and 127 * 12 fp32 roundings of the quotient
            assert (np.abs(want - self.codes[i])[kind > 0] <= 0.5 + 1e-4).all()
            self.codes[i], self.scale[i] = want, scale
        return got


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_until_the_pool_is_empty(captured):
    """One row per sequence, made before it is known which sequences find a page."""
    s = Batch([14, 16, 3, 31, 0, 8], 16, 4, 9)               # 6 pages held, 3 free
    B = s.B
    ones, rows = i32([1] * B), i32(range(B))
    lists = (torch.empty(B + 1, dtype=torch.int32, device="cuda"),
             torch.empty(B, dtype=torch.int64, device="cuda"),
             torch.empty(B, dtype=torch.int32, device="cuda"))
    x = [torch.zeros((B, s.H, s.d), device="cuda") for _ in "kv"]

    def step():
        lla.page_map(s.page, s.ctx, ones, s.bt, s.free, s.nf, B, *lists, status=s.status)
        lla.q8_append(s.cfg, s.table, s.cache, s.ctx, s.bt, lists[0], lists[2], *x,
                      status=s.status, row_start=rows)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    served = []
    for _ in range(8):
        ctx = s.ctx.cpu().numpy().astype(int)
        for t in x:
            t.copy_(torch.from_numpy(s.g.standard_normal(t.shape)))
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        served.append(s.expect(ctx, [1] * B, x).tolist())
    assert int(s.status) == lla.STATUS_PAGES_SHORT
    # some step refused a sequence and served a later one
    assert any(0 in n and 1 in n[n.index(0):] for n in served)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts_of_which_one_is_refused(dtype):
    s = Batch([5, 0, 17, 2], 16, 40, 60, H=5)
    for asked in ([30, 1200, 200, 60], [9, 0, 3, 500]):
        ctx = s.ctx.cpu().numpy().astype(int)
        total = sum(asked)
        x = [torch.from_numpy(s.g.standard_normal((total, 5, 64))).to(dtype).cuda() for _ in "kv"]
        start, _, pos = lla.page_map(s.page, s.ctx, i32(asked), s.bt, s.free, s.nf, total,
                                     status=s.status)
        first = np.concatenate([[0], np.cumsum(asked)])[:-1]
        lla.q8_append(s.cfg, s.table, s.cache, s.ctx, s.bt, start, pos, *x, status=s.status,
                      row_start=i32(first))
        s.expect(ctx, asked, x)
    assert int(s.status) & (lla.STATUS_PAGES_SHORT | lla.STATUS_CTX_RANGE)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_rows_outside_are_skipped_and_told(n):
    """Three sequences of n tokens; the rows of one would lie before, past or across the end."""
    cfg, page = lla.Cfg(4, 2, 64, 16, 32), 16
    width = -(-n // page)
    bt = i32(np.arange(3 * width).reshape(3, width))
    x = torch.randn((3 * n, 2, 64), device="cuda")
    args = (i32([n] * 3), bt, i32([0, n, 2 * n, 3 * n]), None, x, x)
    whole = lla.q8_cache_alloc(cfg, 3 * width, page)
    lla.q8_append(cfg, None, whole, *args)
    for bad in (-1, 2 * n + 1, 3 * n, 2 ** 31 - 1, -2 ** 31):
        cache = lla.q8_cache_alloc(cfg, 3 * width, page)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lla.q8_append(cfg, None, cache, *args, row_start=i32([0, bad, 2 * n]), status=status)
        assert int(status) == lla.STATUS_CTX_RANGE
        assert not cache.k[width:2 * width].any()
        for a, b in ((cache.k, whole.k), (cache.v, whole.v), (cache.k_scale, whole.k_scale)):
            assert torch.equal(a[:width], b[:width]) and torch.equal(a[2 * width:], b[2 * width:])
    # rows may be shared and in any order
    cache = lla.q8_cache_alloc(cfg, 3 * width, page)
    lla.q8_append(cfg, None, cache, *args, row_start=i32([2 * n, 0, 0]))
    assert torch.equal(cache.k[:width], whole.k[2 * width:])
    assert torch.equal(cache.k[width:2 * width], whole.k[:width])
    assert torch.equal(cache.k[2 * width:], whole.k[:width])
    # a sequence without new tokens has no rows, and its entry is not looked at
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = lla.q8_cache_alloc(cfg, 3 * width, page)
    lla.q8_append(cfg, None, cache, i32([n] * 3), bt, i32([0, n, n, 2 * n]), None, x, x,
                  row_start=i32([0, -7, 2 * n]), status=status)
    assert int(status) == 0 and not cache.k[width:2 * width].any()
    assert torch.equal(cache.k[2 * width:], whole.k[2 * width:])
    with pytest.raises(ValueError, match="row_start"):
        lla.q8_append(cfg, None, cache, *args, row_start=i32([0, 1]))
