"""Paged 8-bit cache: append, read and decode attention against the float64 reference.

Tolerances.  A code is the nearest integer of value / scale, so it lies within half a step of
the real quotient, plus the quotient's own error: |value / scale| <= 127 computed with at most
12 fp32 roundings (rotation, amax / 127, its reciprocal, the product), 127 * 12 * 2^-24 < 1e-4.
Attention: with q held to 2^-21 of its largest element and fp32 sums over d + 8 terms, a score
is off by at most ds = sm_scale * ((d + 8) 2^-24 sum |q_i k_i| + 2^-21 max|q| sum |k_i|) over the
tokens' largest, a weight by 2 ds relatively, and n weights, each held to 2^-24 of the largest,
by n 2^-24 of their sum at most; 64 more roundings merge.  All of it scales with the largest
value attended to; bf16 results add half a step.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as P

import looped_transformer_decode_b200 as lla

QUOTIENT = 1e-4


def cfg_of(H, d, d_rope=0, **kw):
    return lla.Cfg(4, H, d, 16, 32, d_rope=d_rope, **kw)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def rows_of(table, pos):
    t = table.double().cpu().numpy()[np.asarray(pos, np.int64)]
    return t[..., 0], t[..., 1]


# ----------------------------------------------------------------------------- reference

def test_reference_rounds_within_its_scale():
    """Tokens appended one by one: every value stays within (1 + 2.5) half steps of the final
    scale, the geometric bound on its repeated roundings."""
    g = np.random.default_rng(0)
    page, H, d = 16, 2, 8
    codes, scale = np.zeros((1, H, page, d)), np.zeros((1, H))
    x = g.standard_normal((page, H, d)) * np.linspace(0.1, 3, page)[:, None, None]
    for i in range(page):
        codes, scale, kind = P.q8_append(codes, scale, [[0]], [i + 1], [0, 1], x[i:i + 1])
        codes = np.where(kind[..., None] > 0, np.round(codes), codes)
        assert np.abs(codes).max() <= 127
    got = codes[0] * scale[0][:, None, None]
    err = np.abs(got - np.moveaxis(x, 0, 1)) / scale[0][:, None, None]
    assert err.max() <= 0.5 / (1 - 1 / P.GROW)


def test_reference_attention_plain_loop():
    g = np.random.default_rng(1)
    q, ks, vs = g.standard_normal((3, 4))
    k, v = g.standard_normal((2, 5, 4))
    w = [np.exp(0.5 * float(q @ x)) for x in list(k) + [ks]]
    want = sum(a * x for a, x in zip(w, list(v) + [vs])) / sum(w)
    assert np.allclose(P.q8_attention(q, ks, vs, k, v, 0.5), want)
    assert np.array_equal(P.q8_attention(q, None, None, k[:0], v[:0], 0.5), np.zeros(4))


# ----------------------------------------------------------------------------- refusals

def test_configuration_copies_after_use():
    """The cached C struct of a configuration stays out of copies and comparisons."""
    import copy
    import dataclasses
    import pickle
    cfg = cfg_of(2, 64)
    assert lla.q8_decode_launches(cfg, 1, 64) == 1               # makes the struct
    for other in (pickle.loads(pickle.dumps(cfg)), copy.deepcopy(cfg), copy.copy(cfg),
                  dataclasses.replace(cfg)):
        assert other == cfg and hash(other) == hash(cfg)
        assert lla.q8_decode_launches(other, 1, 64) == 1
    assert lla.q8_decode_launches(dataclasses.replace(cfg, d_head=80), 1, 64) == -1


PTR = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
BAD, NO = lla.ERR_INVALID, lla.ERR_UNSUPPORTED


def c_cache(n=8, page=16, k=0x10000, v=0x10000, ks=0x10000, vs=0x10000):
    from looped_transformer_decode_b200._lib import CQ8Cache
    return CQ8Cache(k, v, ks, vs, n, page)


def shared_refusals(call):
    for kw, code in ((dict(cache=None), BAD), (dict(cache=c_cache(page=20)), NO),
                     (dict(cache=c_cache(n=-1)), BAD), (dict(cache=c_cache(k=None)), BAD),
                     (dict(cache=c_cache(vs=None)), BAD), (dict(cache=c_cache(v=0x10008)), BAD),
                     (dict(cfg=cfg_of(2, 48)), NO), (dict(cfg=cfg_of(0, 64)), NO)):
        assert call(**kw) == code, kw


def test_append_refusals():
    f = lla.lib.lla_q8_append

    def call(cfg=cfg_of(2, 64), cache=c_cache(), rope=PTR, mp=8, layout=0, dtype=0, B=2, pages=4,
             ctx=PTR, bt=PTR, n=4, ts=PTR, pos=PTR, k=PTR, ks=128, v=PTR, vs=128, st=None):
        return f(ctypes.byref(cfg.c()), None if cache is None else ctypes.byref(cache), rope, mp,
                 layout, dtype, B, pages, ctx, bt, n, ts, pos, k, ks, v, vs, st, None)

    shared_refusals(call)
    assert call(B=0) == call(n=0) == call(pages=0) == call(cache=c_cache(n=0)) == lla.OK
    for kw, code in ((dict(layout=3), BAD), (dict(dtype=7), NO), (dict(B=-1), BAD),
                     (dict(B=65536), NO), (dict(pages=1 << 27), NO), (dict(n=-1), BAD),
                     (dict(mp=0), BAD), (dict(pos=None), BAD), (dict(ctx=None), BAD),
                     (dict(bt=None), BAD), (dict(ts=None), BAD), (dict(k=None), BAD),
                     (dict(v=None), BAD), (dict(k=ODD), BAD), (dict(ks=126), BAD),
                     (dict(vs=64), BAD), (dict(ks=130), BAD), (dict(vs=-128), BAD),
                     (dict(ctx=ctypes.c_void_p(0x10002)), BAD),
                     (dict(st=ctypes.c_void_p(0x10001)), BAD)):
        assert call(**kw) == code, kw


def test_read_refusals():
    f = lla.lib.lla_q8_read

    def call(cfg=cfg_of(2, 64), cache=c_cache(), n=4, slot=PTR, k=PTR, v=PTR, st=None):
        return f(ctypes.byref(cfg.c()), None if cache is None else ctypes.byref(cache), n, slot, k,
                 v, st, None)

    shared_refusals(call)
    assert call(n=0) == lla.OK
    for kw, code in ((dict(n=-1), BAD), (dict(n=1 << 60), NO), (dict(slot=None), BAD),
                     (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=ODD), BAD),
                     (dict(slot=ctypes.c_void_p(0x10004)), BAD)):
        assert call(**kw) == code, kw


def test_decode_refusals():
    f = lla.lib.lla_q8_decode_attn

    def call(cfg=cfg_of(2, 64), cache=c_cache(), rope=PTR, mp=8, layout=0, dtype=0, B=2, pages=4,
             ctx=PTR, bt=PTR, q=PTR, ks=PTR, vs=PTR, qp=PTR, out=PTR, ws=PTR, nb=None):
        if nb is None:
            nb = 1 << 30
        return f(ctypes.byref(cfg.c()), None if cache is None else ctypes.byref(cache), rope, mp,
                 layout, dtype, B, pages, ctx, bt, q, ks, vs, qp, out, ws, nb, None)

    shared_refusals(call)
    assert call(B=0) == lla.OK
    for kw, code in ((dict(layout=-1), BAD), (dict(dtype=2), NO), (dict(B=-1), BAD),
                     (dict(B=65536), NO), (dict(pages=-1), BAD), (dict(pages=1 << 27), NO),
                     (dict(mp=0), BAD), (dict(ctx=None), BAD), (dict(bt=None), BAD),
                     (dict(q=None), BAD), (dict(out=None), BAD), (dict(ws=None), BAD),
                     (dict(qp=None), BAD), (dict(ks=None), BAD), (dict(vs=None), BAD),
                     (dict(q=ODD), BAD), (dict(out=ODD), BAD), (dict(ws=ODD), BAD),
                     (dict(qp=ctypes.c_void_p(0x10001)), BAD),
                     (dict(nb=16), lla.ERR_TOO_SMALL)):
        assert call(**kw) == code, kw
    assert "workspace" in lla.last_error()
    c = ctypes.byref(cfg_of(2, 64).c())
    assert lla.lib.lla_q8_cache_bytes(c, 10, 32) == 10 * 2 * 32 * 64
    assert lla.lib.lla_q8_cache_bytes(c, 10, 33) == 0
    assert lla.lib.lla_q8_decode_workspace_bytes(c, 70000, 64) == 0
    assert lla.q8_decode_launches(cfg_of(2, 64), 0, 64) == 0
    assert lla.q8_decode_launches(cfg_of(2, 64), 4, -1) == -1


def test_binding_refuses_what_is_not_on_a_gpu():
    """The Python entry points name the argument, and no call reaches the library."""
    cfg = cfg_of(2, 64)
    x, one = torch.zeros((1, 2, 64)), torch.zeros(1, dtype=torch.int32)
    cache = lla.q8_cache_alloc(cfg, 2, 16, device="cpu")
    bt, slot = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    calls = {
        "x": lambda v: lla.rope_apply(cfg, torch.zeros((4, 32, 2)), one, v),
        "k": lambda v: lla.q8_append(cfg, None, cache, one, bt, one, None, v, v),
        "q": lambda v: lla.q8_decode_attn(cfg, None, cache, one, bt, v, None, None, None),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"{name} must be a CUDA tensor"):
            call(x)
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            call([1.0])
    with pytest.raises(ValueError, match="slot must be a CUDA tensor"):
        lla.q8_read(cfg, cache, slot)
    with pytest.raises(ValueError, match="ctx_len must be a CUDA tensor"):
        lla.page_map(16, one, one, bt, one, one, 4)


# ----------------------------------------------------------------------------- GPU: append and read

def random_cache(g, cfg, n_pages, page):
    c = lla.q8_cache_alloc(cfg, n_pages, page)
    shape = c.k.shape
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes.copy_(torch.from_numpy(np.clip(np.round(g.standard_normal(shape) * 36), -127, 127)
                                     .astype(np.int8)))
        scale.copy_(torch.from_numpy(np.exp(0.3 * g.standard_normal(shape[:2])) / 36))
    return c


def layout_pages(g, lens, page, spare=2):
    n = [-(-int(x) // page) for x in lens]
    width, total = max(n + [1]) + 1, sum(n) + spare
    perm = g.permutation(total)
    bt = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, m in enumerate(n):
        bt[b, :m] = perm[at:at + m]
        at += m
    return bt, total


def check_append(codes_before, scale_before, cache_codes, cache_scale, bt, after, start, x):
    want, scale, kind = P.q8_append(codes_before, scale_before, bt, after, start, x)
    got = cache_codes.cpu().numpy().astype(np.float64)
    gs = cache_scale.double().cpu().numpy()
    assert np.abs(gs - scale).max() <= 16 * 2.0 ** -24 * np.abs(scale).max()
    np.testing.assert_allclose(gs, scale, rtol=16 * 2.0 ** -24)
    assert (np.abs(got - want)[kind > 0] <= 0.5 + QUOTIENT).all()
    np.testing.assert_array_equal(got[kind == 0], want[kind == 0])
    assert np.abs(got[kind > 0]).max(initial=0) <= 127


APPENDS = [  # lens before, new tokens
    ([0], [1]), ([15], [2]), ([16, 0, 31], [1, 0, 1]), ([5, 70, 0, 128], [40, 1, 129, 0]),
    ([0, 0], [0, 300]), ([7] * 20, [1] * 20),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page,d,d_rope,layout", [
    (16, 128, 0, "half"), (32, 96, 64, "interleaved"), (64, 64, 32, "half"),
    (128, 32, 0, "interleaved"), (16, 96, 0, "half"), (128, 128, 64, "half"), (64, 128, 0, None)])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_matches_reference(dtype, page, d, d_rope, layout, case):
    old, new = (np.array(a) for a in APPENDS[case])
    g = np.random.default_rng(case * 100 + d + page)
    cfg = cfg_of(3, d, d_rope)
    after = old + new
    bt, n_pages = layout_pages(g, after, page)
    cache = random_cache(g, cfg, n_pages, page)
    before = [t.cpu().numpy().astype(np.float64) for t in (cache.k, cache.k_scale, cache.v,
                                                           cache.v_scale)]
    start = np.concatenate([[0], np.cumsum(new)])
    n = int(start[-1])
    wide = torch.from_numpy(g.standard_normal((n + 2, 3, 3, d)) * 1.5).to(dtype).cuda()
    k, v = wide[:, 1], wide[:, 2]                    # two rows more than there are tokens
    pos = np.concatenate([np.arange(o, o + m) for o, m in zip(old, new)] + [[0, 0]]).astype(int)
    table = lla.rope_table(cfg, int(after.max()) + 1) if layout else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lla.q8_append(cfg, table, cache, i32(after), i32(bt), i32(start), i32(pos) if layout else None,
                  k, v, layout=layout or "half", status=st)
    assert int(st) == 0
    x = k[:n].double().cpu().numpy()
    if layout:
        x = P.rope_rows(x, *rows_of(table, pos[:n]), layout)
    check_append(before[0], before[1], cache.k, cache.k_scale, bt, after, start, x)
    check_append(before[2], before[3], cache.v, cache.v_scale, bt, after, start,
                 v[:n].double().cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("H,page,d,d_rope,layout,dtype,old,new", [
    # few tokens for many sequences, but several pages of one of them
    (3, 16, 64, 0, "half", torch.float32, [5] * 20, [100] + [0] * 19),
    (20, 32, 96, 32, "interleaved", torch.bfloat16, [5, 31, 0, 64] * 5, [3, 2, 33, 1] * 5),
    (40, 64, 64, 0, "half", torch.float32, [5, 31, 0, 64] * 5, [13, 2, 33, 10] * 5),
    # prompts of more heads than a block's: its share begins and ends inside pages
    (40, 64, 128, 64, "interleaved", torch.bfloat16, [0, 70, 5], [700, 0, 900]),
    (33, 128, 128, 0, "half", torch.float32, [130, 0], [300, 259]),
    (128, 16, 32, 0, "half", torch.bfloat16, [1, 0, 7, 16], [40, 16, 0, 400]),
    (1, 64, 96, 64, "half", torch.float32, [63, 0], [1, 2000])])
def test_append_of_many_heads_and_uneven_lengths(H, page, d, d_rope, layout, dtype, old, new):
    old, new = np.array(old), np.array(new)
    g = np.random.default_rng(H + page)
    cfg = cfg_of(H, d, d_rope)
    after = old + new
    bt, n_pages = layout_pages(g, after, page)
    cache = random_cache(g, cfg, n_pages, page)
    before = [t.cpu().numpy().astype(np.float64) for t in (cache.k, cache.k_scale, cache.v,
                                                           cache.v_scale)]
    start = np.concatenate([[0], np.cumsum(new)])
    n = int(start[-1])
    k, v = (torch.from_numpy(g.standard_normal((n, H, d)) * 1.5).to(dtype).cuda() for _ in "kv")
    pos = np.concatenate([np.arange(o, o + m) for o, m in zip(old, new)]).astype(int)
    table = lla.rope_table(cfg, int(after.max()) + 1)
    lla.q8_append(cfg, table, cache, i32(after), i32(bt), i32(start), i32(pos), k, v, layout=layout)
    x = P.rope_rows(k.double().cpu().numpy(), *rows_of(table, pos), layout)
    check_append(before[0], before[1], cache.k, cache.k_scale, bt, after, start, x)
    check_append(before[2], before[3], cache.v, cache.v_scale, bt, after, start,
                 v.double().cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 40])
def test_append_onto_a_scale_that_no_append_leaves(n):
    """A scale of 1e-38 counts as zero: the earlier tokens read as zeros, the new ones as
    themselves, or as zeros where they count as zero too."""
    cfg, page = cfg_of(2, 64), 16
    cache = lla.q8_cache_alloc(cfg, 4, page)
    cache.k.fill_(100)
    cache.v.fill_(-100)
    cache.k_scale.fill_(1e-38)
    cache.v_scale.fill_(1e-38)
    x = torch.zeros((n, 2, 64), device="cuda")
    x[:, 0], x[:, 1] = 1e-31, 0.5
    lla.q8_append(cfg, None, cache, i32([5 + n]), i32([[2, 0, 3]]), i32([0, n]), None, x, x)
    at = torch.arange(5 + n, device="cuda")
    k, v = lla.q8_read(cfg, cache, torch.tensor([2, 0, 3], device="cuda")[at // page] * page + at % page)
    want = torch.zeros((5 + n, 2, 64), dtype=torch.bfloat16, device="cuda")
    want[5:, 1] = 0.5
    assert torch.equal(k, want) and torch.equal(v, want)


@pytest.mark.gpu
@pytest.mark.parametrize("n,H,d", [(6001, 5, 96), (40003, 1, 64), (513, 128, 128)])
def test_read_of_many_rows(n, H, d):
    cfg, page = cfg_of(H, d), 16
    g = np.random.default_rng(n)
    cache = random_cache(g, cfg, 9, page)
    slot = torch.from_numpy(g.integers(0, 9 * page, n)).cuda()
    slot[n - 1] = slot[n // 2] = 9 * page
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = lla.q8_read(cfg, cache, slot, status=st)
    ok = slot < 9 * page
    p, r = slot[ok] // page, slot[ok] % page
    assert int(st) == lla.STATUS_SLOT_RANGE and not k[~ok].any() and not v[~ok].any()
    assert torch.equal(k[ok], (cache.k[p, :, r].float() * cache.k_scale[p][..., None]).bfloat16())
    assert torch.equal(v[ok], (cache.v[p, :, r].float() * cache.v_scale[p][..., None]).bfloat16())


@pytest.mark.gpu
def test_token_by_token_append_stays_near_the_values():
    """A sequence grown one token at a time, values rising: each read value is within the
    geometric bound of its repeated roundings, 2.5 final scales."""
    cfg, page, n = cfg_of(2, 64), 32, 70
    g = np.random.default_rng(5)
    x = torch.from_numpy(g.standard_normal((n, 2, 64)) * np.linspace(0.2, 4, n)[:, None, None]).float().cuda()
    cache = lla.q8_cache_alloc(cfg, 4, page)
    bt = i32([[2, 0, 3]])
    for i in range(n):
        lla.q8_append(cfg, None, cache, i32([i + 1]), bt, i32([0, 1]), None, x[i:i + 1], x[i:i + 1])
    slot = torch.tensor([[2, 0, 3][j // page] * page + j % page for j in range(n)], device="cuda")
    k, v = lla.q8_read(cfg, cache, slot)
    assert torch.equal(k, v)
    s = cache.v_scale[slot // page][:, :, None]
    bound = 0.5 / (1 - 1 / P.GROW) * s * (1 + 1e-3) + 2.0 ** -8 * x.abs()
    assert ((v.float() - x).abs() <= bound).all()


@pytest.mark.gpu
def test_unusual_values():
    """Zeros, tiny values, NaN and infinities, and a stale scale that is not a number."""
    cfg, page = cfg_of(1, 32), 16
    cache = lla.q8_cache_alloc(cfg, 3, page)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("inf"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros((20, 1, 32), device="cuda")
    x[:16] = 1e-32                                   # stored as zeros
    x[17, 0, 3], x[18, 0, 4], x[19, 0, 5] = 2.0, float("inf"), float("nan")
    x[18, 0, 6] = -float("inf")
    args = (i32([20]), i32([[1, 2]]), i32([0, 20]), None)
    lla.q8_append(cfg, None, cache, *args, x, x, status=st)
    assert int(st) == lla.STATUS_NONFINITE
    k, v = lla.q8_read(cfg, cache, torch.arange(16, 36, device="cuda"))
    want = torch.nan_to_num(x, nan=0.0, posinf=2.0, neginf=-2.0).float()
    want[:16] = 0
    assert torch.equal(k.float(), want) and torch.equal(v.float(), want)
    # a held page whose scale is damaged keeps nothing of it
    cache.k_scale[2] = float("nan")
    one = torch.full((1, 1, 32), 0.5, device="cuda")
    lla.q8_append(cfg, None, cache, i32([21]), i32([[1, 2]]), i32([0, 1]), None, one, one)
    k, _ = lla.q8_read(cfg, cache, torch.tensor([33, 36], device="cuda"))
    assert torch.equal(k[0].float(), torch.zeros_like(k[0].float())) and torch.equal(k[1], one[0].bfloat16())


@pytest.mark.gpu
def test_read_matches_codes_and_skips_foreign_slots():
    cfg, page = cfg_of(5, 96), 32
    g = np.random.default_rng(8)
    cache = random_cache(g, cfg, 7, page)
    slot = torch.from_numpy(g.integers(0, 7 * page, 300)).cuda()
    slot[17], slot[44], slot[45] = -1, 7 * page, 2 ** 40
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((300, 5, 96), 9.0, dtype=torch.bfloat16, device="cuda")
    k, v = lla.q8_read(cfg, cache, slot, k_out=out, status=st)
    assert int(st) == lla.STATUS_SLOT_RANGE
    ok = (slot >= 0) & (slot < 7 * page)
    p, r = slot[ok] // page, slot[ok] % page
    assert torch.equal(k[ok], (cache.k[p, :, r].float() * cache.k_scale[p][..., None]).bfloat16())
    assert torch.equal(v[ok], (cache.v[p, :, r].float() * cache.v_scale[p][..., None]).bfloat16())
    assert (k[~ok] == 9).all() and (v[~ok] == 0).all()


@pytest.mark.gpu
def test_damaged_append_lists_are_told_and_stay_in_bounds():
    cfg, page = cfg_of(2, 64), 16
    x = torch.randn((40, 2, 64), device="cuda")
    good = (i32([20, 12]), i32([[0, 1, -1], [2, -1, -1]]), i32([0, 20, 32]))

    def run(ctx, bt, start):
        cache = lla.q8_cache_alloc(cfg, 4, page)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        lla.q8_append(cfg, None, cache, ctx, bt, start, None, x, x, status=st)
        return int(st), cache.k

    status, want = run(*good)
    assert status == 0 and want[0].any() and want[1].any() and want[2].any() and not want[3].any()
    # sequence 0 is skipped, sequence 1 written as before
    for ctx, bt, start, bit in (
            (i32([19, 12]), good[1], good[2], lla.STATUS_CTX_RANGE),      # shorter than its tokens
            (i32([49, 12]), good[1], good[2], lla.STATUS_CTX_RANGE),      # longer than the table
            (good[0], i32([[4, -2, -1], [2, -1, -1]]), good[2], lla.STATUS_PAGE_RANGE)):
        status, got = run(ctx, bt, start)
        assert status == bit and torch.equal(got[2], want[2]) and not got[:2].any()
    status, got = run(good[0], good[1], i32([-5, 20, 100]))               # lists out of bounds
    assert status == lla.STATUS_CTX_RANGE and not got.any()


# ----------------------------------------------------------------------------- GPU: attention

def attend(g, cfg, page, lens, layout, dtype, self_tok=True, q_scale=1.0, spread=0.0, pos=None,
           shared=None):
    """Run the decode and return (got, want, bound)."""
    H, d, B = cfg.H, cfg.d_head, len(lens)
    bt, n_pages = layout_pages(g, lens, page, spare=3)
    cache = random_cache(g, cfg, n_pages, page)
    if spread:
        cache.v_scale *= torch.exp(spread * torch.randn(cache.v_scale.shape, device="cuda"))
    used = np.zeros(n_pages, bool)
    used[bt[bt >= 0]] = True
    free = torch.from_numpy(~used).cuda()
    cache.k_scale[free] = float("nan")               # nothing of other pages may reach the output
    cache.v_scale[free] = float("inf")
    if shared:
        bt[1, :shared] = bt[0, :shared]              # a common prefix
    pos = np.asarray(lens) if pos is None else pos
    table = lla.rope_table(cfg, int(max(pos)) + 1) if layout else None
    q, k, v = (torch.from_numpy(g.standard_normal((B, H, d)) * c).to(dtype).cuda()
               for c in (q_scale, 1.0, 1.0))
    ws = lla.q8_decode_workspace(cfg, B, bt.shape[1] * page)
    got = lla.q8_decode_attn(cfg, table, cache, i32(lens), i32(bt), q, k if self_tok else None,
                             v if self_tok else None, i32(pos), layout=layout or "half", ws=ws)
    again = lla.q8_decode_attn(cfg, table, cache, i32(lens), i32(bt), q, k if self_tok else None,
                               v if self_tok else None, i32(pos), layout=layout or "half", ws=ws)
    assert torch.equal(got, again)                   # same inputs, same bits
    assert lla.decode_status(ws) == 0
    scale = cfg.sm_scale or 1 / np.sqrt(d)
    qs, ks, vs = (t.double().cpu().numpy() for t in (q, k, v))
    if layout:
        cs = rows_of(table, pos)
        qs, ks = P.rope_rows(qs, *cs, layout), P.rope_rows(ks, *cs, layout)
    kc, vc = cache.k.cpu().numpy().astype(np.float64), cache.v.cpu().numpy().astype(np.float64)
    ksc, vsc = cache.k_scale.double().cpu().numpy(), cache.v_scale.double().cpu().numpy()
    want, tol = np.zeros((B, H, d)), np.zeros((B, H, d))
    for b, n in enumerate(lens):
        pages = bt[b, :-(-int(n) // page)]
        for h in range(H):
            kk = (kc[pages, h] * ksc[pages, h, None, None]).reshape(-1, d)[:n]
            vv = (vc[pages, h] * vsc[pages, h, None, None]).reshape(-1, d)[:n]
            own = (ks[b, h], vs[b, h]) if self_tok else (None, None)
            want[b, h] = P.q8_attention(qs[b, h], *own, kk, vv, scale)
            if n == 0:
                continue
            ds = scale * ((d + 8) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qs[b, h])).max()
                          + 2.0 ** -21 * np.abs(qs[b, h]).max() * np.abs(kk).sum(1).max())
            big = max(np.abs(vv).max(), np.abs(vs[b, h]).max() if self_tok else 0.0)
            tol[b, h] = big * (2 * ds + (n + 64) * 2.0 ** -24)
    tol += torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -60
    return got.double().cpu().numpy(), want, tol


LENS = [[0], [1], [15, 16, 17, 0], [128], [300, 1, 0, 64, 65, 1000], [4100, 33]]


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,d_rope,layout,dtype,self_tok", [
    (128, 16, 0, "half", torch.float32, True), (128, 64, 64, "interleaved", torch.bfloat16, False),
    (96, 32, 0, "interleaved", torch.float32, False), (96, 128, 32, "half", torch.float32, True),
    (64, 16, 0, "half", torch.bfloat16, True), (64, 128, 32, "interleaved", torch.float32, False),
    (32, 16, 0, "half", torch.float32, True), (32, 64, 0, "interleaved", torch.float32, False),
    (128, 32, 0, None, torch.float32, True)])
@pytest.mark.parametrize("lens", range(len(LENS)))
def test_decode_matches_reference(d, page, d_rope, layout, dtype, self_tok, lens):
    g = np.random.default_rng(d + page + lens)
    got, want, tol = attend(g, cfg_of(3, d, d_rope), page, LENS[lens], layout, dtype, self_tok)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()
    if not self_tok:
        for b, n in enumerate(LENS[lens]):
            assert n or not got[b].any()


@pytest.mark.gpu
@pytest.mark.parametrize("d,page", [(128, 16), (96, 64), (64, 32), (32, 128)])
def test_decode_sharp_and_uneven(d, page):
    """Queries that single tokens out, value scales over orders of magnitude, many heads."""
    g = np.random.default_rng(d)
    for kw in (dict(q_scale=12.0), dict(spread=2.5), dict(q_scale=0.0)):
        got, want, tol = attend(g, cfg_of(17, d), page, [700, 0, 90], "half", torch.float32, **kw)
        assert (np.abs(got - want) <= tol).all(), kw


@pytest.mark.gpu
def test_decode_shared_prefix_and_scale():
    g = np.random.default_rng(77)
    got, want, tol = attend(g, cfg_of(4, 128, sm_scale=0.25), 16, [200, 180], "half",
                            torch.float32, shared=6)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,n", [
    (1, 1, 40000), (2, 16, 9000), (300, 2, 200),      # an item cut into many pieces, many items
    (1000, 3, 70),                                    # items whole to a warp each
    (120, 16, 600), (40, 12, 1500)])                  # ranges that begin and end inside items
def test_decode_many_splits_and_many_sequences(B, H, n):
    g = np.random.default_rng(n)
    lens = np.maximum(1, (n * g.random(B) ** 2).astype(int))
    lens[0] = n
    got, want, tol = attend(g, cfg_of(H, 64), 64, lens, "half", torch.float32)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.gpu
def test_decode_of_zero_scales_and_extreme_codes():
    """Pages of zeros, codes of -128, and every weight on a value of zero."""
    cfg, page = cfg_of(1, 64), 16
    cache = lla.q8_cache_alloc(cfg, 2, page)
    cache.k.fill_(-128)
    cache.v.fill_(-128)
    q = torch.ones((1, 1, 64), device="cuda")
    args = (i32([32]), i32([[0, 1]]), q, None, None, None)
    assert not lla.q8_decode_attn(cfg, None, cache, *args).any()          # all scales zero
    cache.v_scale[1] = 0.5
    got = lla.q8_decode_attn(cfg, None, cache, *args)                     # half the weight each
    assert (got - -32).abs().max() <= 32 * 40 * 2.0 ** -24
    cache.k_scale.fill_(1.0)
    got = lla.q8_decode_attn(cfg, None, cache, *args)
    assert (got - -32).abs().max() <= 32 * 40 * 2.0 ** -24


@pytest.mark.gpu
def test_decode_of_queries_that_are_not_numbers():
    """A NaN or an infinity in q or k_self reaches its own head only; an empty row stays zero.
    A score of minus infinity (q negative where k_self is infinite) has weight zero."""
    cfg, page = cfg_of(3, 64), 16
    cache = random_cache(np.random.default_rng(2), cfg, 4, page)
    q = torch.randn((2, 3, 64), device="cuda")
    k = torch.randn((2, 3, 64), device="cuda")
    args = (i32([20, 0]), i32([[0, 1], [2, 3]]))
    want = lla.q8_decode_attn(cfg, None, cache, *args, q, k, k, None)
    alone = lla.q8_decode_attn(cfg, None, cache, *args, q, None, None, None)
    for bad in (float("nan"), float("inf")):
        for which in (0, 1):
            rows = [q.clone(), k.clone()]
            rows[which][:, 1, 5] = bad
            got = lla.q8_decode_attn(cfg, None, cache, *args, rows[0], rows[1], k, None)
            assert got[1, 1].isnan().all()
            if which == 1 and bad == float("inf") and q[0, 1, 5] < 0:
                assert torch.allclose(got[0, 1], alone[0, 1], rtol=1e-6)
            else:
                assert got[0, 1].isnan().all()
            assert torch.equal(got[:, 0::2], want[:, 0::2])
            got = lla.q8_decode_attn(cfg, None, cache, *args, rows[0], None, None, None)
            assert not got[1].any() and got[0, 1].isnan().all() == (which == 0)


@pytest.mark.gpu
def test_decode_of_damaged_lists():
    cfg, page = cfg_of(2, 64), 16
    g = np.random.default_rng(11)
    cache = random_cache(g, cfg, 4, page)
    q = torch.randn((2, 2, 64), device="cuda")

    def run(lens, bt, pos=(0, 0)):
        table = lla.rope_table(cfg, 4)
        ws = lla.q8_decode_workspace(cfg, 2, len(bt[0]) * page)
        out = lla.q8_decode_attn(cfg, table, cache, i32(lens), i32(bt), q, q, q, i32(pos), ws=ws)
        return out, lla.decode_status(ws), ws

    want, st, ws = run([16, 32], [[0, 3], [1, 2]])
    assert st == 0
    out, st, _ = run([32, 40], [[0, 9], [1, 2]])      # a foreign page; longer than the table
    assert st == lla.STATUS_PAGE_RANGE | lla.STATUS_CTX_RANGE
    assert torch.allclose(out, want, atol=1e-6)       # the page left out, the length clamped
    out, st, _ = run([32, 32], [[9, -1], [1, 2]])     # no page of a sequence there
    assert st == lla.STATUS_PAGE_RANGE and torch.equal(out[0], q[0]) and torch.equal(out[1], want[1])
    out, st, _ = run([-3, 32], [[0, 3], [1, 2]])
    assert st == lla.STATUS_CTX_RANGE and torch.equal(out[0], q[0]) and torch.equal(out[1], want[1])
    out, st, _ = run([16, 32], [[0, 3], [1, 2]], pos=(-1, 4))
    assert st == lla.STATUS_POSITION_RANGE and torch.isfinite(out).all()
    # the next call on a workspace starts clean
    lla.q8_decode_attn(cfg, None, cache, i32([16, 32]), i32([[0, 3], [1, 2]]), q, q, q, None, ws=ws)
    assert lla.decode_status(ws) == 0


@pytest.mark.gpu
def test_python_argument_checks():
    cfg = cfg_of(2, 64)
    cache = lla.q8_cache_alloc(cfg, 2, 16)
    q = torch.zeros((1, 2, 64), device="cuda")
    one, bt = i32([1]), i32([[0]])
    with pytest.raises(TypeError):
        lla.q8_decode_attn(cfg, None, cache, one, bt, q.half(), None, None, None)
    with pytest.raises(ValueError):
        lla.q8_decode_attn(cfg, None, cache, one, bt, q[:, :1], None, None, None)
    with pytest.raises(ValueError):
        lla.q8_decode_attn(cfg, lla.rope_table(cfg_of(2, 96), 4), cache, one, bt, q, None, None, one)
    with pytest.raises(ValueError):
        lla.q8_decode_attn(cfg_of(3, 64), None, cache, one, bt, torch.zeros((1, 3, 64), device="cuda"),
                           None, None, None)
    with pytest.raises(ValueError):
        lla.q8_append(cfg, None, cache, one.cpu(), bt, i32([0, 1]), None, q, q)
    with pytest.raises(ValueError):
        lla.q8_append(cfg, None, cache, one, bt, i32([0, 1]), None, q.transpose(1, 2), q)
    with pytest.raises(ValueError, match="layout"):
        lla.q8_append(cfg, None, cache, one, bt, i32([0, 1]), None, q, q, layout="both")
    with pytest.raises(ValueError, match="heads of a token must be contiguous"):
        lla.rope_apply(cfg, lla.rope_table(cfg, 4), one, torch.zeros((1, 2, 128), device="cuda")[..., ::2])
    with pytest.raises(TypeError, match="slot must be torch.int64"):
        lla.q8_read(cfg, cache, one)
    with pytest.raises(lla.LLAError) as e:
        lla.q8_decode_attn(cfg, None, cache, one, bt, q, None, None, None,
                           ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == lla.ERR_TOO_SMALL and "workspace" in str(e.value)
    with pytest.raises(AttributeError):
        lla.q8_read(None, cache, torch.zeros(1, dtype=torch.int64, device="cuda"))


# ----------------------------------------------------------------------------- GPU: together

@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    """Prompts admitted, then decode steps of one layer and loop: pages, append, attention over
    the history and the in-flight token, all on one side stream; replayed from a graph too."""
    cfg, page, steps = cfg_of(4, 64, 32), 16, 20
    g = np.random.default_rng(9)
    prompt = np.array([37, 0, 100, 5])
    B, n_max = len(prompt), 160
    x = {n: torch.from_numpy(g.standard_normal((B, n_max, 4, 64))).float().cuda() for n in "qkv"}
    scaling = lla.RopeScaling("yarn", 4.0, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        table = lla.rope_table(cfg, n_max, scaling=scaling)
        cache = lla.q8_cache_alloc(cfg, 48, page)
        ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        bt = torch.full((B, n_max // page), -1, dtype=torch.int32, device="cuda")
        free = torch.arange(48, dtype=torch.int32, device="cuda")
        nf = torch.tensor([48], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        total = int(prompt.sum())
        start, slot, pos = lla.page_map(page, ctx, i32(prompt), bt, free, nf, total, status=status)
        rows = [torch.cat([x[n][b, :m] for b, m in enumerate(prompt)]) for n in "kv"]
        lla.q8_append(cfg, table, cache, ctx, bt, start, pos, *rows, layout="interleaved",
                      status=status)
        ones = torch.ones(B, dtype=torch.int32, device="cuda")
        now = {n: torch.zeros((B, 4, 64), device="cuda") for n in "qkv"}
        out = torch.zeros((B, 4, 64), device="cuda")
        ws = lla.q8_decode_workspace(cfg, B, n_max)
        t_ids = (torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                 torch.empty(B, dtype=torch.int64, device="cuda"),
                 torch.empty(B, dtype=torch.int32, device="cuda"))

        def step():
            lla.q8_decode_attn(cfg, table, cache, ctx, bt, now["q"], now["k"], now["v"], ctx,
                               layout="interleaved", out=out, ws=ws)
            lla.page_map(page, ctx, ones, bt, free, nf, B, *t_ids, status=status)
            lla.q8_append(cfg, table, cache, ctx, bt, t_ids[0], t_ids[2], now["k"], now["v"],
                          layout="interleaved", status=status)

        graph = None
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        outs = []
        for i in range(steps):
            for n in "qkv":
                now[n].copy_(torch.stack([x[n][b, int(m) + i] for b, m in enumerate(prompt)]))
            graph.replay() if graph else step()
            outs.append(out.clone())
        k_all, v_all = [], []
        for b in range(B):
            n = int(prompt[b]) + steps
            s = bt[b].long()[torch.arange(n, device="cuda") // page] * page + \
                torch.arange(n, device="cuda") % page
            k_all.append(lla.q8_read(cfg, cache, s))
    torch.cuda.synchronize()
    assert int(status) == 0 and lla.decode_status(ws) == 0
    assert ctx.tolist() == (prompt + steps).tolist()
    assert int(nf) == 48 - sum(-(-(int(m) + steps) // page) for m in prompt)
    t = table.double().cpu().numpy()
    for b in range(B):
        n = int(prompt[b]) + steps
        p = np.arange(n)
        xs = {m: x[m][b, :n].double().cpu().numpy() for m in "qkv"}
        kr = P.rope_rows(xs["k"], t[p, :, 0], t[p, :, 1], "interleaved")
        qr = P.rope_rows(xs["q"], t[p, :, 0], t[p, :, 1], "interleaved")
        # the cache holds the tokens to 2.5 scales: amax < 5 sigma = 5 here, so < 0.1
        assert np.abs(k_all[b][0].double().cpu().numpy() - kr).max() < 0.1
        assert np.abs(k_all[b][1].double().cpu().numpy() - xs["v"]).max() < 0.1
        for i in range(steps):
            m = int(prompt[b]) + i
            for h in range(4):
                want = P.q8_attention(qr[m, h], kr[m, h], xs["v"][m, h], kr[:m, h], xs["v"][:m, h], 0.125)
                # scales of about 4 / 127 with a rounding or a few: elements off by 0.015 rms, scores
                # by 0.125 * 8 * 0.015, outputs of few tokens by as much again: 0.25 is over ten
                # times that, and another token's output is off by about 1
                assert np.abs(outs[i][b, h].double().cpu().numpy() - want).max() < 0.25


@pytest.mark.gpu
def test_two_streams_with_a_workspace_each():
    cfg, page = cfg_of(8, 128), 64
    g = np.random.default_rng(21)
    bt, n_pages = layout_pages(g, [3000, 2500], page)
    cache = random_cache(g, cfg, n_pages, page)
    lens, btd = i32([3000, 2500]), i32(bt)
    q = [torch.randn((2, 8, 128), device="cuda") for _ in range(2)]
    ws = [lla.q8_decode_workspace(cfg, 2, bt.shape[1] * page) for _ in range(2)]
    want = [lla.q8_decode_attn(cfg, None, cache, lens, btd, x, None, None, None) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(lla.q8_decode_attn(cfg, None, cache, lens, btd, q[i], None, None,
                                                  None, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])
