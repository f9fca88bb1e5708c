"""Rotated rows and appended codes, bit by bit against elementary fp32 operations.

Rotation rounds every product and sum, a page's scale is amax * fp32(1 / 127), a code the nearest
integer of value * fp32(1 / scale), an earlier code of code * fp32(older / scale): torch's
elementwise kernels do the same roundings one by one, so nothing may differ.
"""
from __future__ import annotations

import pytest
import torch

import looped_transformer_decode_b200 as lla


def rotated(x, table, pos, layout):
    half = table.shape[1]
    c, s = (t[:, None] for t in table[pos.long()].unbind(-1))
    y = x.float().clone()
    at = torch.arange(half, device=x.device)
    ia, ib = (at, at + half) if layout == "half" else (2 * at, 2 * at + 1)
    a, b = y[..., ia], y[..., ib]
    p, q = a * c, b * s
    r, t = a * s, b * c
    y[..., ia], y[..., ib] = p - q, r + t
    return y


def appended(codes, scale, bt, after, start, x):
    """codes int8, scale fp32 after the append of x fp32, page by page."""
    codes, scale = codes.clone(), scale.clone()
    per = torch.tensor(1 / 127, device=x.device)
    P = codes.shape[2]
    for b in range(len(after)):
        t, e = start[b], start[b + 1]
        at = after[b] - (e - t)
        while t < e:
            page, off = bt[b][at // P], at % P
            m = min(P - off, e - t)
            rows = x[t:t + m].transpose(0, 1)
            asked = rows.abs().amax((1, 2)) * per
            older = scale[page] if off else torch.zeros_like(asked)
            now = torch.where(asked > older, torch.maximum(asked, older * 1.25), older)
            again = (codes[page, :, :off].float() * (older / now)[:, None, None]).round()
            codes[page, :, :off] = again.to(torch.int8)
            codes[page, :, off:off + m] = (rows * (1.0 / now)[:, None, None]).round().to(torch.int8)
            scale[page] = now
            t, at = t + m, at + m
    return codes, scale


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page,H,d,d_rope,layout,old,new", [
    (64, 16, 128, 0, "half", [0, 100, 7], [900, 64, 1300]),
    (128, 5, 32, 0, "interleaved", [0, 17], [2000, 1500]),
    (16, 3, 96, 64, "half", [0, 5, 31], [700, 3, 900]),
    (32, 8, 64, 32, "interleaved", [20] * 40, [1, 2] * 20)])
def test_codes_and_scales_equal_elementary_operations(dtype, page, H, d, d_rope, layout, old, new):
    """bf16 values against a scale from a bf16 maximum: quotients at half a step are common."""
    g = torch.Generator(device="cuda").manual_seed(d + page)
    cfg = lla.Cfg(4, H, d, 16, 32, d_rope=d_rope)
    after = [o + n for o, n in zip(old, new)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    used = [-(-n // page) for n in after]
    order = torch.randperm(sum(used), generator=g, device="cuda").tolist()
    width = max(used)
    bt, at = [], 0
    for m in used:
        bt.append(order[at:at + m] + [-1] * (width - m))
        at += m
    shape = (sum(used), H, page, d)
    cache = lla.q8_cache_alloc(cfg, shape[0], page)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_(torch.randint(-127, 128, shape, generator=g, device="cuda"))
        scale.copy_(torch.rand(shape[:2], generator=g, device="cuda") * 0.03 + 0.01)
    k, v = (torch.randn((start[-1], H, d), generator=g, device="cuda").to(dtype) for _ in "kv")
    pos = torch.cat([torch.arange(o, o + n) for o, n in zip(old, new)]).int().cuda()
    table = lla.rope_table(cfg, max(after))
    want = [appended(cache.k, cache.k_scale, bt, after, start, rotated(k, table, pos, layout)),
            appended(cache.v, cache.v_scale, bt, after, start, v.float())]
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (after, bt, start)]
    lla.q8_append(cfg, table, cache, *ints, pos, k, v, layout=layout)
    for (codes, scale), (c, s) in zip(want, ((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert torch.equal(scale, s)
        assert torch.equal(codes, c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,H,d,d_rope", [(65, 3, 96, 0), (4000, 16, 128, 64)])
def test_rotated_rows_equal_elementary_operations(dtype, layout, n, H, d, d_rope):
    g = torch.Generator(device="cuda").manual_seed(n)
    cfg = lla.Cfg(4, H, d, 16, 32, d_rope=d_rope)
    table = lla.rope_table(cfg, 5000)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((n, H, d), generator=g, device="cuda").to(dtype)
    got = lla.rope_apply(cfg, table, pos, x, layout=layout)
    assert torch.equal(got, rotated(x, table, pos, layout).to(dtype))
