"""Paged 8-bit cache and the operators around it, float64 NumPy.

Written from the definitions: rotary frequencies and rows, growing and shrinking
sequences page by page, quantised appends, and attention over dequantised rows.
"""
from __future__ import annotations

import math

import numpy as np

PAGE_RANGE, PAGES_SHORT, CTX_RANGE = 16, 32, 2


# ---------------------------------------------------------------- rotary positions

def rope_angles(rd: int, base: float, kind: str = "none", factor: float = 1.0, orig_len: int = 1,
                beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    """Angle per position of each of the rd/2 pairs."""
    i = np.arange(rd // 2, dtype=np.float64)
    if kind == "ntk":
        return np.power(base * factor ** (rd / (rd - 2.0)), -2 * i / rd)
    th = np.power(float(base), -2 * i / rd)
    if kind == "linear":
        return th / factor
    if kind == "yarn":
        def at(turns):
            return rd * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(base))
        lo = max(math.floor(at(beta_fast)), 0)
        hi = min(math.ceil(at(beta_slow)), rd - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return th * (1 - ramp) + th / factor * ramp
    return th


def rope_rows(x, cos, sin, layout: str, inverse: bool = False) -> np.ndarray:
    """x [n, H, d] rotated; cos, sin [n, rd/2]."""
    half = cos.shape[-1]
    rd = 2 * half
    y = np.array(x, dtype=np.float64)
    ia = np.arange(half) if layout == "half" else 2 * np.arange(half)
    ib = ia + half if layout == "half" else ia + 1
    c = np.asarray(cos, np.float64)[:, None]
    s = np.asarray(sin, np.float64)[:, None] * (-1 if inverse else 1)
    a, b = np.array(x[..., ia], np.float64), np.array(x[..., ib], np.float64)
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    assert rd <= y.shape[-1]
    return y


# ---------------------------------------------------------------- pages

def page_map(page, ctx_len, n_new, block_table, free_list, n_free, tok_cap):
    """One call, sequence by sequence.  Returns new state and the token lists."""
    ctx = [int(x) for x in ctx_len]
    bt = np.array(block_table, copy=True)
    n_pages, limit = len(free_list), bt.shape[1] * page
    fl, nf, status = [int(x) for x in free_list], int(n_free), 0
    if nf < 0 or nf > n_pages:
        status |= PAGE_RANGE
        nf = min(max(nf, 0), n_pages)
    B = len(ctx)
    grow = []
    back = []
    for b in range(B):
        old, new = ctx[b], ctx[b] + int(n_new[b])
        if old < 0 or old > limit:
            status |= CTX_RANGE
            continue
        new = max(new, 0)
        if new > limit:
            status |= CTX_RANGE
            continue
        if new < old:
            for j in range(-(-new // page), -(-old // page)):
                p = int(bt[b, j])
                if not 0 <= p < n_pages:
                    status |= PAGE_RANGE
                    p = -1
                back.append(p)
                bt[b, j] = -1
            ctx[b] = new
        elif new > old:
            grow.append((b, new))
    for p in reversed(back):
        if nf < n_pages:
            fl[nf] = p
            nf += 1
        else:
            status |= PAGE_RANGE
    top = nf
    asked_pages = asked_toks = 0
    counts = [0] * B
    for b, new in grow:
        have = -(-ctx[b] // page)
        need = -(-new // page) - have
        asked_pages += need
        asked_toks += new - ctx[b]
        if (need and asked_pages > top) or asked_toks > tok_cap:
            status |= PAGES_SHORT
            continue
        for j in range(need):
            nf -= 1
            p = fl[nf]
            if not 0 <= p < n_pages:
                status |= PAGE_RANGE
                p = -1
            bt[b, have + j] = p
        counts[b] = new - ctx[b]
        ctx[b] = new
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    slot, pos = np.full(tok_cap, -1, np.int64), np.zeros(tok_cap, np.int64)
    for b in range(B):
        for i in range(counts[b]):
            at = ctx[b] - counts[b] + i
            p = int(bt[b, at // page])
            if not 0 <= p < n_pages:
                status |= PAGE_RANGE
            slot[start[b] + i] = p * page + at % page if 0 <= p < n_pages else -1
            pos[start[b] + i] = at
    return dict(ctx_len=np.array(ctx, np.int64), block_table=bt, free_list=np.array(fl, np.int64),
                n_free=nf, tok_start=start, slot=slot, positions=pos, status=status)


# ---------------------------------------------------------------- 8-bit cache

GROW, TINY = 1.25, 1e-30


def q8_append(codes, scale, block_table, ctx_len, tok_start, x):
    """One of the two caches after an append: codes float64 [pages, H, P, d] before rounding of
    the rows written (their real-valued code), scale [pages, H], and which rows were written
    anew (1) or rounded again (2)."""
    P = codes.shape[2]
    codes, scale = np.array(codes, np.float64), np.array(scale, np.float64)
    kind = np.zeros((codes.shape[0], codes.shape[1], P), np.int8)
    for b in range(len(ctx_len)):
        s, e = int(tok_start[b]), int(tok_start[b + 1])
        at = int(ctx_len[b]) - (e - s)
        while s < e:
            page, off = int(block_table[b][at // P]), at % P
            m = min(P - off, e - s)
            rows = np.moveaxis(np.asarray(x[s:s + m], np.float64), 0, 1)     # [H, m, d]
            amax = np.abs(rows).max((1, 2))
            for h in range(codes.shape[1]):
                asked = amax[h] / 127 if amax[h] > TINY else 0.0
                old = scale[page, h] if off else 0.0
                new = max(asked, GROW * old) if asked > old else old
                if off and new > old:
                    codes[page, h, :off] *= old / new
                    kind[page, h, :off] = 2
                codes[page, h, off:off + m] = rows[h] / new if new > 0 else 0.0
                kind[page, h, off:off + m] = 1
                scale[page, h] = new
            s, at = s + m, at + m
    return codes, scale, kind


def q8_attention(q, k_self, v_self, k, v, sm_scale):
    """One head: q [d] rotated, k, v [n, d] dequantised, the in-flight row or None."""
    if k_self is not None:
        k, v = np.concatenate([k, k_self[None]]), np.concatenate([v, v_self[None]])
    if not len(k):
        return np.zeros_like(q)
    s = k @ q * sm_scale
    p = np.exp(s - s.max())
    return (p / p.sum()) @ v
