"""Timed cases of the paged 8-bit cache and the operators around it.

Four operators: rotary positions (tables scaled for long contexts, applied to
rows of heads), block tables and slot maps from request lengths, the append that
writes keys and values into an 8-bit cache with one scale per page and head, and
decode attention over that cache.  ``run`` computes each either in its plain form
(elementary torch operations in fp32, angles in fp64) or, with ``own`` set, by the
library's calls.

Definitions, d = head width, rd = rotated dims, P = tokens per page:

  rotary      (y_a, y_b) = (x_a c - x_b s, x_a s + x_b c) on the pairs (i, i + rd/2)
              or (2i, 2i + 1), with (c, s) the table's row at the token's position;
              the gradient is the same with s negated.
  pages       sequence b grows by n[b] tokens (drops -n[b]); it gets the pages that its
              new length needs from the top of the free list, in the order of (b, page).
  append      s = amax / 127 over the tokens written to a page's head; a page that holds
              tokens already keeps its scale, or grows it to max(s, 1.25 old) and rounds
              its codes again; code = round(x / s).
  attention   softmax over the cached tokens and the in-flight one, per head.
"""
import math
import types

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
GROW = 1.25          # least growth of a page's scale
TINY = 1e-30         # a largest value at or below this stores zeros


def _lla():
    import looped_transformer_decode_b200 as lla
    return lla


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # the queries of one decode step of 64 sequences, 16 heads of 128: latency only
        dict(name="rope_decode_64", op="rope", tokens=64, H=16, d=128, d_rope=0, layout="half",
             dtype="fp32", inverse=False, max_pos=4097),
        # a prompt's keys, one third of a fused projection's rows, rotated on half of each head
        dict(name="rope_prompt_32k_partial", op="rope", tokens=32768, H=16, d=128, d_rope=64,
             layout="interleaved", dtype="bf16", inverse=False, max_pos=32769),
        # the gradient of an odd number of rotated rows, the deep loop's heads of 96
        dict(name="rope_backward_d96", op="rope", tokens=4099, H=8, d=96, d_rope=0, layout="half",
             dtype="fp32", inverse=True, max_pos=32768),
        # the table of a context stretched from 4k to 128k positions
        dict(name="rope_table_128k", op="table", max_pos=131072, d=128, kind="yarn", factor=32.0,
             orig_len=4096),
        # one decode step of 256 sequences: one new token each, a page now and then
        dict(name="pages_decode_256", op="pages", B=256, page=16, max_len=4096, grow="one",
             tokens=256, short=False),
        # prompts admitted together, some sequences waiting
        dict(name="pages_prompts_37", op="pages", B=37, page=64, max_len=32768, grow="prompt",
             tokens=100003, short=False),
        # one decode step's keys and values of one loop, 64 sequences
        dict(name="append_decode_64", op="append", B=64, H=16, d=128, d_rope=0, page=16,
             layout="half", dtype="fp32", grow="one", tokens=64),
        # prompts of uneven length written at once
        dict(name="append_prompts_20k", op="append", B=7, H=16, d=128, d_rope=0, page=64,
             layout="half", dtype="bf16", grow="prompt", tokens=20011),
        # the smallest call: one sequence, two heads of 64
        dict(name="attn_tiny", op="attn", B=1, H=2, d=64, d_rope=0, page=16, n=128, ragged=False,
             layout="half", dtype="fp32", self=True),
        # eight sequences of 4096 tokens
        dict(name="attn_8x4k", op="attn", B=8, H=16, d=128, d_rope=0, page=16, n=4096,
             ragged=False, layout="half", dtype="fp32", self=True),
        # the deep loop's shape, uneven lengths up to 32768
        dict(name="attn_ragged_32k_d96", op="attn", B=16, H=8, d=96, d_rope=32, page=64, n=32768,
             ragged=True, layout="interleaved", dtype="bf16", self=True),
        # 256 sequences of 4096 tokens, over the history alone
        dict(name="attn_256x4k", op="attn", B=256, H=16, d=128, d_rope=0, page=64, n=4096,
             ragged=False, layout="half", dtype="bf16", self=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head(rng):
    d = rng.choice([32, 64, 96, 128])
    d_rope = rng.choice([0, 0] + [r for r in (32, 64) if r < d])
    return d, d_rope, rng.choice(["half", "interleaved"]), rng.choice(["fp32", "bf16"])


def draw(rng):
    op = rng.choice(["rope", "rope", "table", "pages", "pages", "append", "append", "attn", "attn",
                     "attn"])
    if op == "rope":
        d, d_rope, layout, dtype = _head(rng)
        H = _log(rng, 1, 32)
        return dict(op=op, tokens=_log(rng, 1, min(65536, (1 << 26) // (H * d))), H=H, d=d,
                    d_rope=d_rope, layout=layout, dtype=dtype, inverse=rng.random() < 0.4,
                    max_pos=_log(rng, 64, 131072))
    if op == "table":
        return dict(op=op, max_pos=_log(rng, 16, 131072), d=rng.choice([32, 64, 96, 128]),
                    kind=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=round(rng.uniform(1.0, 40.0), 2), orig_len=_log(rng, 256, 8192))
    if op == "pages":
        B, page = _log(rng, 1, 2000), rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            return dict(op=op, B=B, page=page, max_len=_log(rng, 128, 16384), grow="one", tokens=B,
                        short=rng.random() < 0.3)
        return dict(op=op, B=B, page=page, max_len=32768, grow="prompt",
                    tokens=_log(rng, max(64, B), 131072), short=rng.random() < 0.3)
    if op == "append":
        d, d_rope, layout, dtype = _head(rng)
        H, page = _log(rng, 1, 32), rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            B = _log(rng, 1, max(1, min(256, (1 << 22) // (H * d * page) * 4)))
            return dict(op=op, B=B, H=H, d=d, d_rope=d_rope, page=page, layout=layout, dtype=dtype,
                        grow="one", tokens=B)
        return dict(op=op, B=_log(rng, 1, 24), H=H, d=d, d_rope=d_rope, page=page, layout=layout,
                    dtype=dtype, grow="prompt", tokens=_log(rng, 64, (1 << 25) // (H * d)))
    d, d_rope, layout, dtype = _head(rng)
    H, page = _log(rng, 1, 32), rng.choice([16, 32, 64, 128])
    n = _log(rng, 1, 65536)
    B = _log(rng, 1, max(1, min(128, (1 << 29) // (n * H * d))))
    return dict(op=op, B=B, H=H, d=d, d_rope=d_rope, page=page, n=n, ragged=rng.random() < 0.7,
                layout=layout, dtype=dtype, self=rng.random() < 0.6)


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device=DEV, dtype=torch.int64)


def _table(max_pos, rd):
    """(cos, sin) rows [max_pos, rd/2, 2] of base 10000, as a program keeps them."""
    th = 10000.0 ** (-torch.arange(rd // 2, device=DEV, dtype=torch.float64) * 2 / rd)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * th
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def _codes(g, shape):
    """Cache codes: values of one normal distribution on 127 steps, chunk by chunk."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        part = flat[a:a + (1 << 27)]
        part.copy_((torch.randn(part.numel(), generator=g, device=DEV, dtype=torch.float32) * 36)
                   .round_().clamp_(-127, 127))
    return out


def _scales(g, shape):
    return torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.25) / 36


def _lengths(case, g):
    """Sequence lengths before and after the call, for pages and append."""
    B, total = case["B"], case["tokens"]
    if case["grow"] == "one":
        top = case.get("max_len", 4096 if case["op"] == "pages" else 512)
        old = _randint(g, 0, max(1, top), B)
        return old, torch.ones_like(old)
    if case["op"] == "pages":
        old = _randint(g, 0, 2000, B) * (_randint(g, 0, 3, B) > 0)
    else:
        old = _randint(g, 0, 300, B) * (_randint(g, 0, 2, B) > 0)
    share = torch.rand(B, generator=g, device=DEV, dtype=torch.float64) + 0.05
    share = share * (_randint(g, 0, 5, B) > 0)            # some sequences wait
    share[0] += 0.2
    new = (share / share.sum() * total).floor().long()
    new[0] += total - new.sum()
    if case["op"] == "pages":
        new = torch.minimum(new, case["max_len"] - old)
    return old, new


def _pages_of(g, used, n_pages, width):
    """Block table of the sequences' pages (-1 behind them) and the list of free pages."""
    perm = torch.randperm(n_pages, generator=g, device=DEV)
    first = torch.cumsum(used, 0) - used
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    bt = torch.where(col < used[:, None], perm[at], -1).int().contiguous()
    n = int(used.sum())
    free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    free[:n_pages - n] = perm[n:].int()
    return bt, free, n_pages - n


def prepare(case, seed):
    g = _gen(seed)
    s = types.SimpleNamespace(case=case, keep={})
    op = case["op"]
    if op == "table":
        s.base = float(torch.rand(1, generator=g, device=DEV)[0] * 9000 + 6000)    # an fp32 value
        return s
    if op == "rope":
        rd = case["d_rope"] or case["d"]
        n = case["tokens"]
        wide = torch.randn((n, 3, case["H"], case["d"]), generator=g, device=DEV)
        s.x = wide.to(DTYPES[case["dtype"]])[:, 1]        # keys inside q, k, v rows
        s.table = _table(case["max_pos"], rd)
        s.positions = _randint(g, 0, case["max_pos"], n).int()
        s.out = torch.empty((n, case["H"], case["d"]), dtype=s.x.dtype, device=DEV)
        return s
    if op == "pages":
        P, B = case["page"], case["B"]
        old, new = _lengths(case, g)
        s.ctx_len, s.n_new = old.int(), new.int()
        width = -(-case["max_len"] // P) + 1
        used = (old + P - 1) // P
        n_pages = B * (-(-(case["max_len"] if case["grow"] == "one" else 2000) // P) + 2)
        n_pages += case["tokens"] // P + 7
        s.bt, s.free, nf = _pages_of(g, used, n_pages, width)
        if case["short"]:
            nf = min(nf, case["tokens"] // (2 * P))           # later sequences are left waiting
        s.n_free = torch.tensor([nf], dtype=torch.int32, device=DEV)
        s.cap = case["tokens"] + 5
        return s
    H, d, P, dt = case["H"], case["d"], case["page"], DTYPES[case["dtype"]]
    rd = case["d_rope"] or d
    if op == "append":
        old, new = _lengths(case, g)
        after = old + new
        used = (after + P - 1) // P
        width = (case["tokens"] + 512) // P + 2
        n_pages = case["B"] * (512 // P + 2) + case["tokens"] // P + 3
        s.bt, _, _ = _pages_of(g, used, n_pages, width)
        s.ctx_len = after.int()
        s.tok_start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)]).int()
        n = int(new.sum())
        b = torch.repeat_interleave(torch.arange(case["B"], device=DEV), new)
        pos = torch.arange(n, device=DEV) - s.tok_start.long()[b] + old[b]
        s.positions = pos.int()
        s.table = _table(int(after.max()) + 1, rd)
        s.k = torch.randn((n, H, d), generator=g, device=DEV).to(dt)
        s.v = torch.randn((n, H, d), generator=g, device=DEV).to(dt)
        s.kc, s.vc = _codes(g, (n_pages, H, P, d)), _codes(g, (n_pages, H, P, d))
        s.ks, s.vs = _scales(g, (n_pages, H)), _scales(g, (n_pages, H))
        # rows read back: the new tokens', and the whole page where each sequence went on
        page = s.bt.long().gather(1, (old // P)[:, None]).clamp(min=0)
        s.rows = torch.cat([s.bt.long()[b, pos // P] * P + pos % P,
                            (page * P + torch.arange(P, device=DEV)).reshape(-1)])
        shape = (s.rows.numel(), H, d)
        s.k_out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        s.v_out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        return s
    B, n = case["B"], case["n"]
    lens = torch.full((B,), n, device=DEV, dtype=torch.int64)
    if case["ragged"]:
        lens = (torch.rand(B, generator=g, device=DEV) ** 2 * n).long()
        lens[0] = n
    s.ctx_len = lens.int()
    used = (lens + P - 1) // P
    n_pages = int(used.sum()) + 2
    s.bt, _, _ = _pages_of(g, used, n_pages, -(-n // P))
    s.kc, s.vc = _codes(g, (n_pages, H, P, d)), _codes(g, (n_pages, H, P, d))
    s.ks, s.vs = _scales(g, (n_pages, H)), _scales(g, (n_pages, H))
    s.table = _table(n + 1, rd)
    s.q_pos = s.ctx_len.clone()
    s.q = torch.randn((B, H, d), generator=g, device=DEV).to(dt)
    s.k = torch.randn((B, H, d), generator=g, device=DEV).to(dt) if case["self"] else None
    s.v = torch.randn((B, H, d), generator=g, device=DEV).to(dt) if case["self"] else None
    s.out = torch.empty((B, H, d), dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------------------- the library's calls

def _cfg(lla, case, base=10000.0):
    return lla.Cfg(T=4, H=case.get("H", 1), d_head=case["d"], r_k=16, r_v=32, rope_base=base,
                   d_rope=case.get("d_rope", 0))


def _run_own(s):
    lla, case = _lla(), s.case
    op = case["op"]
    if op == "pages":
        tok_start, slot, positions = lla.page_map(case["page"], s.ctx_len, s.n_new, s.bt, s.free,
                                                  s.n_free, s.cap)
        back = tok_start[:-1] - tok_start[1:]
        lla.page_map(case["page"], s.ctx_len, back, s.bt, s.free, s.n_free, 0)
        return [tok_start, slot, positions, s.ctx_len, s.bt, s.n_free, s.free]
    if op == "table":
        cfg = _cfg(lla, case, s.base)
        scaling = lla.RopeScaling(case["kind"], case["factor"], case["orig_len"])
        return [lla.rope_table(cfg, case["max_pos"], scaling=scaling)]
    cfg = _cfg(lla, case)
    if op == "rope":
        return [lla.rope_apply(cfg, s.table, s.positions, s.x, layout=case["layout"],
                               inverse=case["inverse"], out=s.out)]
    cache = lla.Q8Cache(s.kc, s.vc, s.ks, s.vs)
    if op == "append":
        lla.q8_append(cfg, s.table, cache, s.ctx_len, s.bt, s.tok_start, s.positions, s.k, s.v,
                      layout=case["layout"])
        lla.q8_read(cfg, cache, s.rows, s.k_out, s.v_out)
        return [s.k_out, s.v_out]
    if "ws" not in s.keep:
        s.keep["ws"] = lla.q8_decode_workspace(cfg, case["B"], s.bt.shape[1] * case["page"])
    return [lla.q8_decode_attn(cfg, s.table, cache, s.ctx_len, s.bt, s.q, s.k, s.v, s.q_pos,
                               layout=case["layout"], out=s.out, ws=s.keep["ws"])]


# ---------------------------------------------------------------------------- plain forms

def _rotate(x, table, positions, layout, inverse=False):
    """x fp32 [n, H, d] rotated at its positions on the table's dims."""
    half = table.shape[1]
    rd = 2 * half
    cs = table[positions.long()]
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sn = -sn
    y = x.clone()
    if layout == "half":
        a, b = x[..., :half], x[..., half:rd]
        y[..., :half] = a * c - b * sn
        y[..., half:rd] = a * sn + b * c
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2] = a * c - b * sn
        y[..., 1:rd:2] = a * sn + b * c
    return y


def _frequencies(case, rd, base):
    """Angles per position, fp64."""
    i = torch.arange(rd // 2, device=DEV, dtype=torch.float64)
    kind, f = case["kind"], case["factor"]
    if kind == "ntk":
        return (base * f ** (rd / (rd - 2))) ** (-2 * i / rd)
    th = base ** (-2 * i / rd)
    if kind == "linear":
        return th / f
    if kind == "yarn":
        def at(turns):
            return rd * math.log(case["orig_len"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo = max(math.floor(at(32.0)), 0)
        hi = min(math.ceil(at(1.0)), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return th * (1 - ramp) + th / f * ramp
    return th


def _plain_pages(s):
    P = s.case["page"]
    old, n_new = s.ctx_len.long(), s.n_new.long()
    limit = s.bt.shape[1] * P
    new = (old + n_new).clamp(min=0)
    fits = new <= limit
    new = torch.where(fits, new, old)
    need = (new + P - 1) // P - (old + P - 1) // P
    count = new - old
    ok = (need.cumsum(0) <= s.n_free) | (need == 0)
    ok &= (count.cumsum(0) <= s.cap) | (count == 0)
    new = torch.where(ok, new, old)
    need, count = need * ok, count * ok
    zero = torch.zeros_like(count[:1])
    tok_start = torch.cat([zero, count.cumsum(0)])
    first = need.cumsum(0) - need
    col = torch.arange(s.bt.shape[1], device=DEV)
    have = (old + P - 1) // P
    k = col - have[:, None]
    mine = (k >= 0) & (k < need[:, None])
    at = (s.n_free.long() - 1 - first[:, None] - k).clamp(0, s.free.numel() - 1)
    bt = torch.where(mine, s.free[at], s.bt)
    i = torch.arange(s.cap, device=DEV)
    b = torch.searchsorted(tok_start, i, right=True) - 1
    live = i < tok_start[-1]
    b = b.clamp(max=old.numel() - 1)
    pos = old[b] + i - tok_start[b]
    pos = torch.where(live, pos, 0)
    slot = torch.where(live, bt[b, pos // P].long() * P + pos % P, -1)
    # the tokens dropped again: every page goes back to where it came from
    gone = (col >= have[:, None]) & (col < have[:, None] + need[:, None])
    bt = torch.where(gone, -1, bt)
    free = s.free.clone()
    back_to = torch.where(gone, at, free.numel())
    free = torch.cat([free, free[:1]]).scatter(0, back_to.reshape(-1),
                                               torch.where(mine, s.free[at], 0).reshape(-1))[:-1]
    return [tok_start.int(), slot, pos.int(), old.int(), bt, s.n_free.clone(), free]


def _plain_append(s):
    case = s.case
    P, H = case["page"], case["H"]
    start = s.tok_start.long()
    count = start[1:] - start[:-1]
    i = torch.arange(s.k.shape[0], device=DEV)
    b = torch.searchsorted(start, i, right=True) - 1
    before = s.ctx_len.long() - count
    at = before[b] + i - start[b]
    page, row = s.bt.long()[b, at // P], at % P
    n_pages = s.ks.shape[0]
    held = torch.zeros(n_pages, dtype=torch.int64, device=DEV)      # tokens held before the call
    held.scatter_reduce_(0, page, (before[b] - at // P * P).clamp(min=0), "amax")
    k = _rotate(s.k.float(), s.table, s.positions, case["layout"])
    v = s.v.float()
    rows = torch.arange(P, device=DEV)
    touched = torch.zeros(n_pages, dtype=torch.bool, device=DEV)
    touched[page] = True
    t = touched.nonzero()[:, 0]
    found = []
    for x, codes, scale, out in ((k, s.kc, s.ks, s.k_out), (v, s.vc, s.vs, s.v_out)):
        amax = torch.zeros((n_pages, H), device=DEV)
        amax.scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        asked = torch.where(amax > TINY, amax / 127, 0.0)
        older = torch.where((held > 0)[:, None], scale, 0.0)
        new = torch.where(asked > older, torch.maximum(asked, older * GROW), older)
        ratio = torch.where(new > 0, older / new, 0.0)[t]
        kept = codes[t].float()
        again = (kept * ratio[:, :, None, None]).round()
        mine = rows < held[t][:, None]
        codes[t] = torch.where(mine[:, None, :, None], again, kept).to(torch.int8)
        scale[t] = new[t]
        inv = torch.where(new > 0, 1 / new, 0.0)[page]
        codes[page, :, row] = (x * inv[:, :, None]).round().clamp(-127, 127).to(torch.int8)
        rp, rr = s.rows // P, s.rows % P
        out.copy_(codes[rp, :, rr].float() * scale[rp][:, :, None])
        found.append(out)
    return found


def _plain_attention(s):
    case = s.case
    P, H, d = case["page"], case["H"], case["d"]
    B = case["B"]
    bt = s.bt.long().clamp(min=0)
    q = _rotate(s.q.float(), s.table, s.q_pos, case["layout"]) / math.sqrt(d)

    def values(codes, scale):
        x = codes[bt].float() * scale[bt][..., None, None]          # [B, pages, H, P, d]
        return x.transpose(1, 2).reshape(B, H, -1, d)

    k = values(s.kc, s.ks)
    score = torch.matmul(k, q[..., None])[..., 0]                    # [B, H, n]
    del k
    dead = torch.arange(score.shape[-1], device=DEV) >= s.ctx_len[:, None]
    score = score.masked_fill(dead[:, None], -math.inf)
    if s.k is not None:
        mine = (q * _rotate(s.k.float(), s.table, s.q_pos, case["layout"])).sum(-1, keepdim=True)
        score = torch.cat([score, mine], -1)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    hist = p[..., :dead.shape[-1]]
    v = values(s.vc, s.vs).masked_fill(dead[:, None, :, None], 0.0)
    o = torch.matmul(hist[..., None, :], v)[..., 0, :]
    if s.k is not None:
        o = o + p[..., -1:] * s.v.float()
    return [(o / torch.where(total > 0, total, 1.0)).to(s.q.dtype)]


def run(state):
    if own:
        return _run_own(state)
    case = state.case
    op = case["op"]
    if op == "table":
        pos = torch.arange(case["max_pos"], device=DEV, dtype=torch.float64)
        ang = pos[:, None] * _frequencies(case, case["d"], state.base)
        return [torch.stack([torch.cos(ang), torch.sin(ang)], -1).float()]
    if op == "rope":
        y = _rotate(state.x.float(), state.table, state.positions, case["layout"], case["inverse"])
        return [y.to(state.x.dtype)]
    if op == "pages":
        return _plain_pages(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ---------------------------------------------------------------------------- cost

def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": case["max_pos"] * case["d"] * 4, "flops": case["max_pos"] * case["d"]}
    size = 4 if case.get("dtype") == "fp32" else 2
    if op == "rope":
        n, H, d = case["tokens"], case["H"], case["d"]
        rd = case["d_rope"] or d
        table = min(n, case["max_pos"]) * rd * 4
        return {"bytes": 2 * n * H * d * size + table + 4 * n, "flops": 3 * n * H * rd}
    if op == "pages":
        n, B, P = case["tokens"], case["B"], case["page"]
        return {"bytes": 12 * n + 20 * B + 8 * (n // P), "flops": 4 * n}
    H, d, P = case["H"], case["d"], case["page"]
    if op == "append":
        n, B = case["tokens"], case["B"]
        new = 2 * n * H * d
        # the tokens in, their codes out, the rows read back as 2-byte values
        return {"bytes": new * size + new + (n + B * P) * H * d * 2 * (1 + 2),
                "flops": new * 4}
    n = case["B"] * case["n"] * ((1 / 3) if case["ragged"] else 1.0)
    rows = case["B"] * H * d * size
    return {"bytes": n * H * d * 2 + n / P * H * 8 + rows * (4 if case["self"] else 2),
            "flops": 4 * n * H * d}


# ---------------------------------------------------------------------------- 64 bits

def _exact_pairs(table_rd, positions):
    """cos and sin in fp64 of the fp32 table's own values: the table is an input."""
    return table_rd.double()[positions.long()]


def _turn(x, cs, layout, sign=1.0):
    """Rotation as complex products: x fp64 [n, H, d], cs fp64 [n, rd/2, 2]."""
    half = cs.shape[1]
    w = torch.complex(cs[..., 0], sign * cs[..., 1])[:, None]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        z = torch.complex(rot[..., :half].contiguous(), rot[..., half:].contiguous()) * w
        rot = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(rot.reshape(*rot.shape[:-1], half, 2).contiguous()) * w
        rot = torch.view_as_real(z).reshape(rot.shape)
    return torch.cat([rot, rest], -1)


def _exact_attention(s, case):
    P, H, d = case["page"], case["H"], case["d"]
    lens = s.ctx_len.tolist()
    cs = _exact_pairs(s.table, s.q_pos)
    q = _turn(s.q.double(), cs, case["layout"])
    k_own = _turn(s.k.double(), cs, case["layout"]) if s.k is not None else None
    out = torch.zeros((case["B"], H, d), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        pages = s.bt[b, :-(-n // P)].long()
        k = (s.kc[pages].double() * s.ks[pages].double()[..., None, None])
        k = k.permute(1, 0, 2, 3).reshape(H, -1, d)[:, :n]
        v = (s.vc[pages].double() * s.vs[pages].double()[..., None, None])
        v = v.permute(1, 0, 2, 3).reshape(H, -1, d)[:, :n]
        if s.k is not None:
            k = torch.cat([k, k_own[b][:, None]], 1)
            v = torch.cat([v, s.v[b].double()[:, None]], 1)
        if k.shape[1]:
            p = torch.softmax((k * q[b][:, None]).sum(-1) / d ** 0.5, -1)
            out[b] = (p[..., None] * v).sum(1)
    return [out]


def _exact_append(s, case):
    """Sequence by sequence and page by page, from the definition."""
    P = case["page"]
    n_seq, start = case["B"], s.tok_start.tolist()
    after = s.ctx_len.tolist()
    k = _turn(s.k.double(), _exact_pairs(s.table, s.positions), case["layout"])
    got = []
    for x, codes, scale in ((k, s.kc, s.ks), (s.v.double(), s.vc, s.vs)):
        value = codes.double() * scale.double()[..., None, None]      # [pages, H, P, d]
        for b in range(n_seq):
            n = start[b + 1] - start[b]
            at = after[b] - n
            t = start[b]
            while t < start[b + 1]:
                off = at % P
                m = min(P - off, start[b + 1] - t)
                page = int(s.bt[b, at // P])
                rows = x[t:t + m].transpose(0, 1)                   # [H, m, d]
                asked = rows.abs().amax((1, 2)) / 127
                older = scale[page].double() if off else torch.zeros_like(asked)
                new = torch.where(asked > older, torch.maximum(asked, older * 1.25), older)
                c = codes[page].double()
                c[:, :off] = torch.round(c[:, :off] * (older / new)[:, None, None])
                c[:, off:off + m] = torch.round(rows / new[:, None, None]).clamp(-127, 127)
                value[page] = c * new[:, None, None]
                t += m
                at += m
        got.append(value[s.rows // P, :, s.rows % P])
    return got


def _exact_table(case, base):
    rd, f = case["d"], case["factor"]
    rows = []
    for i in range(rd // 2):
        inv = math.exp(-2.0 * i / rd * math.log(base))
        if case["kind"] == "linear":
            inv = inv / f
        elif case["kind"] == "ntk":
            inv = math.exp(-2.0 * i / rd * (math.log(base) + rd / (rd - 2) * math.log(f)))
        elif case["kind"] == "yarn":
            def dim(turns):
                return rd / 2 * math.log(case["orig_len"] / (turns * 2 * math.pi)) / math.log(base)
            lo, hi = max(0, math.floor(dim(32))), min(rd - 1, math.ceil(dim(1)))
            part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            inv = inv * (1.0 - part + part / f)
        rows.append(inv)
    ang = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * \
        torch.tensor(rows, dtype=torch.float64, device=DEV)
    return [torch.view_as_real(torch.polar(torch.ones_like(ang), ang))]


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None                                                  # whole numbers only
    s = prepare(case, seed)
    if op == "table":
        return _exact_table(case, s.base)
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return [_turn(s.x.double(), _exact_pairs(s.table, s.positions), case["layout"], sign)]
    if op == "append":
        return _exact_append(s, case)
    return _exact_attention(s, case)
