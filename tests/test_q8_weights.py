"""8-bit decode attention where the weights of a head differ by many orders of magnitude.

Tolerance, from the probabilities: with p the softmax, the output is off by at most
  sum_j p_j |v_j| * (2 ds + r 2^-24)
ds being the largest error of a score (fp32 sums of d + 8 terms, each element of the query held to
2^-24 of the largest of its 16 neighbours, of 12 in heads of 96) and r the roundings of a token's
contribution: one sum per 16 tokens, one rescale per 32, and 80 for the exponential, the products
and the merges.  No term depends on values that have no weight, and nothing is lost beside a heavy
token.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import looped_transformer_decode_b200 as lla


def attend(kc, vc, ks, vs, q, page, dtype=torch.float32, sm_scale=1.0):
    """Codes [n, d], scales [pages], q [d] of one sequence and head: (got, want, tolerance)."""
    n, d = kc.shape
    pages = -(-n // page)
    cfg = lla.Cfg(4, 1, d, 16, 32, sm_scale=sm_scale)
    cache = lla.q8_cache_alloc(cfg, pages, page)
    for codes, scale, c, s in ((cache.k, cache.k_scale, kc, ks), (cache.v, cache.v_scale, vc, vs)):
        padded = np.zeros((pages * page, d), np.int8)
        padded[:n] = c
        codes.copy_(torch.from_numpy(padded.reshape(pages, 1, page, d)))
        scale.copy_(torch.from_numpy(np.asarray(s, np.float32)[:, None]))
    qt = torch.from_numpy(np.asarray(q, np.float64)).to(dtype).cuda().view(1, 1, d)
    bt = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = lla.q8_decode_attn(cfg, None, cache, lens, bt, qt, None, None, None)
    at = np.arange(n) // page
    k = kc.astype(np.float64) * np.asarray(ks, np.float32).astype(np.float64)[at, None]
    v = vc.astype(np.float64) * np.asarray(vs, np.float32).astype(np.float64)[at, None]
    q = qt.double().cpu().numpy().reshape(d)
    s = k @ q * sm_scale
    p = np.exp(s - s.max())
    p /= p.sum()
    top = np.abs(q).reshape(-1, 12 if d == 96 else 16)
    top = np.broadcast_to(top.max(1, keepdims=True), top.shape).reshape(d)
    ds = sm_scale * 2.0 ** -24 * ((d + 8) * (np.abs(k) @ np.abs(q)).max() + (np.abs(k) @ top).max())
    r = n / 16 + n / 32 + 80
    want = p @ v
    tol = (p @ np.abs(v)) * (2 * ds + r * 2.0 ** -24) + torch.finfo(dtype).eps / 2 * np.abs(want)
    return got.double().cpu().numpy().reshape(d), want, tol


def codes_of(g, shape):
    return np.clip(np.round(g.standard_normal(shape) * 36), -127, 127).astype(np.int8)


@pytest.mark.gpu
@pytest.mark.parametrize("d,page", [(128, 16), (96, 64), (64, 32), (32, 128)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("ratio", [1e4, 1e6, 1e8])
def test_a_page_of_large_values_without_weight(d, page, where, ratio):
    """Its scores lie 80 below the rest's: e^-80 * 1e8 is nothing, and takes nothing with it."""
    n = 2048
    g = np.random.default_rng(d)
    kc, vc = np.zeros((n, d), np.int8), codes_of(g, (n, d))
    kc[:, 1] = codes_of(g, n) // 8
    heavy = {"first": 0, "middle": n // page // 2, "last": n // page - 1}[where]
    kc[heavy * page:(heavy + 1) * page, 0] = -100
    ks = np.full(n // page, 1 / 127)
    vs = np.full(n // page, 1 / 36)
    vs[heavy] *= ratio
    q = np.zeros(d)
    q[0], q[1] = 80 * 1.27, 1.0
    got, want, tol = attend(kc, vc, ks, vs, q, page)
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,n", [(128, 64, 4096), (96, 16, 512), (64, 16, 65536), (32, 32, 8192)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("sink", [0.9, 0.999, 1 - 1e-6])
def test_a_heavy_token_of_value_zero(d, page, n, where, sink):
    """The output is what the light tokens give, each of weight (1 - sink) / n, down to 2^-36."""
    g = np.random.default_rng(n)
    kc, vc = np.zeros((n, d), np.int8), codes_of(g, (n, d))
    kc[:, 1] = codes_of(g, n) // 8
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[where]
    kc[at], vc[at] = 0, 0
    kc[at, 0] = 127
    ks, vs = np.full(n // page, 1 / 127), np.full(n // page, 1 / 36)
    q = np.zeros(d)
    q[1] = 1.0
    light = np.exp(kc[:, 1] / 127.0).sum() - 1
    q[0] = np.log(sink / (1 - sink) * light)
    got, want, tol = attend(kc, vc, ks, vs, q, page)
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,dtype", [(128, 32, torch.float32), (96, 32, torch.bfloat16),
                                          (64, 64, torch.float32), (32, 16, torch.float32)])
def test_scores_that_rise_to_the_end_and_fall(d, page, dtype):
    """Every tile brings a new largest score, or none does."""
    n = 3008
    g = np.random.default_rng(d)
    for sign in (1, -1):
        kc, vc = np.zeros((n, d), np.int8), codes_of(g, (n, d))
        kc[:, 0] = np.linspace(-127, 127, n).astype(np.int8) * sign
        ks = np.full(n // page, 1 / 127)
        vs = np.exp(g.standard_normal(n // page) * 2) / 36
        q = np.zeros(d)
        q[0] = 30.0
        got, want, tol = attend(kc, vc, ks, vs, q, page, dtype)
        assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,dtype", [(128, 16, torch.float32), (96, 64, torch.float32),
                                          (64, 32, torch.bfloat16), (32, 128, torch.float32)])
@pytest.mark.parametrize("outlier", [30.0, 1e4, -1e7])
def test_a_query_with_an_outlier(d, page, dtype, outlier):
    """One element far above the rest, among 16 (or 12) dims where the keys are zero: the other
    dims decide, and keep all their bits."""
    n, group = 1000, 12 if d == 96 else 16
    g = np.random.default_rng(d)
    kc, vc = codes_of(g, (n, d)), codes_of(g, (n, d))
    kc[:, group:2 * group] = 0
    ks, vs = np.full(-(-n // page), 1 / 36), np.full(-(-n // page), 1 / 36)
    q = g.standard_normal(d)
    q[group + 3] = outlier
    got, want, tol = attend(kc, vc, ks, vs, q, page, dtype, sm_scale=0.25)
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()
