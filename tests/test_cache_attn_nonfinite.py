"""Infinities and NaN in queries, NaN codes among keys (lidx_cache_attn): a row that takes one in is NaN, the other rows
and heads are as without."""

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_cache_attn import Case, _status_ok

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _check(c, nan, **kw):
    """nan [B,S,Hq]: rows that are NaN.  The others, by the definition, as if the queries were finite."""
    t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
    o, lse = lidx.lidx_cache_attn(*c.args(), q_pos=t(kw.get("q_pos")), topk_indices=t(kw.get("idx")), want_lse=True)
    _status_ok()
    kc = np.where((c.kc & 0x7F) == 0x7F, 0, c.kc).astype(np.uint8)
    ro, rl, so, sl = plain.attention(torch.nan_to_num(c.q, 0.0, 0.0, 0.0), kc, c.vc, c.ks, c.vs, c.table, c.lens, **kw)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    nan = nan & np.isfinite(rl)               # a row that sees no key takes nothing in
    assert np.array_equal(np.isnan(o).all(-1), nan) and np.array_equal(np.isnan(o).any(-1), nan)
    ok = ~nan
    assert (np.abs(o - ro)[ok] <= so[ok]).all()
    seen = ok & np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse)[ok], ~np.isfinite(rl)[ok]) and (np.abs(lse[seen] - rl[seen]) <= sl[seen]).all()


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("S,Hq,Hkv,D,lens", [
    (1, 8, 1, 64, [300, 0, 5]), (1, 32, 1, 128, [9000, 200, 1]), (1, 64, 1, 128, [9000, 0, 130]),
    (1, 256, 2, 80, [700, 0, 128]), (3, 20, 4, 80, [300, 2, 40]), (40, 12, 4, 32, [300, 41, 10])])
@pytest.mark.parametrize("selected", [False, True])
def test_queries(S, Hq, Hkv, D, lens, bad, selected):
    c = Case(S + Hq, 3, S, Hq, Hkv, D, 16, lens)
    rows = np.zeros((3, S, Hq), bool)
    for b, s, h, d in ((0, 0, 1, 0), (0, S - 1, Hq - 1, D - 1), (1, 0, 0, 17), (2, S // 2, Hq // 2, 3)):
        rows[b, s, h] = True
        c.q[b, s, h, d] = bad
    c.q[0, 0, 1, 5], rows[0, 0, 1] = -bad, True
    idx = c.g.integers(-2, max(lens), (3, S, 150)) if selected else None
    _check(c, rows, q_pos=[n - S for n in lens] if S > 1 else None, idx=idx)


@pytest.mark.parametrize("S,Hq,Hkv,D,lens", [
    (1, 8, 2, 64, [300, 200]), (1, 32, 1, 128, [9000, 200]), (1, 64, 1, 128, [9000, 130]), (1, 256, 2, 80, [700, 128]),
    (16, 2, 1, 64, [2000, 30]), (40, 12, 4, 32, [300, 41])])
def test_keys(S, Hq, Hkv, D, lens):
    c = Case(S + Hq + 1, 2, S, Hq, Hkv, D, 32, lens)
    pos = [n - S for n in lens] if S > 1 else None
    rows = np.zeros((2, S, Hq), bool)
    G = Hq // Hkv
    t = lens[0] - 1 - S // 2
    c.kc[c.table[0, t // 32], Hkv - 1, t % 32, D // 2] = 0xFF
    rows[0, (S - 1 - S // 2 if S > 1 else 0):, (Hkv - 1) * G:] = True
    _check(c, rows, q_pos=pos)
    idx = c.g.integers(0, t, (2, S, 60))
    idx[0, :, 30] = t
    _check(c, rows, q_pos=pos, idx=idx)


@pytest.mark.parametrize("what", ["q", "q inf", "k"])
@pytest.mark.parametrize("Hq,n", [(8, 300), (32, 300), (64, 300), (128, 300), (16, 20000), (32, 20000), (48, 20000), (80, 20000)])
def test_log_sum_exp_of_nan_rows(Hq, n, what):
    """NaN rows say so: -inf is for rows that see no key.  Short rows and rows joined from parts, early keys and late ones."""
    c = Case(Hq + n, 4, 1, Hq, 1, 64, 64, [n, n, 0, n])
    nan = np.zeros((4, 1, Hq), bool)
    if what == "k":
        for b, t in ((0, 3), (1, n - 1)):
            c.kc[c.table[b, t // 64], 0, t % 64, 11] = 0x7F
        nan[:2] = True
    else:
        c.q[0, 0, 2, 7] = c.q[3, 0, Hq - 1, 0] = c.q[2, 0, 1, 0] = NAN if what == "q" else INF
        nan[0, 0, 2] = nan[3, 0, Hq - 1] = True
    idx = np.stack([np.concatenate([c.g.permutation(n - 2)[:200], [3, n - 1]]) for _ in range(4)])[:, None]
    for given in (None, torch.from_numpy(idx.astype(np.int32)).to(DEV)):
        o, lse = lidx.lidx_cache_attn(*c.args(), topk_indices=given, want_lse=True)
        _status_ok()
        o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
        assert np.array_equal(np.isnan(lse), nan) and np.array_equal(np.isnan(o).all(-1), nan)
        assert np.isneginf(lse[2]).all() and np.isfinite(lse[~nan & (c.lens > 0)[:, None, None]]).all()
