"""Attention over the paged 4-bit cache, every output against a bound of its own row.

plain.attention's slack counts the rounding of small weights once, for the largest value.  What every key adds: with the
scores' softmax p and a page's value scale g, the products are formed from weights p g, scaled so that a tile's largest is 2^8.
They are held as e4m3 hi + lo, off by 2^-8 of the weight or by 2^-10, whichever is larger (half the step of lo's
subnormals), and 2^-10 is 2^-18 of the tile's largest, which is at most the row's.  So beyond the 2^-8 that the slack has, an
output dim is off by at most
    2^-18 max_s(p_s g_s) sum_t |v_t| / g_t
over the keys t that the row sees, as often as it lists them.  Ids out of range are no keys and add nothing."""

import numpy as np
import pytest
import torch

import plain
import plain4
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_cache4_attn import DEV, Case


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def small_weights(c, q_pos, ratio, idx):
    """The bound above, [B,S,Hq,D], and how many keys each row sees [B,S]."""
    B, S, Hq, D = c.q.shape
    P, Hkv = c.vs.shape
    G, out, keys = Hq // Hkv, np.zeros((B, S, Hq, D)), np.zeros((B, S), int)
    q = c.q.double().numpy()
    for b in range(B):
        n = int(min(max(int(c.lens[b]), 0), c.table.shape[1] * c.page))
        for s in range(S):
            end = plain.row_end(n, s, None if q_pos is None else int(q_pos[b]), ratio)
            t = np.arange(end) if idx is None else np.asarray(idx[b, s], np.int64)
            t = t[(t >= 0) & (t < end)]
            pid = c.table[b, t // c.page].astype(np.int64)
            t, pid = t[(pid >= 0) & (pid < P)], pid[(pid >= 0) & (pid < P)]
            keys[b, s] = len(t)
            if len(t) == 0:
                continue
            for h in range(Hkv):
                at = (pid, h, t % c.page)
                k = plain4.numbers(c.kc[at], c.ke[at]) * c.ks[pid, h].astype(np.float64)[:, None]
                rows = slice(h * G, (h + 1) * G)
                x = D ** -0.5 * (q[b, s, rows] @ k.T)
                p = np.exp(x - x.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                top = (p * c.vs[pid, h].astype(np.float64)).max(1, keepdims=True)
                out[b, s, rows] = 2.0 ** -18 * top * np.abs(plain4.numbers(c.vc[at], c.ve[at])).sum(0)
    return out, keys


def want(c, q_pos, ratio, idx):
    ro, rl, so, sl = plain.attention(c.q, plain4.as_8(c.kc, c.ke), plain4.as_8(c.vc, c.ve), c.ks * 32, c.vs * 32, c.table, c.lens,
                                     q_pos, ratio, idx)
    more, keys = small_weights(c, q_pos, ratio, idx)
    return ro, rl, so + more, sl, keys


def selected(S, Hq, Hkv, D, page, lens, topk, ratio, causal):
    c = Case(S * 11 + topk, len(lens), S, Hq, Hkv, D, page, lens)
    idx = c.g.integers(-3, max(lens) + 40, (len(lens), S, topk))  # many out of range, some twice
    idx[0, 0, 0], idx[0, 0, topk // 2 + 1:] = 0, -1
    if S > 1:
        idx[0, -1] = 2 ** 31 - 1                                  # a row that sees nothing
        idx[-1, 1, :] = np.resize(idx[-1, 1, :max(1, topk // 4)], topk)  # keys listed four times
    return c, [n * ratio - S for n in lens] if causal else None, ratio if causal else 1, idx


def dense(S, Hq, Hkv, D, page, lens, ratio):
    return Case(S * 13 + Hq, len(lens), S, Hq, Hkv, D, page, lens), [n * ratio - S for n in lens], ratio, None


SELECTED = [
    (1, 64, 1, 128, 64, [500, 3, 0], 130, 1),
    (1, 8, 2, 80, 16, [300], 1, 1),
    (3, 20, 4, 64, 32, [200, 40], 37, 1),
    (50, 16, 1, 128, 64, [100], 64, 4),
    (4, 128, 1, 128, 128, [400], 256, 1),
    (6, 100, 1, 48, 16, [90, 60], 129, 1),
    (3, 30, 1, 16, 16, [500], 300, 1),
    (2, 6, 2, 112, 32, [260, 700], 400, 1),
    (9, 33, 1, 96, 16, [64], 33, 1),
]
DENSE = [
    (1, 8, 2, 64, 16, [1, 130], 1),
    (5, 20, 4, 80, 32, [77, 300, 0], 1),
    (40, 12, 4, 32, 16, [300, 41], 1),
    (37, 16, 1, 128, 64, [9], 4),
    (9, 128, 1, 64, 64, [200], 1),
    (130, 1, 1, 16, 16, [130], 1),
    (90, 8, 2, 80, 16, [200, 0, 100], 1),  # pages widened first
]
CASES = [("selected", c, causal) for c in SELECTED for causal in (False, True)] + [("dense", c, True) for c in DENSE]


def make(kind, c, causal):
    return selected(*c, causal) if kind == "selected" else dense(*c)


@pytest.mark.parametrize("kind,c,causal", CASES)
def test_the_bounds_tell_rows_apart(kind, c, causal):
    """What the bounds are worth: of the outputs that are not zero, few are within them of zero."""
    case, q_pos, ratio, idx = make(kind, c, causal)
    ro, _, tol, _, keys = want(case, q_pos, ratio, idx)
    some = (ro != 0) & (keys > 0)[..., None, None]
    assert some.any() and np.mean(np.abs(ro[some]) <= tol[some]) < 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("kind,c,causal", CASES)
def test_rows(kind, c, causal):
    case, q_pos, ratio, idx = make(kind, c, causal)
    ro, rl, tol, sl, keys = want(case, q_pos, ratio, idx)
    t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
    kw = dict(q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx), want_lse=True)
    o, lse = lidx.lidx_cache4_attn(*case.args(), **kw)
    o8, lse8 = lidx.lidx_cache_attn(*case.args8(), **kw)
    torch.cuda.synchronize()
    assert lidx.lidx_device_status() == 0
    for got, got_l in ((o, lse), (o8, lse8)):  # the 8-bit call on the same numbers, too
        got, got_l = got.double().cpu().numpy(), got_l.double().cpu().numpy()
        assert (got[keys == 0] == 0).all() and np.isneginf(got_l[keys == 0]).all()
        err = np.abs(got - ro)
        assert (err <= tol).all(), f"{np.max(err - tol):.3e} over, at {np.argwhere(~(err <= tol))[:3]}"
        some = keys > 0
        assert (np.abs(got_l[some] - rl[some]) <= sl[some]).all()
