"""NaN codes among cached values (lidx_cache_attn): an output element is NaN if its row sees a key whose value is NaN in its
dim.  Nothing else is, except that in a causal call over all keys the dim may be NaN in the 127 tokens before the first
that sees the key.  The log-sum-exp does not change."""

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_cache_attn import Case, _status_ok

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _put(c, b, t, h, dims, code=0x7F):
    c.vc[c.table[b, t // c.page], h, t % c.page, dims] = code


def _check(c, bad, q_pos=None, ratio=1, idx=None):
    """bad: (sequence, key, kv head, dims) of NaN values.  Everywhere else the output is that of the cache with zeros there."""
    kw = dict(q_pos=q_pos, ratio=ratio, idx=idx)
    args = lambda: (c.q, c.kc, c.vc, c.ks, c.vs, c.table, c.lens)
    for at in bad:
        _put(c, *at, code=0)
    ro, rl, so, sl = plain.attention(*args(), **kw)
    for i, at in enumerate(bad):
        _put(c, *at, code=0x7F if i % 2 else 0xFF)
    must = np.isnan(plain.attention(*args(), **kw)[0])
    may = must.copy()                                # in a causal call: 127 tokens earlier
    if q_pos is not None and idx is None:
        for s in range(may.shape[1]):
            may[:, s] = must[:, s:s + 128].any(1)
    t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
    o, lse = lidx.lidx_cache_attn(*c.args(), q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx), want_lse=True)
    _status_ok()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    nan = np.isnan(o)
    assert must.any()
    assert nan[must].all(), f"{(~nan)[must].sum()} of {must.sum()} are not NaN"
    assert not nan[~may].any(), f"{nan[~may].sum()} are NaN that may not be"
    assert (np.abs(o - ro)[~nan] <= so[~nan]).all()
    seen = np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), ~seen) and (np.abs(lse[seen] - rl[seen]) <= sl[seen]).all()


@pytest.mark.parametrize("S,Hq,Hkv,D,page,lens,ratio", [
    (4, 8, 2, 64, 16, [40, 300], 1),        # 16 rows a unit
    (5, 20, 4, 80, 32, [77, 300], 1),       # 25
    (16, 2, 1, 128, 64, [2000], 1),         # 32, units cut between CTAs
    (33, 4, 4, 128, 64, [200], 1),          # 33
    (12, 5, 1, 112, 16, [130], 1),          # 60: laid out twice
    (40, 12, 4, 32, 16, [300, 41], 1),      # 120, the last unit with fewer
    (128, 2, 2, 128, 128, [3000, 128], 1),  # 128, several units, many tiles
    (37, 16, 1, 128, 64, [9], 4),           # compressed keys
    (200, 8, 1, 64, 64, [170], 1),          # more queries than keys
])
def test_causal_rows(S, Hq, Hkv, D, page, lens, ratio):
    c = Case(S + D, len(lens), S, Hq, Hkv, D, page, lens)
    pos = [n * ratio - S for n in lens]
    last = Hkv - 1
    # in the last key alone
    _check(Case(S + D, len(lens), S, Hq, Hkv, D, page, lens), [(0, lens[0] - 1, last, slice(0, 1))], pos, ratio)
    # in several dims and keys, and then in the first, too
    n = lens[0]
    bad = [(0, n - 1, last, slice(D - 3, D)), (0, max(0, n - 1 - S // (2 * ratio)), 0, slice(1, 2))]
    if len(lens) > 1:
        bad.append((1, lens[1] - 2, last, slice(5, 6)))
    _check(c, bad, pos, ratio)
    _check(c, bad + [(0, 0, 0, slice(7, 8))], pos, ratio)


def test_many_units():
    """Many units of a CTA behind each other, NaN in some: it does not go from one to the next."""
    lens = [64 + 3 * i for i in range(60)]
    S = 16
    c = Case(3, len(lens), S, 8, 8, 64, 16, lens)
    bad = [(b, lens[b] - 1 - b % 5, b % 8, slice(b % 64, b % 64 + 1)) for b in range(0, 60, 7)]
    _check(c, bad, [n - S for n in lens])
    S = 128
    c = Case(4, len(lens), S, 8, 8, 64, 16, lens)
    _check(c, bad, [n - S for n in lens])


@pytest.mark.parametrize("Hq", [8, 32, 48, 128])
def test_single_tokens_and_selected_keys(Hq):
    c = Case(Hq, 3, 1, Hq, 1, 128, 64, [300, 129, 77])
    bad = [(0, 299, 0, slice(3, 4)), (1, 0, 0, slice(9, 12))]
    _check(c, bad)
    c = Case(Hq, 3, 3, Hq, 1, 128, 64, [300, 129, 77])  # all keys for every token
    _check(c, bad)
    c = Case(Hq, 3, 2, Hq, 1, 128, 64, [300, 129, 77])
    idx = c.g.integers(1, 290, (3, 2, 40))
    idx[0, 1, 17] = 299                     # one row of the two lists the key
    idx[1, 0, 0] = 0
    _check(c, bad, idx=idx)
