"""Attention over the 4-bit cache with tables so wide that the sequences' pages, had the table as many as it has places, would
take more than 2 GiB in 8 bits: such calls of many rows widen their tiles as they read them, several query tiles a sequence,
where calls with a narrow table widen the pages once.  Both are within the bounds of the definition."""

import numpy as np
import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_cache4_attn import DEV
from test_cache4_attn_rows import dense, selected, want


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def widen_table(c):
    """Places behind the sequences' ends, up to 2 GiB of pages and one more; what they hold is never read."""
    B, MP = c.table.shape
    Hkv = c.vs.shape[1]
    places = (1 << 31) // (2 * B * Hkv * c.page * c.D) + 1
    table = np.full((B, places), 2 ** 31 - 1, np.int32)
    table[:, :MP] = c.table
    return table


def bytes_of(c, MP, topk=0):
    B, S, Hq, D = c.q.shape
    return lidx.lidx_cache4_attn_workspace_bytes(B, S, Hq, c.vs.shape[1], D, c.page, MP, topk)


CASES = [
    ("dense", (130, 8, 1, 128, 128, [700], 1)),         # 8 heads: 16 tokens a tile, nine tiles
    ("dense", (70, 12, 2, 128, 64, [300, 0, 129], 1)),  # 6 heads: tiles that tokens do not fill
    ("dense", (300, 1, 1, 96, 128, [513, 20], 1)),      # compressed to one head
    ("dense", (90, 128, 1, 64, 128, [40], 4)),          # a token a tile, first rows without a key
    ("dense", (33, 16, 4, 80, 64, [200, 31], 1)),
    ("selected", (90, 8, 2, 128, 64, [200, 70], 40, 1)),
    ("selected", (70, 64, 1, 128, 128, [300], 130, 1)),
    ("selected", (60, 100, 1, 48, 128, [90], 64, 1)),
]


@pytest.mark.parametrize("kind,c", CASES)
def test_which_calls_take_a_copy(kind, c):
    case = dense(*c)[0] if kind == "dense" else selected(*c, True)[0]
    topk = 0 if kind == "dense" else c[6]
    MP, wide = case.table.shape[1], widen_table(case).shape[1]
    B, S, Hq, D = case.q.shape
    Hkv = case.vs.shape[1]
    parts = lidx.lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk)
    assert bytes_of(case, MP, topk) >= parts + 2 * B * MP * case.page * Hkv * D
    assert bytes_of(case, wide, topk) == parts


@pytest.mark.gpu
@pytest.mark.parametrize("kind,c", CASES)
def test_wide_tables(kind, c):
    case, q_pos, ratio, idx = dense(*c) if kind == "dense" else selected(*c, True)
    ro, rl, tol, sl, keys = want(case, q_pos, ratio, idx)
    t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
    kw = dict(q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx), want_lse=True)
    args = case.args()
    for table in (t(widen_table(case)), args[7]):
        o, lse = lidx.lidx_cache4_attn(*args[:7], table, args[8], **kw)
        torch.cuda.synchronize()
        assert lidx.lidx_device_status() == 0
        again, _ = lidx.lidx_cache4_attn(*args[:7], table, args[8], **kw)
        assert torch.equal(o, again)
        got, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (got[keys == 0] == 0).all() and np.isneginf(got_l[keys == 0]).all()
        err = np.abs(got - ro)
        assert (err <= tol).all(), f"{np.max(err - tol):.3e} over, at {np.argwhere(~(err <= tol))[:3]}"
        some = keys > 0
        assert (np.abs(got_l[some] - rl[some]) <= sl[some]).all()
