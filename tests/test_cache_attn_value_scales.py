"""Value scales at both ends of their range (lidx_cache_attn): 2^-80 to 2^100, those of a row's keys within 2^100.

Tolerance of the log-sum-exp beside plain.attention's: a score carries log2 of its value scale, which the sum takes off
again.  At magnitudes below 128 an fp32 rounding is 2^-18; the score's, the maximum's and the result's together stay
below 2^-16."""

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


def _check(c, idx=None):
    o, lse = lidx.lidx_cache_attn(*c.args(), want_lse=True,
                                  topk_indices=None if idx is None else torch.from_numpy(idx.astype(np.int32)).to(DEV))
    _status_ok()
    ro, rl, so, sl = plain.attention(c.q, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, idx=idx)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(o - ro)
    assert (err <= so).all(), f"out: {np.max(err / so):.2f} of the slack"
    assert (np.abs(lse - rl) <= sl + 2.0 ** -16).all(), f"lse is off by {np.abs(lse - rl).max():.3e}"


@pytest.mark.parametrize("exps", [(-80, -80), (-70, -70), (-80, -60), (100, 100), (60, 100), (-80, 20), (0, 100)])
@pytest.mark.parametrize("Hq", [8, 32, 64, 128])
@pytest.mark.parametrize("n", [300, 5000])
def test_range_of_value_scales(Hq, exps, n):
    c = Case(Hq + n, 2, 1, Hq, 1, 64, 64, [n, 77], poison=False)
    c.vs[:] = np.exp2(c.g.integers(exps[0], exps[1] + 1, c.vs.shape)).astype(np.float32)
    for b in (0, 1):                                # both ends in every sequence
        c.vs[c.table[b, 0]], c.vs[c.table[b, 1]] = 2.0 ** exps[0], 2.0 ** exps[1]
    if exps == (-70, -70):                          # no powers of two
        c.vs *= np.float32(1.37)
    _check(c)
    _check(c, idx=np.stack([c.g.permutation(n)[:200] for _ in (0, 1)])[:, None])


@pytest.mark.parametrize("Hq", [8, 128])
def test_what_the_writer_gives(Hq):
    """Small, ordinary and very large values go through lidx_cache_append and come back."""
    for e in (-30, 0, 100):
        g = torch.Generator(device=DEV).manual_seed(e + 50)
        x = (torch.randn(1, 200, 1, 64, generator=g, device=DEV).double() * 2.0 ** e).to(torch.bfloat16)
        k = torch.randn(1, 200, 1, 64, generator=g, device=DEV).to(torch.bfloat16)
        f8 = lambda: torch.zeros(4, 1, 64, 64, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        kc, vc, ks, vs = f8(), f8(), torch.ones(4, 1, device=DEV), torch.ones(4, 1, device=DEV)
        table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
        lidx.lidx_cache_append(k, x, kc, vc, ks, vs, table, torch.zeros(1, dtype=torch.int32, device=DEV))
        c = Case(1, 1, 1, Hq, 1, 64, 64, [200], poison=False)
        c.table = table.cpu().numpy()
        c.kc, c.vc = (t.view(torch.uint8).cpu().numpy() for t in (kc, vc))
        c.ks, c.vs = ks.cpu().numpy(), vs.cpu().numpy()
        _check(c)


@pytest.mark.parametrize("exps,q", [((-80, -80), 1.0), ((100, 100), 2.0 ** -107), ((60, 100), 2.0 ** -107), ((-80, -10), 2.0 ** 9)])
@pytest.mark.parametrize("Hq", [8, 32, 64, 128])
def test_range_of_key_scales(Hq, exps, q):
    """Key scales of the same range, with queries that bring the scores to ordinary sizes or below."""
    c = Case(Hq, 2, 1, Hq, 1, 64, 64, [300, 77], q_scale=q, poison=False)
    c.ks[:] = np.exp2(c.g.integers(exps[0], exps[1] + 1, c.ks.shape)).astype(np.float32)
    _check(c)
    _check(c, idx=np.stack([c.g.permutation(300)[:200] for _ in (0, 1)])[:, None])
