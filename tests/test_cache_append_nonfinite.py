"""Infinities and NaN among appended tokens (lidx_cache_append): they are stored as NaN codes, e4m3 having no infinity, and
the page's scale is that of its finite values, so the tokens beside them keep theirs."""

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


@pytest.mark.parametrize("bad", [(INF,), (-INF,), (NAN,), (-NAN, INF, -INF)])
@pytest.mark.parametrize("B,S,Hkv,D,page,starts", [
    (1, 1, 1, 16, 16, [0]),               # the token alone in a fresh page
    (1, 1, 2, 128, 64, [5]),              # behind earlier tokens
    (2, 40, 3, 80, 16, [7, 16]),          # several pages of a call
    (1, 300, 1, 128, 128, [100]),
])
def test_nonfinite_tokens_leave_the_others_alone(B, S, Hkv, D, page, starts, bad):
    g = np.random.default_rng(S + D)
    MP = (max(starts) + S) // page + 1
    NP = B * MP
    table = g.permutation(NP).reshape(B, MP).astype(np.int32)
    x = torch.from_numpy(g.standard_normal((B, S, Hkv, D)) * 5).to(torch.bfloat16)
    for i, z in enumerate(bad):           # here and there, in the last head of a few tokens, at both ends of a row
        x[B - 1, (i * 17) % S, Hkv - 1, [0, D - 1, 9][i % 3]] = z
        x[0, S // 2, 0, 3 + i] = z
    cache, scale = plain.random_cache(g, NP, Hkv, page, D, -10, -9)
    got = [plain.to_cuda(cache), plain.to_cuda(cache), torch.from_numpy(scale).to(DEV), torch.from_numpy(scale).to(DEV)]
    lidx.lidx_cache_append(x.to(DEV), x.to(DEV), *got, torch.from_numpy(table).to(DEV),
                           torch.tensor(starts, dtype=torch.int32, device=DEV))
    finite = torch.isfinite(x)
    plain.append(torch.where(finite, x, torch.zeros_like(x)), cache, scale, table, starts, [S] * B)
    nan = np.zeros(cache.shape, bool)
    for b in range(B):
        for i in range(S):
            p = starts[b] + i
            nan[table[b, p // page], :, p % page] = ~finite[b, i].numpy()
    for codes, s in zip(got[:2], got[2:]):
        codes = codes.view(torch.uint8).cpu().numpy()
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal((codes & 0x7F) == 0x7F, nan)
        assert np.array_equal(codes[~nan], cache[~nan])


def test_a_page_of_infinities():
    """No finite value at all: the smallest scale, and earlier tokens keep theirs."""
    cache = torch.full((2, 1, 16, 32), 0x38, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # ones
    scale = torch.full((2, 1), 0.25, device=DEV)
    x = torch.full((1, 14, 1, 32), INF, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    lidx.lidx_cache_append(x, x, cache, cache.clone(), scale, scale.clone(), table,
                           torch.tensor([8], dtype=torch.int32, device=DEV))
    codes = cache.view(torch.uint8).cpu().numpy()
    assert scale.tolist() == [[0.25], [2.0 ** -40]]
    assert (codes[0, 0, :8] == 0x38).all() and ((codes[0, 0, 8:] & 0x7F) == 0x7F).all()
    assert ((codes[1, 0, :6] & 0x7F) == 0x7F).all() and (codes[1, 0, 6:] == 0x38).all()
