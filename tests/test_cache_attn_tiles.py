"""What the lanes of a softmax warp hand to each other for a tile (lidx_cache_attn): shift and fade of its own."""

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_cache_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("Hq", [8, 16, 32, 64, 128])
def test_each_tile_has_its_own_shift(Hq, up):
    """Every tile counts alike in the sum and has another maximum: value scales fall (no running maximum grows, so no sum
    is faded) or grow (every tile fades) by 2^5 a tile of 128 keys, scores are nearly flat.  A tile that took the shift or fade
    of the tile before would be off by 2^5."""
    n = 128 * 7 - 5
    for B in (1, 50):  # tiles spread over CTAs; several tiles a CTA
        c = Case(Hq + B, B, 1, Hq, 1, 64, 128, [n] * B, q_scale=0.01, poison=False)
        step = np.arange(7) if up else -np.arange(7)
        for b in range(B):
            c.vs[c.table[b], 0] = np.exp2(5.0 * step + (-15 if up else 15)).astype(np.float32)
        c.check(whole=False)
        c.check(idx=np.tile(np.arange(n), (B, 1, 1)), whole=False)
