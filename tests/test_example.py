"""The example that serves one sparse-attention layer end to end runs and agrees with plain torch: weights of
8 bits and a bf16 output, 5e-3 of the output's norm (see test_cache_attn.py)."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_sparse_decode_example():
    from sparse_attention_top_tcgen05_gb300 import build

    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sparse_decode

    assert sparse_decode.main(prompt=130, steps=6, verbose=False) <= 5e-3
