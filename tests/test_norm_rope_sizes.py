"""Gradients of norms with rotation (lidx_norm_rope_bwd) for rows of huge and of tiny elements.

A finite row whose sum of squares is infinite in fp32 has r = 0, as in the forward: its gradient is 0, and it adds 0 to dw.
Where the sum of squares and its root are normal numbers (sizes of 2^-60 to 2^60, up to 66 dims), the tolerances of
test_norm_rope hold as they are: every step of their derivation is relative."""

import numpy as np
import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_norm_rope import DEV, angles, check, f64, want_bwd

CASES = [("interleaved", 64), ("half", 64), ("interleaved", 66), ("half", 66)]  # 66 dims: the kernel without vectors


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _inputs(D, dtype):
    g = torch.Generator(device=DEV).manual_seed(D)
    x, gr = (torch.randn(1, 9, 5, D, generator=g, device=DEV).to(dtype) for _ in (0, 1))
    w = torch.rand(D, generator=g, device=DEV) + 0.5
    return x, gr, w, torch.arange(700, 709, dtype=torch.int32, device=DEV), lidx.lidx_rope_freqs(64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout,D", CASES)
def test_rows_whose_squares_are_infinite_have_no_gradient(layout, D, dtype):
    x, gr, w, pos, freqs = _inputs(D, dtype)
    largest = torch.finfo(dtype).max
    huge = {(0, 1): 2.0 ** 64, (3, 4): 2.0 ** 126, (7, 0): largest, (8, 2): -largest}
    rest = torch.ones(9, 5, dtype=torch.bool, device=DEV)
    bad, none = x.clone(), gr.clone()
    for (t, h), v in huge.items():
        bad[0, t, h] = v
        rest[t, h] = False
    bad[0, 5, 3, 17] = largest  # one huge element among ordinary ones
    rest[5, 3] = False
    none[0, ~rest] = 0  # a gradient of 0 adds 0 to dw, whatever the row
    dx, dw = lidx.lidx_norm_rope_bwd(gr, bad, w, pos, freqs, layout=layout)
    want, want_w = lidx.lidx_norm_rope_bwd(none, x, w, pos, freqs, layout=layout)
    assert (dx[0, ~rest] == 0).all()
    assert torch.equal(dx[0, rest], want[0, rest]) and torch.equal(dw, want_w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout,D", CASES)
@pytest.mark.parametrize("exp", [-60, 60])
def test_rows_of_all_normal_sizes(layout, D, dtype, exp):
    x, gr, w, pos, freqs = _inputs(D, dtype)
    x = x * 2.0 ** exp
    ang = angles(freqs, pos.cpu().numpy()[None, None], None)
    dx, tol, dw, dw_tol = want_bwd(f64(gr), f64(x), f64(w), 0.0, ang, 64, 0, layout, 1.0)
    got, got_w = lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs, eps=0.0, layout=layout)
    assert np.isfinite(f64(got)).all()
    check(got, dx, tol, "dx")
    check(got_w, dw, dw_tol, "dw")
