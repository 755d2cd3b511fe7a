"""Rotary positions of prompts: sizes that take the kernel with four items a thread (1024 items a block, at least two blocks an
SM), against the 64-bit definition on the device.  Tolerance of an element as derived in test_rope.py."""

import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

pytestmark = pytest.mark.gpu
DEV = "cuda"
ITEMS = 2 * 1024 * 152  # from here on a block takes 1024 items


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _definition(x, pos, omega, layout, off, m, inverse):
    """(value, |a| + |b| of the element's pair or 0) in float64."""
    y = x.double()
    size = torch.zeros_like(y)
    half = omega.numel()
    i = torch.arange(half, device=DEV)
    ia, ib = (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + i + half)
    angle = (pos.double()[..., None] * omega)[:, :, None]
    c, s = m * angle.cos(), m * angle.sin() * (-1.0 if inverse else 1.0)
    a, b = y[..., ia], y[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


CASES = [
    # T0, T1, H, H2, D, R, off
    (3, 177, 64, 1, 128, 64, 64),     # 65 heads: a token's items do not divide a block's
    (1, 1999, 20, 5, 128, 128, 0),
    (1, 3501, 9, 0, 80, 40, 40),      # 40 of 80 dims
    (7, 700, 8, 8, 64, 32, 0),
    (1, 110001, 3, 0, 16, 16, 0),     # many tokens a block
    (2, 160001, 1, 0, 16, 16, 0),     # and too many angles for it: one item a thread
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T0,T1,H,H2,D,R,off", CASES)
def test_prompts_against_the_definition(T0, T1, H, H2, D, R, off, layout, dtype):
    vec = 16 // dtype.itemsize
    items = (R // 2 // vec if layout == "half" else R // vec) + (D - R) // vec
    whole = (R // 2 if layout == "half" else R) % vec == 0
    if dtype == torch.bfloat16 and whole and H > 1:
        assert T0 * T1 * (H + H2) * items >= ITEMS
    g = torch.Generator(device=DEV).manual_seed(T1)
    x = torch.randn(T0, T1, H, D, generator=g, device=DEV).to(dtype)
    x2 = torch.randn(T0, T1, H2, D, generator=g, device=DEV).to(dtype) if H2 else None
    pos = torch.randint(0, 1 << 20, (T0, T1), generator=g, device=DEV).to(torch.int32)
    m = 1.3466
    freqs = lidx.lidx_rope_freqs(R, scaling="yarn", factor=32.0)
    omega = freqs.double() * (6.283185307179586476925286766559 / 2.0 ** 64)  # (below 2^62: the sign bit is clear)
    for inverse, call in ((False, lidx.lidx_rope), (True, lidx.lidx_rope_bwd)):
        got = call(x, pos, freqs, x2=x2, layout=layout, rot_off=off, mscale=m)
        for y, t in zip(got if H2 else (got,), (x, x2)):
            want, size = _definition(t, pos, omega, layout, off, m, inverse)
            tol = 16 * 2.0 ** -24 * m * size + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)
            err = (y.double() - want).abs()
            assert (err <= tol).all(), f"inverse={inverse}: {(err - tol).max().item():.3e} over"


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_prompt_strides_and_in_place(layout):
    """Slices of a fused projection, both tensors, in place: the bits of the contiguous call, and nothing else written."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T0, T1, H, H2, D = 2, 301, 32, 8, 128
    fused = torch.randn(T1, T0, H + H2 + 2, D, generator=g, device=DEV).to(torch.bfloat16)
    x, x2 = (fused.transpose(0, 1)[:, :, a:z] for a, z in ((1, 1 + H), (1 + H, 1 + H + H2)))
    freqs = lidx.lidx_rope_freqs(64)
    pos = torch.arange(50, 50 + T1, dtype=torch.int32, device=DEV)
    kw = dict(layout=layout, rot_off=32)
    want = lidx.lidx_rope(x.contiguous(), pos, freqs, x2=x2.contiguous(), **kw)
    got = lidx.lidx_rope(x, pos, freqs, x2=x2, **kw)
    before = fused.clone()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(fused, before)
    lidx.lidx_rope(x, pos, freqs, x2=x2, out=(x, x2), **kw)
    assert torch.equal(x, want[0]) and torch.equal(x2, want[1])
    assert torch.equal(fused[:, :, [0, H + H2 + 1]], before[:, :, [0, H + H2 + 1]])
