"""Norms with rotation of prompts: sizes that take the forward kernel with two rows a thread and several chunks a block of the
backward, and more rows than 31 bits count.  Against the 64-bit definition on the device; tolerances as derived in
test_norm_rope.py.  (dw there counts at most rows-a-thread + 128 additions in order; a block of 256 threads with 32 lanes a row,
the most, has eight rows at a time, and there are two blocks an SM at least, so a thread has at most rows / 2400 + 1.)"""

import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

pytestmark = pytest.mark.gpu
DEV, U = "cuda", 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _pairs(R, off, layout):
    i = torch.arange(R // 2, device=DEV)
    return (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + i + R // 2)


def _angles(pos, freqs):
    """cos and sin [T0,T1,1,pairs] of the fixed-point angles: positions below 2^20, so the product's upper 43 bits decide."""
    f = [int(v) % 2 ** 64 for v in freqs.tolist()]
    hi = torch.tensor([v >> 32 for v in f], dtype=torch.float64, device=DEV)
    lo = torch.tensor([v & 0xFFFFFFFF for v in f], dtype=torch.float64, device=DEV)
    p = pos.double()[..., None]
    t = (p * hi).remainder(2.0 ** 32) / 2.0 ** 32 + p * lo / 2.0 ** 64  # both products are exact
    a = (plain.TWO_PI * t)[:, :, None]
    return a.cos(), a.sin()


def _turn(x, cs, R, off, layout, m, inverse):
    ia, ib = _pairs(R, off, layout)
    c, s = m * cs[0], m * cs[1] * (-1.0 if inverse else 1.0)
    y = x.clone()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def _size(x, R, off, layout, m):
    ia, ib = _pairs(R, off, layout)
    y = x.abs()
    y[..., ia] = y[..., ib] = m * (y[..., ia] + y[..., ib])
    return y


def _check(got, want, tol, what):
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    over = ((got.double() - want).abs() - tol).max().item()
    assert over <= 0, f"{what}: {over:.3e} over"


CASES = [
    # T0, T1, H, H2, D, R, off
    (2, 700, 32, 4, 128, 128, 0),
    (1, 3001, 16, 2, 128, 64, 64),
    (3, 999, 20, 0, 64, 64, 0),
    (1, 40009, 3, 0, 32, 32, 0),      # four lanes a row, many tokens a block
    (1, 1501, 13, 5, 512, 256, 256),  # 32 lanes a row in bf16, too wide for the vectors in fp32
    (1, 5003, 9, 3, 80, 40, 0),       # no vector fits the halves in bf16
    (1, 150001, 1, 0, 64, 64, 0),     # too many angles for two rows a thread
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T0,T1,H,H2,D,R,off", CASES)
def test_prompts_against_the_definition(T0, T1, H, H2, D, R, off, layout, dtype):
    g = torch.Generator(device=DEV).manual_seed(T1)
    rnd = lambda h: torch.randn(T0, T1, h, D, generator=g, device=DEV).to(dtype) if h else None
    xs, gs = (rnd(H), rnd(H2)), (rnd(H), rnd(H2))
    ws = [torch.rand(D, generator=g, device=DEV) + 0.5 for _ in xs]
    pos = torch.randint(0, 1 << 20, (T0, T1), generator=g, device=DEV).to(torch.int32)
    freqs, m, eps = lidx.lidx_rope_freqs(R), 1.25, 1e-5
    kw = dict(eps=eps, layout=layout, rot_off=off, mscale=m)
    second = dict(x2=xs[1], weight2=ws[1]) if H2 else {}
    y = lidx.lidx_norm_rope(xs[0], ws[0], pos, freqs, **second, **kw)
    y = y if H2 else (y,)
    d = lidx.lidx_norm_rope_bwd(gs[0], xs[0], ws[0], pos, freqs, g2=gs[1], **second, **kw)
    cs = _angles(pos, freqs)
    for i in range(2 if H2 else 1):
        x, gr, w = xs[i].double(), gs[i].double(), ws[i].double()
        rows = x.numel() // D
        r = 1.0 / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
        n = x * r * w
        _check(y[i], _turn(n, cs, R, off, layout, m, False), 48 * U * _size(n, R, off, layout, m), "y")
        u, h = _turn(gr, cs, R, off, layout, m, True), x * r
        t, us = u * w, _size(gr, R, off, layout, m)
        ts = us * w
        _check(d[2 * i], r * (t - h * (t * h).mean(-1, keepdim=True)),
               96 * U * r * (ts + h.abs() * (ts * h.abs()).mean(-1, keepdim=True)), "dx")
        _check(d[2 * i + 1], (u * h).sum((0, 1, 2)), (128 + rows / 2400 + 1 + 48) * U * (us * h.abs()).sum((0, 1, 2)), "dw")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_more_rows_than_31_bits(layout):
    """2^31 rows of eight dims: 64 tokens of 16 heads over and over, of which only the outputs take memory.  (In halves no
    vector fits.)"""
    g = torch.Generator(device=DEV).manual_seed(3)
    T0, T1, H, D = 1 << 21, 64, 16, 8
    x, gr = (torch.randn(1, T1, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in (0, 1))
    w, freqs = torch.rand(D, generator=g, device=DEV) + 0.5, lidx.lidx_rope_freqs(D)
    pos = torch.arange(1000, 1000 + T1, dtype=torch.int32, device=DEV)
    many = lambda t: t.expand(T0, T1, H, D)
    y = torch.zeros(T0, T1, H, D, dtype=torch.bfloat16, device=DEV)
    lidx.lidx_norm_rope(many(x), w, pos, freqs, layout=layout, out=y)
    same = lambda t: all((c == t).all().item() for c in y.split(1 << 17))
    assert same(lidx.lidx_norm_rope(x, w, pos, freqs, layout=layout))
    y.zero_()
    _, dw = lidx.lidx_norm_rope_bwd(many(gr), many(x), w, pos, freqs, layout=layout, out=(y, None))
    dx, one = lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs, layout=layout)
    assert same(dx)
    # a thread of the fewest, 32 rows at a time and two blocks an SM: 2^31 / (2 * 152 * 8) additions in order, at most
    size = (_size(gr.double(), D, 0, layout, 1.0) * (x.double() * (x.double() ** 2).mean(-1, keepdim=True).rsqrt()).abs()).sum((0, 1, 2))
    assert ((dw.double() - T0 * one.double()).abs() <= (2.0 ** 31 / (2 * 152 * 8) + 256) * U * T0 * size).all()
