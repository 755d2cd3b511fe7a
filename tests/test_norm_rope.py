"""Norms of each head with rotary positions (lidx_norm_rope, lidx_norm_rope_bwd) and positions of several axes (lidx_rope with
axes) against their 64-bit definitions.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32; D at most 1024):
  * a sum of D squares on up to 32 lanes: D/32 + 5 additions in a row, each off by u: below 40 u; mean, eps and the root add
    3 u, so r is off by 24 u of itself (half of 40 u and 3 u), and n = x r w by 28 u
  * a turn adds 16 u of mscale (|a| + |b|) (angle, cosine, sine and two products, as for lidx_rope)
  * forward: 28 u |n| turned, which is at most 28 u (|a| + |b|), and 16 u (|a| + |b|): below 48 u m (|a| + |b|)
  * backward: u' = turn of g (16 u m (|a| + |b|)), t = u' w, c = mean(t h): sums of D products (40 u of the sum of sizes); dx = r
    (t - h c): below 96 u r (m T + |h| mean(m T |h|)) with T the pair's sizes |a w| + |b w| (or the element's own)
  * dw: sums over N rows, in order at most rows-a-thread + 64 + 32 + 32 of them: bounded by (128 + N / 16) u of the sum of sizes
  * bf16 outputs are rounded once more: 2^-8 of the value
"""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


# ------------------------------------------------------------------ the definition

def pairs_of(R, off, layout):
    i = np.arange(R // 2)
    return (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + i + R // 2)


def angles(freqs, pos, axes):
    """[T0,T1,pairs] radians of int positions [A,T0,T1], from the fixed-point frequencies exactly."""
    f = [int(v) for v in freqs.cpu().numpy().view(np.uint64)]
    A = pos.shape[0]
    out = np.empty(pos.shape[1:] + (len(f),))
    for at in np.ndindex(*pos.shape[1:]):
        for u, fu in enumerate(f):
            p = int(pos[(min(int(axes[u]), A - 1) if axes is not None else 0,) + at])
            out[at + (u,)] = plain.TWO_PI * ((p * fu) % 2 ** 64 / 2.0 ** 64)
    return out


def turn(x, ang, R, off, layout, m, inverse):
    c, s = m * np.cos(ang)[:, :, None], m * np.sin(ang)[:, :, None] * (-1 if inverse else 1)
    ia, ib = pairs_of(R, off, layout)
    y = x.copy()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    return y


def pair_size(x, R, off, layout, m):
    """|a| + |b| of an element's pair, times m; the element itself where it is not rotated."""
    y = np.abs(x)
    ia, ib = pairs_of(R, off, layout)
    s = m * (y[..., ia] + y[..., ib])
    y[..., ia] = y[..., ib] = s
    return y


def norm(x, w, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * w, r


def want_fwd(x, w, eps, ang, R, off, layout, m):
    n, _ = norm(x, w, eps)
    return turn(n, ang, R, off, layout, m, False), 48 * U * pair_size(n, R, off, layout, abs(m))


def want_bwd(g, x, w, eps, ang, R, off, layout, m):
    D = x.shape[-1]
    _, r = norm(x, 1.0, eps)
    u = turn(g, ang, R, off, layout, m, True)
    h, t = x * r, u * w
    dx = r * (t - h * (t * h).mean(-1, keepdims=True))
    us = pair_size(g, R, off, layout, abs(m))
    ts = us * np.abs(w)
    tol = 96 * U * r * (ts + np.abs(h) * (ts * np.abs(h)).mean(-1, keepdims=True))
    rows = x.reshape(-1, D).shape[0]
    dw = (u * h).sum((0, 1, 2))
    dw_tol = (128 + rows / 16 + 48) * U * (us * np.abs(h)).sum((0, 1, 2))
    return dx, tol, dw, dw_tol


def check(got, want, tol, what):
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert got.shape == want.shape and (err <= tol).all(), f"{what}: {np.nanmax(err - tol):.3e} over"


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ refusals (CPU)

def test_axis_map():
    assert lidx.lidx_rope_axis_map((2, 3, 1), device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert lidx.lidx_rope_axis_map((2, 3, 1), interleaved=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 1]
    for bad in ((), (0, 0), (-1, 2), (1,) * 256):
        with pytest.raises(ValueError):
            lidx.lidx_rope_axis_map(bad, device="cpu")


def _turn_c(pos=16, freqs=16, axis=16, axes=1, R=32, off=0, layout=0, m=1.0):
    return lidx._RopeTurn(pos, (C.c_int64 * 3)(1, 1, 1), freqs, axis, axes, R, off, layout, m)


def test_axes_refusals_without_gpu():
    L = lidx.lib()

    def call(nt=1, x=16, y=16, H=2, T0=1, T1=1, D=64, inv=0, dt=1, turn=True, **kw):
        t = (lidx._RopeTensor * 2)()
        for a in t:
            a.x, a.y, a.H = x, y, H
        r = _turn_c(**kw)
        return L.lidx_rope_axes(t, nt, C.byref(r) if turn else None, T0, T1, D, inv, dt, None)

    assert call(turn=False) == 1 and call(pos=None) == 1 and call(freqs=None) == 1 and call(x=None) == 1
    for bad in (dict(axes=0), dict(axes=256), dict(axes=2, axis=None), dict(R=0), dict(R=33), dict(R=66), dict(off=34),
                dict(layout=2), dict(m=math.inf), dict(inv=2), dict(dt=2), dict(nt=3), dict(H=0), dict(T0=0), dict(D=63)):
        assert call(**bad) == 2, bad
    assert call(pos=18) == 3 and call(freqs=20) == 3 and call(x=17) == 3


def test_norm_refusals_without_gpu():
    L = lidx.lib()

    def call(bwd, nt=1, x=16, g=16, y=16, w=16, dw=16, H=2, T0=1, T1=1, D=64, dt=1, wdt=1, eps=1e-6, null=False, ws=256,
             wsb=1 << 24, **kw):
        t = (lidx._NormTensor * 2)()
        for a in t:
            a.x, a.g, a.y, a.w, a.dw, a.H = x, g, y, w, dw, H
        r = _turn_c(**kw)
        t = None if null else t
        if bwd:
            return L.lidx_norm_rope_bwd(t, nt, C.byref(r), eps, T0, T1, D, dt, wdt, C.c_void_p(ws), wsb, None)
        return L.lidx_norm_rope(t, nt, C.byref(r), eps, T0, T1, D, dt, wdt, None)

    for bwd in (False, True):
        assert call(bwd, null=True) == 1 and call(bwd, x=None) == 1 and call(bwd, y=None) == 1 and call(bwd, pos=None) == 1
        for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(nt=0), dict(nt=3), dict(dt=2), dict(wdt=2),
                    dict(H=0), dict(H=1 << 16), dict(T0=0), dict(T0=1 << 20, T1=1 << 20), dict(D=1026), dict(R=2, off=64),
                    dict(axes=3, axis=None)):
            assert call(bwd, **bad) == 2, bad
        assert call(bwd, x=17) == 3 and call(bwd, w=17) == 3 and call(bwd, wdt=0, w=18) == 3 and call(bwd, pos=17) == 3
    assert call(True, g=None) == 1 and call(True, dw=18) == 3 and call(True, g=17) == 3
    assert lidx.lib().lidx_norm_rope_bwd_workspace_bytes(1026) == 0
    assert lidx.lib().lidx_norm_rope_bwd_workspace_bytes(128) >= 148 * 128 * 4


# ------------------------------------------------------------------ GPU

CASES = [
    # T0, T1, H, H2, D, R, off, axes
    (1, 1, 1, 0, 16, 16, 0, 1),
    (16, 1, 64, 8, 128, 128, 0, 1),
    (2, 7, 3, 2, 128, 64, 64, 3),
    (1, 33, 20, 4, 80, 36, 44, 2),     # a rotated part that no vector fits
    (1, 9, 2, 0, 48, 2, 7, 1),
    (3, 5, 4, 1, 64, 64, 0, 1),
    (3, 11, 5, 5, 80, 80, 0, 2),
    (1, 300, 1, 0, 128, 64, 0, 4),
    (1, 2, 130, 130, 32, 16, 8, 1),
    (1, 3, 1, 1, 1024, 1024, 0, 3),    # too wide for the lanes of a row
    (2, 9, 3, 1, 512, 512, 0, 1),
    (2, 5, 3, 1, 256, 96, 160, 2),
    (2, 3, 5, 0, 6, 4, 2, 1),
    (1, 1300, 9, 2, 96, 32, 32, 1),    # several chunks a block
]


def _inputs(T0, T1, H, H2, D, A, dtype, wdtype, seed):
    g = np.random.default_rng(seed)

    def rows(h):
        # sizes of rows differ, and one is nothing but zeros
        x = g.standard_normal((T0, T1, h, D)) * np.exp(g.standard_normal((T0, T1, h, 1)))
        x[0, 0, 0] = 0
        return torch.from_numpy(x).to(dtype).to(DEV)

    x, gr = rows(H), rows(H)
    x2, gr2 = (rows(H2), rows(H2)) if H2 else (None, None)
    w, w2 = (torch.from_numpy(1 + 0.3 * g.standard_normal(D)).to(wdtype).to(DEV) for _ in (0, 1))
    pos = g.integers(0, 200000, (A, T0, T1)).astype(np.int32)
    pos.flat[0] = 2 ** 31 - 1
    if pos.size > 2:
        pos.flat[1], pos.flat[2] = -2 ** 31, -17
    return x, gr, x2, gr2, w, w2, pos


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T0,T1,H,H2,D,R,off,A", CASES)
def test_norm_against_the_definition(T0, T1, H, H2, D, R, off, A, layout, dtype, wdtype):
    x, g, x2, g2, w, w2, pos = _inputs(T0, T1, H, H2, D, A, dtype, wdtype, T1 * 31 + D)
    freqs = lidx.lidx_rope_freqs(R, scaling="yarn", factor=32.0)
    axes = torch.arange(R // 2, device=DEV).remainder(A + 1).to(torch.uint8) if A > 1 else None  # an id past the last axis
    ang = angles(freqs, pos, None if axes is None else axes.cpu().numpy())
    m, eps = 1.3466, 1e-5
    p = torch.from_numpy(pos).to(DEV)
    kw = dict(eps=eps, layout=layout, rot_off=off, mscale=m, axes=axes)
    p = p if A > 1 else p[0]
    got = lidx.lidx_norm_rope(x, w, p, freqs, x2=x2, weight2=w2 if H2 else None, **kw)
    for y, xi, wi in zip(got if H2 else (got,), (x, x2), (w, w2)):
        check(y, *want_fwd(f64(xi), f64(wi), eps, ang, R, off, layout, m), "y")
    got = lidx.lidx_norm_rope_bwd(g, x, w, p, freqs, g2=g2, x2=x2, weight2=w2 if H2 else None, **kw)
    again = lidx.lidx_norm_rope_bwd(g, x, w, p, freqs, g2=g2, x2=x2, weight2=w2 if H2 else None, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i, (gi, xi, wi) in enumerate(((g, x, w), (g2, x2, w2))[:2 if H2 else 1]):
        dx, tol, dw, dw_tol = want_bwd(f64(gi), f64(xi), f64(wi), eps, ang, R, off, layout, m)
        check(got[2 * i], dx, tol, "dx")
        check(got[2 * i + 1], dw, dw_tol, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T0,T1,H,H2,D,R,off,A", [c for c in CASES if c[-1] > 1])
def test_axes_against_the_definition(T0, T1, H, H2, D, R, off, A, layout, dtype):
    x, _, x2, _, _, _, pos = _inputs(T0, T1, H, H2, D, A, dtype, dtype, 5 * T1 + R)
    freqs = lidx.lidx_rope_freqs(R)
    axes = lidx.lidx_rope_axis_map([R // 2 - (A - 1)] + [1] * (A - 1), interleaved=layout == "half")
    ang = angles(freqs, pos, axes.cpu().numpy())
    p = torch.from_numpy(pos).to(DEV)
    for inverse, call in ((False, lidx.lidx_rope), (True, lidx.lidx_rope_bwd)):
        got = call(x, p, freqs, x2=x2, layout=layout, rot_off=off, mscale=0.7, axes=axes)
        for y, t in zip(got if H2 else (got,), (x, x2)):
            t = f64(t)
            tol = 16 * U * np.maximum(2 * np.abs(t).max(-1, keepdims=True), np.abs(t))
            check(y, turn(t, ang, R, off, layout, 0.7, inverse), tol, f"inverse={inverse}")


@pytest.mark.gpu
def test_one_axis_for_all_is_the_plain_call():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(2, 9, 3, 64, generator=g, device=DEV)
    pos = torch.randint(0, 9999, (2, 9), generator=g, device=DEV).to(torch.int32)
    freqs = lidx.lidx_rope_freqs(32)
    want = lidx.lidx_rope(x, pos, freqs)
    ids = torch.full((16,), 2, dtype=torch.uint8, device=DEV)
    other = torch.randint(0, 9999, (2, 2, 9), generator=g, device=DEV).to(torch.int32)
    assert torch.equal(lidx.lidx_rope(x, torch.cat((other, pos[None])), freqs, axes=ids), want)
    # positions that are the same for every sequence, and for every token
    assert torch.equal(lidx.lidx_rope(x, pos[:1].expand(3, 9), freqs, axes=ids),
                       lidx.lidx_rope(x, pos[0], freqs))
    three = torch.tensor([1, 2, 77], dtype=torch.int32, device=DEV)
    assert torch.equal(lidx.lidx_rope(x, three, freqs, axes=ids), lidx.lidx_rope(x, three[2:], freqs))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_strides_in_place_and_streams(layout):
    """Heads of a fused, transposed projection, not aligned to 16 bytes too; in place; on a stream of its own: the same
    results as the contiguous call's (bits on the same path, else the tolerance's)."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T0, T1, H, D, R, off = 3, 11, 6, 64, 32, 16
    freqs = lidx.lidx_rope_freqs(R)
    w = torch.rand(D, generator=g, device=DEV) + 0.5
    fused = torch.randn(T1, T0, H + 3, D + 8, generator=g, device=DEV).to(torch.bfloat16)
    x = fused.transpose(0, 1)[:, :, 1:1 + H, :D]
    gr = torch.randn(T0, T1, H, D, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.arange(100, 100 + T1, dtype=torch.int32, device=DEV)
    kw = dict(layout=layout, rot_off=off)
    want = lidx.lidx_norm_rope(x.contiguous(), w, pos, freqs, **kw)
    assert torch.equal(lidx.lidx_norm_rope(x, w, pos, freqs, **kw), want)
    dx, dw = lidx.lidx_norm_rope_bwd(gr, x.contiguous(), w, pos, freqs, **kw)
    got = lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs, **kw)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    odd = fused.transpose(0, 1)[:, :, 1:1 + H, 3:3 + D]
    ang = angles(freqs, pos.cpu().numpy()[None, None].repeat(T0, 1), None)
    check(lidx.lidx_norm_rope(odd, w, pos, freqs, **kw), *want_fwd(f64(odd), f64(w), 1e-6, ang, R, off, layout, 1.0), "odd")
    # the gradient into the incoming gradient's memory
    held, dwo = gr.clone(), torch.empty(D, device=DEV)
    assert lidx.lidx_norm_rope_bwd(held, x, w, pos, freqs, out=(held, dwo), **kw)[0] is held
    assert torch.equal(held, dx) and torch.equal(dwo, dw)
    before = fused.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lidx.lidx_norm_rope(x, w, pos, freqs, out=x, stream=st, **kw)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(x, want)
    rest = torch.ones(fused.shape, dtype=torch.bool, device=DEV)
    rest.transpose(0, 1)[:, :, 1:1 + H, :D] = False
    assert torch.equal(fused[rest], before[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradients_against_differences(layout):
    """<g, y(x + s e) - y(x - s e)> / 2s against <dx, e>, and the same for w, of the 64-bit definition's forward: dx and dw in
    fp32 are off by their tolerances, the difference by its third derivative, s^2 = 2^-20 of sizes of order one."""
    gen = np.random.default_rng(11)
    T, H, D, R = 5, 3, 32, 24
    freqs = lidx.lidx_rope_freqs(R)
    pos = gen.integers(0, 5000, (1, 1, T)).astype(np.int32)
    ang = angles(freqs, pos, None)
    x, g, e = (gen.standard_normal((1, T, H, D)).astype(np.float32) for _ in range(3))
    w, ew = 1 + 0.3 * gen.standard_normal(D).astype(np.float32), gen.standard_normal(D).astype(np.float32)
    kw = dict(layout=layout, rot_off=8, mscale=1.25)
    cu = lambda a: torch.from_numpy(a).to(DEV)
    dx, dw = lidx.lidx_norm_rope_bwd(cu(g), cu(x), cu(w), cu(pos[0]), freqs, **kw)
    f = lambda xx, ww: turn(norm(xx, ww, 1e-6)[0], ang, R, 8, layout, 1.25, False)
    s = 2.0 ** -10
    x, g, e, w, ew = (a.astype(np.float64) for a in (x, g, e, w, ew))
    left = (g * (f(x + s * e, w) - f(x - s * e, w))).sum() / (2 * s)
    right = (f64(dx) * e).sum()
    size = (np.abs(g).max() * np.abs(e).max() * 20) * T * H * D
    assert abs(left - right) <= 2.0 ** -20 * size
    left = (g * (f(x, w + s * ew) - f(x, w - s * ew))).sum() / (2 * s)
    assert abs(left - (f64(dw) * ew).sum()) <= 2.0 ** -20 * size


@pytest.mark.gpu
def test_no_weight_and_rows_that_are_not_finite():
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(1, 6, 4, 64, generator=g, device=DEV)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    freqs = lidx.lidx_rope_freqs(64)
    one = torch.ones(64, device=DEV)
    want = lidx.lidx_norm_rope(x, one, pos, freqs)
    assert torch.equal(lidx.lidx_norm_rope(x, None, pos, freqs), want)
    dx, dw = lidx.lidx_norm_rope_bwd(x, x, None, pos, freqs)
    assert dw is None and torch.equal(dx, lidx.lidx_norm_rope_bwd(x, x, one, pos, freqs)[0])
    bad = x.clone()
    bad[0, 1, 2, 5], bad[0, 4, 0, 63] = float("inf"), float("nan")
    y = lidx.lidx_norm_rope(bad, one, pos, freqs)
    rows = torch.zeros(1, 6, 4, dtype=torch.bool, device=DEV)
    rows[0, 1, 2] = rows[0, 4, 0] = True
    assert torch.equal(y[~rows], want[~rows])
    assert y[0, 4, 0].isnan().all() and y[0, 1, 2].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 66])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rows_whose_squares_are_infinite(layout, D):
    """r is 0: the infinity and its pair are NaN, everything else and rows of finite, huge elements are 0; no other row
    differs, forward or backward.  (66 dims take the kernel without vectors.)"""
    g = torch.Generator(device=DEV).manual_seed(9)
    x, gr = (torch.randn(1, 5, 3, D, generator=g, device=DEV) for _ in (0, 1))
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    w, freqs = torch.rand(D, generator=g, device=DEV) + 0.5, lidx.lidx_rope_freqs(64)
    want = lidx.lidx_norm_rope(x, w, pos, freqs, layout=layout)
    dwant, _ = lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs, layout=layout)
    bad = x.clone()
    bad[0, 2, 1, 5], bad[0, 4, 2] = float("inf"), 2.0 ** 64
    y = lidx.lidx_norm_rope(bad, w, pos, freqs, layout=layout)
    dx, dw = lidx.lidx_norm_rope_bwd(gr, bad, w, pos, freqs, layout=layout)
    rest = torch.ones(1, 5, 3, dtype=torch.bool, device=DEV)
    rest[0, 2, 1] = rest[0, 4, 2] = False
    assert torch.equal(y[rest], want[rest]) and torch.equal(dx[rest], dwant[rest])
    pair = [4, 5] if layout == "interleaved" else [5, 37]
    row = y[0, 2, 1]
    assert row[pair].isnan().all() and row.isnan().sum() == 2 and (row[~row.isnan()] == 0).all()
    assert (y[0, 4, 2] == 0).all()
    assert dx[0, 2, 1].isnan().any() and dw[5].isnan()


@pytest.mark.gpu
def test_captured_and_replayed_with_two_graphs():
    """Two captured backward passes, each with its workspace, replayed with new inputs while eager calls go on."""
    g = torch.Generator(device=DEV).manual_seed(5)
    freqs = lidx.lidx_rope_freqs(128)
    pos = torch.arange(70, dtype=torch.int32, device=DEV)
    x, gr = (torch.randn(1, 70, 8, 128, generator=g, device=DEV) for _ in (0, 1))
    w = torch.rand(128, generator=g, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            outs.append(lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs) + (lidx.lidx_norm_rope(x, w, pos, freqs),))
        graphs.append(gph)
    x.copy_(torch.randn(x.shape, generator=g, device=DEV))
    want = lidx.lidx_norm_rope_bwd(gr, x, w, pos, freqs) + (lidx.lidx_norm_rope(x, w, pos, freqs),)
    for gph, out in zip(graphs, outs):
        gph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_binding_refusals():
    freqs = lidx.lidx_rope_freqs(16)
    x = torch.zeros(1, 2, 1, 32, device=DEV)
    w = torch.ones(32, device=DEV)
    pos = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    ids = torch.zeros(8, dtype=torch.uint8, device=DEV)
    call, bwd = lidx.lidx_norm_rope, lidx.lidx_norm_rope_bwd
    for bad in (lambda: call(x.half(), w, pos, freqs), lambda: call(x, w.half(), pos, freqs),
                lambda: call(x, w, pos.long(), freqs), lambda: call(x, w, pos, freqs.float()),
                lambda: call(x, w, pos[None], freqs, axes=ids.int()), lambda: call(x, w, pos, freqs, x2=x, weight2=w.bfloat16()),
                lambda: bwd(None, x, w, pos, freqs), lambda: bwd(x, x, w, pos, freqs, x2=x),
                lambda: bwd(x.bfloat16(), x, w, pos, freqs)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: call(x, w[:16], pos, freqs), lambda: call(x, w, pos, freqs, x2=x[:, :1]),
                lambda: call(x, w, pos, freqs, layout="other"), lambda: call(x, w, pos, freqs, out=x[:, :1]),
                lambda: call(x, w, pos[None], freqs, axes=ids[:4]), lambda: bwd(x[:, :1], x, w, pos, freqs),
                lambda: call(x, w.cpu(), pos, freqs), lambda: bwd(x, x, w, pos, freqs, out=(x.clone(), w[:8]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(x, w, pos, freqs, rot_off=20), lambda: call(x, w, pos, freqs, eps=-1.0),
                lambda: bwd(x, x, w, pos, freqs, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(lidx.LidxError):
            bad()


def test_a_second_weight_needs_a_second_tensor():
    x = torch.zeros(1, 1, 1, 64)
    with pytest.raises(TypeError, match="weight2"):
        lidx.lidx_norm_rope(x, None, None, None, weight2=torch.ones(64))
    with pytest.raises(TypeError, match="weight2"):
        lidx.lidx_norm_rope_bwd(x, x, None, None, None, weight2=torch.ones(64))
