"""Rotary positions (lidx_rope, lidx_rope_bwd, lidx_rope_freqs) against their 64-bit definition.

Tolerance of an element, from the arithmetic: the angle is exact to 2^-32 turns and rounded once to
fp32 (2^-24 of at most pi), cosine and sine are good to 2 units in the last place, and a rotation
adds two rounded products: together below 16 * 2^-24 of mscale (|a| + |b|).  bf16 outputs are rounded
once more: 2^-8 of the value."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import plain
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


# ------------------------------------------------------------------ frequencies (CPU)

@pytest.mark.parametrize("R", [2, 4, 36, 64, 128])
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_freqs_match_the_formula(R, scaling):
    kw = {} if scaling is None else dict(scaling=scaling, factor=8.0)
    got = lidx.lidx_rope_freqs(R, 50000.0, device="cpu", **kw).numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = plain.rope_omega(R, 50000.0, **kw) / plain.TWO_PI
    # pow of two maths libraries: a few units in the last place; the fixed point rounds at 2^-65
    assert np.all(np.abs(got - want) <= 2.0 ** -48 * want + 2.0 ** -64)
    if scaling == "yarn" and R == 128:
        raw = plain.rope_omega(R, 50000.0) / plain.TWO_PI
        assert abs(got[0] - raw[0]) < 1e-12 and abs(got[-1] - raw[-1] / 8.0) < 1e-12


def test_freqs_refusals():
    L = lidx.lib()
    buf = (C.c_uint64 * 512)()
    ok = dict(R=64, theta=1e4, scaling=0, factor=1.0, L0=4096.0, bf=32.0, bs=1.0)

    def call(**kw):
        a = {**ok, **kw}
        return L.lidx_rope_freqs(a["R"], a["theta"], a["scaling"], a["factor"], a["L0"], a["bf"], a["bs"],
                                 kw.get("out", C.cast(buf, C.c_void_p)))

    assert call() == 0
    assert call(out=None) == 1
    for bad in (dict(R=0), dict(R=3), dict(R=1026), dict(theta=1.0), dict(theta=math.nan), dict(scaling=4),
                dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.inf),
                dict(scaling=3, factor=2.0, L0=0.0), dict(scaling=3, factor=2.0, bf=1.0),
                dict(scaling=3, factor=2.0, bf=math.inf)):
        assert call(**bad) == 2, bad


def test_rope_refusals_without_gpu():
    L = lidx.lib()
    ps = (C.c_int64 * 2)(1, 1)

    def call(nt=1, x=16, y=16, H=2, pos=16, freqs=16, T0=1, T1=1, D=64, R=32, off=0, layout=0, inv=0, m=1.0, dt=1,
             null_strides=False):
        t = (lidx._RopeTensor * 2)()
        for a in t:
            a.x, a.y, a.H = x, y, H
        return L.lidx_rope(t, nt, C.c_void_p(pos), None if null_strides else ps, C.c_void_p(freqs), T0, T1, D, R,
                           off, layout, inv, m, dt, None)

    assert call(x=None) == 1 and call(y=None) == 1 and call(pos=None) == 1 and call(freqs=None) == 1
    assert call(null_strides=True) == 1
    for bad in (dict(nt=0), dict(nt=3), dict(H=0), dict(T0=0), dict(T1=0), dict(T0=1 << 20, T1=1 << 20), dict(D=0),
                dict(D=63), dict(D=2048), dict(R=0), dict(R=33), dict(R=66), dict(off=-2), dict(off=34),
                dict(layout=2), dict(inv=2), dict(dt=2), dict(m=math.inf)):
        assert call(**bad) == 2, bad
    assert call(x=17) == 3 and call(dt=0, y=18) == 3 and call(pos=18) == 3 and call(freqs=20) == 3


# ------------------------------------------------------------------ GPU

def _close(got, want, x, m, what):
    x = np.abs(x.double().cpu().numpy())
    amp = np.abs(m) * 2 * x.max(-1, keepdims=True)  # bounds |a| + |b| of every pair
    tol = 16 * 2.0 ** -24 * np.maximum(amp, x)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{what}: {np.max(err - tol):.3e} over"


CASES = [
    # T0, T1, H, H2, D, R, off
    (1, 1, 1, 0, 16, 16, 0),
    (3, 5, 4, 1, 64, 64, 0),
    (2, 7, 3, 2, 128, 64, 64),
    (1, 33, 20, 4, 80, 36, 44),
    (1, 9, 2, 0, 48, 2, 7),       # a rotated part that no vector fits
    (5, 1, 64, 8, 128, 128, 0),
    (1, 300, 1, 0, 128, 64, 0),
    (1, 2, 130, 130, 32, 16, 8),
    (1, 3, 1, 1, 1024, 1024, 0),
    (2, 3, 5, 0, 6, 4, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T0,T1,H,H2,D,R,off", CASES)
def test_against_the_definition(T0, T1, H, H2, D, R, off, layout, dtype):
    g = np.random.default_rng(T1 * 31 + D)
    x = torch.from_numpy(g.standard_normal((T0, T1, H, D))).to(dtype)
    x2 = torch.from_numpy(g.standard_normal((T0, T1, H2, D))).to(dtype) if H2 else None
    # positions to both ends of int32: the reduction is exact everywhere
    pos = g.integers(0, 200000, (T0, T1)).astype(np.int32)
    pos.flat[0] = 2 ** 31 - 1
    if pos.size > 2:
        pos.flat[1], pos.flat[2] = -2 ** 31, -17
    m = 1.3466
    freqs = lidx.lidx_rope_freqs(R, scaling="yarn", factor=32.0)
    # the definition with the fixed-point frequencies: 2^31 positions of a frequency rounded at 2^-65
    # are 2^-34 turns off, below the tolerance; pow's last places are kept out by taking them from it
    om = freqs.cpu().numpy().view(np.uint64)
    turns = [[[(int(p) * int(f)) % 2 ** 64 / 2.0 ** 64 for f in om] for p in row] for row in pos]
    unit = np.array(turns)

    def want(t, inverse):
        # pos = 1 and omega = the reduced angle of each token
        y = np.empty(t.shape)
        for i in range(T0):
            for j in range(T1):
                y[i, j] = plain.rope(t[i:i + 1, j:j + 1], [[1]], plain.TWO_PI * unit[i, j], layout, off, m, inverse)[0, 0]
        return y

    p = torch.from_numpy(pos).to(DEV)
    for inverse, call in ((False, lidx.lidx_rope), (True, lidx.lidx_rope_bwd)):
        got = call(x.to(DEV), p, freqs, x2=None if x2 is None else x2.to(DEV), layout=layout, rot_off=off, mscale=m)
        got = got if H2 else (got,)
        for y, t in zip(got, (x, x2)):
            _close(y, want(t, inverse), t, m, f"inverse={inverse}")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_strides_broadcast_in_place_and_streams(layout):
    """A slice of a fused projection, transposed token axes, one position for the whole batch, in place,
    on a stream of its own: the same bits as the plain contiguous call."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T0, T1, H, D, R = 3, 11, 6, 64, 32
    freqs = lidx.lidx_rope_freqs(R)
    fused = torch.randn(T1, T0, H + 3, D + 8, generator=g, device=DEV).to(torch.bfloat16)
    x = fused.transpose(0, 1)[:, :, 1:1 + H, :D]
    pos = torch.arange(100, 100 + T1, dtype=torch.int32, device=DEV)
    want = lidx.lidx_rope(x.contiguous(), pos.expand(T0, T1).contiguous(), freqs, layout=layout, rot_off=8)
    assert torch.equal(lidx.lidx_rope(x, pos, freqs, layout=layout, rot_off=8), want)
    odd = fused.transpose(0, 1)[:, :, 1:1 + H, 3:3 + D]  # not aligned to 16 bytes
    want_odd = lidx.lidx_rope(odd.contiguous(), pos, freqs, layout=layout, rot_off=8)
    assert torch.equal(lidx.lidx_rope(odd, pos, freqs, layout=layout, rot_off=8), want_odd)
    before = fused.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lidx.lidx_rope(x, pos, freqs, layout=layout, rot_off=8, out=x, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(x, want)
    rest = torch.ones(fused.shape, dtype=torch.bool, device=DEV)
    rest.transpose(0, 1)[:, :, 1:1 + H, :D] = False
    assert torch.equal(fused[rest], before[rest])  # nothing beside the heads is written


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradient_against_differences(layout):
    """The map is linear: <g, rope(x + e) - rope(x - e)> / 2 = <rope_bwd(g), e>, in fp32 to the forward
    tolerance of both sides (16 * 2^-24 an element, D elements of size about 1)."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    T, H, D, R = 6, 3, 32, 24
    freqs = lidx.lidx_rope_freqs(R)
    pos = torch.randint(0, 5000, (1, T), generator=gen, device=DEV).to(torch.int32)
    x, e, g = (torch.randn(1, T, H, D, generator=gen, device=DEV) for _ in range(3))
    kw = dict(layout=layout, rot_off=8, mscale=1.25)
    d = (lidx.lidx_rope(x + e, pos, freqs, **kw).double() - lidx.lidx_rope(x - e, pos, freqs, **kw).double()) / 2
    left = (g.double() * d).sum((2, 3))
    right = (lidx.lidx_rope_bwd(g, pos, freqs, **kw).double() * e.double()).sum((2, 3))
    size = (g.abs().double().amax() * (x.abs() + e.abs()).double().amax() * H * D).item()
    assert (left - right).abs().max().item() <= 4 * 16 * 2.0 ** -24 * size


@pytest.mark.gpu
def test_binding_refusals():
    freqs = lidx.lidx_rope_freqs(16)
    x = torch.zeros(1, 2, 1, 32, device=DEV)
    pos = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        lidx.lidx_rope(x.half(), pos, freqs)
    with pytest.raises(TypeError):
        lidx.lidx_rope(x, pos.long(), freqs)
    with pytest.raises(TypeError):
        lidx.lidx_rope(x, pos, freqs.float())
    with pytest.raises(ValueError):
        lidx.lidx_rope(x[0], pos, freqs)
    with pytest.raises(ValueError):
        lidx.lidx_rope(x, pos, freqs, layout="other")
    with pytest.raises(lidx.LidxError):
        lidx.lidx_rope(x.transpose(2, 3), pos, freqs)  # one dim a head
    with pytest.raises(ValueError):
        lidx.lidx_rope(torch.zeros(1, 2, 32, 3, device=DEV).transpose(2, 3), pos, freqs)
    with pytest.raises(ValueError):
        lidx.lidx_rope(x, pos, freqs, x2=x[:, :1])
    with pytest.raises(ValueError):
        lidx.lidx_rope(x, pos, freqs, out=x[:, :1])
    with pytest.raises(lidx.LidxError):
        lidx.lidx_rope(x, pos, freqs, rot_off=20)  # [20, 36) of 32 dims
