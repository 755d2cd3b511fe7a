"""Writing into the paged caches with the norm and the rotation of the keys on the way (lidx_rope_cache_append,
lidx_cache4_append), and a 4-bit cache as an 8-bit one (lidx_cache4_to_8).

Without a norm and a rotation codes, exponents and scales are whole results of exact divisions by powers of two: they are
equal bit for bit.  With them a key is off by 48 * 2^-24 of its pair (as for lidx_norm_rope) before it is rounded: the
number held may be as far from the exact key as the nearest number of its scale, and twice that more; a scale or an
exponent may differ where the largest size lies that near to a border (relative 2^-17)."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import plain
import plain4
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_norm_rope import U, angles, norm, pair_size, turn

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


# ------------------------------------------------------------------ CPU

def test_refusals_without_gpu():
    L = lidx.lib()
    P = lambda v: None if v is None else C.c_void_p(v)
    st, odd = (C.c_int64 * 3)(64, 64, 64), (C.c_int64 * 3)(64, 4, 64)

    def call(bits, k=16, v=16, ks=st, vs=st, w=None, wdt=0, eps=1e-6, table=16, start=16, count=None, B=1, S=1, H=1, D=64,
             page=16, MP=1, NP=1, kc=16, vc=16, ke=16, ve=16, ksc=16, vsc=16, turn=True, pos=16, freqs=16, axis=None, axes=1,
             R=32, off=0, layout=0, m=1.0):
        r = lidx._RopeTurn(pos, (C.c_int64 * 3)(1, 1, 1), freqs, axis, axes, R, off, layout, m)
        head = [P(k), P(v), ks, vs, C.byref(r) if turn else None, P(w), wdt, eps, P(table), P(start), P(count), B, S, H, D, page,
                MP, NP, P(kc), P(vc)]
        if bits == 8:
            return L.lidx_rope_cache_append(*head, P(ksc), P(vsc), None)
        return L.lidx_cache4_append(*head, P(ke), P(ve), P(ksc), P(vsc), None)

    for bits in (4, 8):
        for name in ("k", "v", "ks", "vs", "table", "start", "kc", "vc", "ksc", "vsc", "freqs"):
            assert call(bits, **{name: None}) == 1, name
        for bad in (dict(B=0), dict(S=0), dict(H=0), dict(D=8), dict(D=72), dict(D=144), dict(page=8), dict(page=48),
                    dict(MP=0), dict(NP=0), dict(MP=1 << 30), dict(NP=1 << 30), dict(B=1 << 20, S=1 << 20), dict(R=0),
                    dict(R=33), dict(R=66), dict(off=34), dict(layout=2), dict(m=math.inf), dict(axes=2), dict(axes=256),
                    dict(w=16, eps=-1.0), dict(w=16, eps=math.nan), dict(w=16, wdt=2)):
            assert call(bits, **bad) == 2, bad
        for bad in (dict(k=24), dict(v=24), dict(kc=8), dict(vc=8), dict(ks=odd), dict(vs=odd), dict(table=18), dict(start=18),
                    dict(count=18), dict(ksc=18), dict(w=18), dict(w=17, wdt=1), dict(pos=18), dict(freqs=20)):
            assert call(bits, **bad) == 3, bad
    assert call(8, turn=False) == 1
    assert call(4, ke=None) == 1 and call(4, ve=None) == 1 and call(4, ke=18) == 3
    wide = lambda kc=16, vc=16, ke=16, ve=16, H=1, D=64, page=16, NP=1, k8=16, v8=16: L.lidx_cache4_to_8(
        P(kc), P(vc), P(ke), P(ve), H, D, page, NP, P(k8), P(v8), None)
    for name in ("kc", "vc", "ke", "ve", "k8", "v8"):
        assert wide(**{name: None}) == 1
    for bad in (dict(H=0), dict(D=24), dict(page=17), dict(NP=0)):
        assert wide(**bad) == 2
    assert wide(kc=8) == 3 and wide(k8=8) == 3 and wide(ke=18) == 3


def test_plain_rounding():
    """The definition's own rounding: every border goes to the even code, everything else to the nearer number."""
    x = np.array([0, 0.25, 0.26, 0.5, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7.0])
    want = [0, 0, 1, 1, 2, 1, 2, 3, 4, 4, 5, 6, 6, 7, 7]
    assert plain4.code4(x).tolist() == want and plain4.code4(-x[1:]).tolist() == [w | 8 for w in want[1:]]
    g = np.random.default_rng(0)
    codes, words, _ = plain4.random_cache(g, 2, 1, 16, 80)
    assert np.array_equal(plain4.pack(plain4.unpack(codes)), codes)
    assert np.array_equal(plain4.pack_exps(plain4.exps_of(words, 80)), words)
    # every number of every exponent is an e4m3 number of 32 times the scale
    every = np.arange(16, dtype=np.uint8)[None].repeat(12, 0)
    plain4.as_8(plain4.pack(every), np.arange(12, dtype=np.int32))


# ------------------------------------------------------------------ GPU

CASES = [
    # B, S, Hkv, D, page, starts, counts (None: S)
    (1, 1, 1, 16, 16, [0], None),
    (1, 1, 2, 128, 64, [63], None),              # the last slot of a page
    (2, 1, 8, 128, 128, [128, 5], None),         # a fresh page; a page with tokens
    (3, 5, 4, 80, 16, [14, 0, 31], [5, 0, 4]),   # across a page border; nothing; ragged
    (2, 40, 3, 64, 16, [7, 16], [40, 33]),
    (1, 300, 1, 112, 128, [100], None),
    (2, 129, 2, 128, 128, [0, 127], [129, 2]),
    (4, 3, 1, 48, 32, [-2, 125, 1000, 30], [3, 3, 3, -5]),  # before 0, past the table, negative counts
]


def _setup(B, S, Hkv, D, page, starts, counts, bits, spread, seed):
    g = np.random.default_rng(seed)
    MP = max(2, (min(max(starts), 400) + S) // page + 1) if max(starts) < 1000 else 4
    NP = B * MP + 3
    table = g.permutation(NP)[:B * MP].reshape(B, MP).astype(np.int32)
    if B > 2:
        table[0, 0] = NP       # an id out of range: its tokens are dropped
        table[2, -1] = -1
    size = np.exp(3 * g.standard_normal((B, S, Hkv, 1))) if spread else 1.0
    k, v = (torch.from_numpy(g.standard_normal((B, S, Hkv, D)) * size).to(torch.bfloat16) for _ in (0, 1))
    if bits == 4:
        sides = [list(plain4.random_cache(g, NP, Hkv, page, D)), list(plain4.random_cache(g, NP, Hkv, page, D, -22, -18))]
    else:
        sides = [list(plain.random_cache(g, NP, Hkv, page, D)), list(plain.random_cache(g, NP, Hkv, page, D, -14, -12))]
    return g, table, k, v, sides, [S] * B if counts is None else counts


def _cuda(side, bits):
    t = [torch.from_numpy(a.copy()).to(DEV) for a in side]
    return [t[0].view(torch.float8_e4m3fn)] + t[1:] if bits == 8 else t


def _numpy(t):
    return (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).cpu().numpy()


def _call(bits, k, v, kd, vd, table, starts, counts, **kw):
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)
    rest = (i32(table), i32(starts))
    kw = dict(count=i32(counts), **kw)
    if bits == 8:
        lidx.lidx_rope_cache_append(k, v, kw.pop("freqs"), kd[0], vd[0], kd[1], vd[1], *rest, **kw)
    else:
        lidx.lidx_cache4_append(k, v, kd[0], vd[0], kd[1], vd[1], kd[2], vd[2], *rest, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("B,S,Hkv,D,page,starts,counts", CASES)
def test_four_bits_against_the_definition(B, S, Hkv, D, page, starts, counts, spread):
    g, table, k, v, sides, cnt = _setup(B, S, Hkv, D, page, starts, counts, 4, spread, S + D + page)
    if S * Hkv >= 2:
        v[0, -1] = 0
    if S >= 3:  # at the borders of a scale, an exponent and a code, and below all of them
        k[0, 0, 0, 0], k[0, 1, 0, 0], k[0, 2, 0, 0], k[0, 2, 0, 1] = 12288.0, -12352.0, 2.0 ** -60, 5.0
        k[0, 1, -1, :16] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 2).bfloat16()
    kd, vd = (_cuda(s, 4) for s in sides)
    _call(4, k.to(DEV), v.to(DEV), kd, vd, table, starts, cnt)
    for x, s in ((k, sides[0]), (v, sides[1])):
        plain4.append(x.double().numpy(), *s, table, starts, cnt)
    for got, want, name in zip(kd + vd, sides[0] + sides[1], ("k", "k_exps", "k_scale", "v", "v_exps", "v_scale")):
        got = _numpy(got)
        assert np.array_equal(got, want), f"{name}: {np.argwhere(got != want)[:4]}"


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hkv,D,page,starts,counts", CASES)
def test_eight_bits_without_a_turn_are_the_plain_call(B, S, Hkv, D, page, starts, counts):
    """Frequencies of zero turn nothing: bit for bit lidx_cache_append."""
    g, table, k, v, sides, cnt = _setup(B, S, Hkv, D, page, starts, counts, 8, True, 7 * S + D)
    a, b = [_cuda(s, 8) for s in sides], [_cuda(s, 8) for s in sides]
    freqs = torch.zeros(D // 2, dtype=torch.int64, device=DEV)
    _call(8, k.to(DEV), v.to(DEV), *a, table, starts, cnt, freqs=freqs)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    lidx.lidx_cache_append(k.to(DEV), v.to(DEV), b[0][0], b[1][0], b[0][1], b[1][1], i32(table), i32(starts), count=i32(cnt))
    for x, y in zip(a[0] + a[1], b[0] + b[1]):
        assert np.array_equal(_numpy(x), _numpy(y))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("normed,A,given", [(False, 1, False), (True, 1, True), (True, 3, True), (False, 2, True)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_turned_keys_against_the_definition(case, bits, normed, A, given, layout):
    B, S, Hkv, D, page, starts, counts = CASES[case]
    g, table, k, v, sides, cnt = _setup(B, S, Hkv, D, page, starts, counts, bits, False, 31 * S + D + case)
    # rotated parts of whole groups, of half groups, of single pairs at an odd offset
    R, off = [(D, 0), (D // 2, D // 2), (D // 2 - 2, 3)][case % 3]
    w = torch.from_numpy(1 + 0.3 * g.standard_normal(D)).to(torch.bfloat16) if normed else None
    pos = g.integers(0, 200000, (A, B, S)).astype(np.int32)
    if not given:
        pos = (np.asarray(starts)[:, None] + np.arange(S))[None].astype(np.int32)
    freqs = lidx.lidx_rope_freqs(R)
    axes = torch.arange(R // 2).remainder(A).to(torch.uint8).to(DEV) if A > 1 else None
    ang = angles(freqs, pos, None if axes is None else axes.cpu().numpy())
    kd, vd = (_cuda(s, bits) for s in sides)
    before = [s[0].copy() for s in sides]
    p = torch.from_numpy(pos).to(DEV)
    _call(bits, k.to(DEV), v.to(DEV), kd, vd, table, starts, cnt, freqs=freqs, pos=(p if A > 1 else p[0]) if given else None,
          weight=None if w is None else w.to(DEV), eps=1e-5, layout=layout, rot_off=off, mscale=1.25, axes=axes)
    n = k.double().numpy()
    if normed:
        n = norm(n, w.double().numpy(), 1e-5)[0]
    want = turn(n, ang, R, off, layout, 1.25, False)
    tol = 48 * U * pair_size(n, R, off, layout, 1.25)
    # values are as without a turn
    (plain4 if bits == 4 else plain).append(v.double().numpy() if bits == 4 else v, *sides[1], table, starts, cnt)
    assert all(np.array_equal(_numpy(a), b) for a, b in zip(vd, sides[1]))
    got = [_numpy(a) for a in kd]
    scale0, scale = sides[0][-1], got[-1]
    touched = np.zeros(got[0].shape[:3], bool)
    limit = 448.0 if bits == 8 else 6.0 * 2.0 ** 11
    for b in range(B):
        for i in range(min(max(cnt[b], 0), S)):
            at = starts[b] + i
            if at < 0 or at // page >= table.shape[1] or not 0 <= table[b, at // page] < len(scale):
                continue
            j, pid = at // page, table[b, at // page]
            for h in range(Hkv):
                touched[pid, h] = True
                first = max(0, j * page - starts[b])
                new = [t for t in range(first, min(cnt[b], S)) if 0 <= starts[b] + t and (starts[b] + t) // page == j]
                top = np.abs(want[b, new, h]).max()
                allowed = [2.0 ** plain4.smallest(top * f, limit, -40) for f in (1 - 2.0 ** -17, 1 + 2.0 ** -17)]
                if j * page < starts[b]:
                    allowed = [max(a, scale0[pid, h]) for a in allowed]
                s = float(scale[pid, h])
                assert s in allowed, (b, i, h)
                y, t = want[b, i, h], tol[b, i, h]
                if bits == 8:
                    held = plain.E4M3[got[0][pid, h, at % page]] * s
                    best = plain.E4M3[plain.e4m3_round(y / s)] * s
                else:
                    e = plain4.exps_of(got[1][pid, h, at % page], D)
                    tops = np.abs(y).reshape(-1, 16).max(-1) / s
                    for q in range(D // 16):
                        assert min(11, max(0, plain4.smallest(tops[q] * (1 - 2.0 ** -17), 6.0, 0))) <= e[q] <= min(
                            11, plain4.smallest(tops[q] * (1 + 2.0 ** -17), 6.0, 0))
                    f = s * 2.0 ** np.repeat(e, 16)
                    held = plain4.numbers(got[0][pid, h, at % page], got[1][pid, h, at % page]) * s
                    c = plain4.code4(y / f)
                    best = plain4.E2M1[c & 7] * np.where(c & 8, -1, 1) * f
                assert (np.abs(held - y) <= np.abs(best - y) + 2 * t).all(), (b, i, h)
    assert np.array_equal(got[0][~touched], before[0][~touched])  # other pages are left as they were
    assert np.array_equal(scale[~touched.any(2)], scale0[~touched.any(2)])


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,Hkv,S", [(128, 128, 8, 300), (80, 64, 5, 200), (64, 16, 3, 40), (16, 16, 1, 3)])
def test_norm_alone_and_blocks_of_several_heads(D, page, Hkv, S):
    """A norm without a rotation is that with frequencies of zero (cosines of 1, sines of 0: exact), and a call of many heads
    and tokens, whose blocks take several heads, holds what calls of one head each hold."""
    starts, cnt = [5, 0, 2 * page], [S, S - 2, S]
    g, table, k, v, sides, _ = _setup(3, S, Hkv, D, page, starts, cnt, 4, True, D)
    table = g.permutation(table.size).reshape(table.shape).astype(np.int32)
    w = torch.from_numpy(1 + 0.3 * g.standard_normal(D)).float().to(DEV)
    a, b, c = ([_cuda(s, 4) for s in sides] for _ in range(3))
    zero = torch.zeros(D // 2, dtype=torch.int64, device=DEV)
    k, v = k.to(DEV), v.to(DEV)
    _call(4, k, v, *a, table, starts, cnt, weight=w)
    _call(4, k, v, *b, table, starts, cnt, weight=w, freqs=zero)
    for x, y in zip(a[0] + a[1], b[0] + b[1]):
        assert torch.equal(x, y)
    freqs = lidx.lidx_rope_freqs(D)
    _call(4, k, v, *b, table, starts, cnt, weight=w, freqs=freqs, layout="half")
    for h in range(Hkv):
        one = [[t[:, h:h + 1].contiguous() for t in side] for side in c]
        _call(4, k[:, :, h:h + 1], v[:, :, h:h + 1], *one, table, starts, cnt, weight=w)
        _call(4, k[:, :, h:h + 1], v[:, :, h:h + 1], *one, table, starts, cnt, weight=w, freqs=freqs, layout="half")
        for x, y in zip(b[0] + b[1], one[0] + one[1]):
            assert torch.equal(x[:, h:h + 1], y)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_infinities_and_nan(bits):
    """They read as NaN (in 4 bits their group does), change no scale and nothing else; a key's partner in the turn is NaN,
    too: b cos + a sin with an infinity a is NaN even where the sine is 0."""
    g, table, k, v, sides, cnt = _setup(2, 40, 2, 64, 32, [5, 32], [40, 33], bits, False, 3)
    a = [_cuda(s, bits) for s in sides]
    b = [_cuda(s, bits) for s in sides]
    freqs = torch.zeros(32, dtype=torch.int64, device=DEV)
    k, v = k.clone(), v.clone()
    k[0, 1, 0, 20], v[0, 3, 1, 63], v[1, 30, 0, 0] = 0.0, 0.0, 0.0
    _call(bits, k.to(DEV), v.to(DEV), *a, table, [5, 32], cnt, freqs=freqs)
    bad = [(0, 0, 1, 0, 20, float("inf")), (1, 0, 3, 1, 63, float("nan")), (1, 1, 30, 0, 0, float("-inf"))]
    for which, bb, i, h, d, val in bad:
        (k, v)[which][bb, i, h, d] = val
    _call(bits, k.to(DEV), v.to(DEV), *b, table, [5, 32], cnt, freqs=freqs)
    for which in (0, 1):
        x, y = [_numpy(t) for t in a[which]], [_numpy(t) for t in b[which]]
        assert np.array_equal(x[-1], y[-1])
        num = (lambda z: plain.E4M3[z[0]]) if bits == 8 else (lambda z: plain4.numbers(z[0], z[1]))
        nx, ny = num(x), num(y)
        off = np.zeros(nx.shape, bool)
        for w, bb, i, h, d, _ in bad:
            if w == which:
                at = (5, 32)[bb] + i
                lane = slice(d - d % 2 * (w == 0), d + 1 + (d + 1) % 2 * (w == 0)) if bits == 8 else slice(d // 16 * 16, d // 16 * 16 + 16)
                off[table[bb, at // 32], h, at % 32, lane] = True
        assert np.isnan(ny[off]).all() and np.array_equal(nx[~off], ny[~off])


@pytest.mark.gpu
def test_norm_of_a_row_that_is_not_finite():
    g, table, k, v, sides, cnt = _setup(1, 3, 2, 64, 16, [0], None, 8, False, 4)
    kd, vd = (_cuda(s, 8) for s in sides)
    k[0, 1, 1, 7] = float("nan")
    _call(8, k.to(DEV), v.to(DEV), kd, vd, table, [0], cnt, freqs=lidx.lidx_rope_freqs(64), weight=torch.ones(64, device=DEV))
    held = plain.E4M3[_numpy(kd[0])[table[0, 0]]]
    assert np.isnan(held[1, 1]).all() and not np.isnan(held[0]).any() and not np.isnan(held[1, [0, 2]]).any()


@pytest.mark.gpu
def test_norm_of_a_row_with_an_infinity():
    """Its pair is NaN, the rest of the key 0; nothing else differs."""
    g, table, k, v, sides, cnt = _setup(1, 3, 2, 64, 16, [0], None, 8, False, 4)
    a, b = ([_cuda(s, 8) for s in sides] for _ in (0, 1))
    kw = dict(freqs=lidx.lidx_rope_freqs(64), weight=torch.ones(64, device=DEV))
    k[0, 1, 1] = 0.0
    _call(8, k.to(DEV), v.to(DEV), *a, table, [0], cnt, **kw)
    k[0, 1, 1] = 1.0
    k[0, 1, 1, 7] = float("inf")
    _call(8, k.to(DEV), v.to(DEV), *b, table, [0], cnt, **kw)
    x, y = (plain.E4M3[_numpy(t[0][0])[table[0, 0]]] for t in (a, b))
    assert np.isnan(y[1, 1, 6:8]).all() and np.isnan(y).sum() == 2
    assert np.array_equal(np.nan_to_num(y), x)


@pytest.mark.gpu
def test_token_by_token_equals_at_once_in_four_bits():
    """Powers of two move exponents only, so a page filled token by token holds what it holds when filled at once, where no
    group falls below the lowest exponent: sizes here lie within 2^6 of each other.  The single calls read slices of a fused,
    transposed projection."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, S, Hkv, D, page = 2, 37, 2, 64, 16
    fused = torch.randn(S, B, 2 * Hkv + 1, D, generator=g, device=DEV)
    fused = (fused.sign() * (fused.abs() + 0.25) * torch.exp2(torch.randint(0, 4, (S, B, 1, 1), generator=g, device=DEV))).bfloat16()
    k, v = fused.transpose(0, 1)[:, :, :Hkv], fused.transpose(0, 1)[:, :, Hkv:2 * Hkv]
    table = torch.arange(B * 3, dtype=torch.int32, device=DEV).view(B, 3)

    def empty():
        new = lambda *s, dt=torch.uint8: [torch.zeros(B * 3, Hkv, *s, dtype=dt, device=DEV) for _ in (0, 1)]
        return new(page, D // 2) + new(page, dt=torch.int32) + new(dt=torch.float32)

    a, b = empty(), empty()
    lidx.lidx_cache4_append(k.contiguous(), v.contiguous(), *a, table, torch.zeros(B, dtype=torch.int32, device=DEV))
    for i in range(S):
        lidx.lidx_cache4_append(k[:, i:i + 1], v[:, i:i + 1], *b, table, torch.full((B,), i, dtype=torch.int32, device=DEV))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,Hkv", [(16, 16, 1), (80, 32, 3), (128, 128, 2)])
def test_as_an_eight_bit_cache(D, page, Hkv):
    g = np.random.default_rng(D)
    codes, words, _ = plain4.random_cache(g, 5, Hkv, page, D)
    codes2, words2 = codes[::-1].copy(), g.integers(-2 ** 31, 2 ** 31, words.shape).astype(np.int32)  # any exponents
    t = [torch.from_numpy(a).to(DEV) for a in (codes, codes2, words, words2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    k8, v8 = lidx.lidx_cache4_to_8(*t, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert np.array_equal(_numpy(k8), plain4.as_8(codes, words)) and np.array_equal(_numpy(v8), plain4.as_8(codes2, words2))


@pytest.mark.gpu
def test_binding_refusals():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)
    k = z(1, 1, 1, 32, dt=torch.bfloat16)
    ok = dict(k=k, v=k, k_cache=z(2, 1, 16, 16), v_cache=z(2, 1, 16, 16), k_exps=z(2, 1, 16, dt=torch.int32),
              v_exps=z(2, 1, 16, dt=torch.int32), k_scale=z(2, 1, dt=torch.float32), v_scale=z(2, 1, dt=torch.float32),
              block_table=z(1, 2, dt=torch.int32), start=z(1, dt=torch.int32))
    freqs, pos = lidx.lidx_rope_freqs(32), z(1, 1, dt=torch.int32)
    lidx.lidx_cache4_append(**ok)
    for bad in (dict(k=k.float()), dict(k_cache=z(2, 1, 16, 16, dt=torch.int8)), dict(k_exps=z(2, 1, 16)),
                dict(weight=z(32, dt=torch.float16)), dict(freqs=freqs, pos=pos.long()), dict(freqs=freqs.float()),
                dict(start=z(1, dt=torch.int64))):
        with pytest.raises(TypeError):
            lidx.lidx_cache4_append(**{**ok, **bad})
    for bad in (dict(v=k[..., :16]), dict(v_cache=z(2, 1, 16, 32)), dict(k_exps=z(2, 1, 8, dt=torch.int32)),
                dict(v_scale=z(1, 1, dt=torch.float32)), dict(weight=z(16, dt=torch.float32)), dict(pos=pos),
                dict(freqs=freqs, axes=z(16)), dict(freqs=freqs, layout="other"), dict(count=z(2, dt=torch.int32)),
                dict(freqs=freqs, pos=pos, axes=z(8))):
        with pytest.raises(ValueError):
            lidx.lidx_cache4_append(**{**ok, **bad})
    with pytest.raises(lidx.LidxError):
        lidx.lidx_cache4_append(**{**ok, "freqs": freqs, "rot_off": 2})
    c8 = z(2, 1, 16, 32).view(torch.float8_e4m3fn)
    sc = z(2, 1, dt=torch.float32)
    with pytest.raises(TypeError):
        lidx.lidx_rope_cache_append(k, k, None, c8, c8.clone(), sc, sc.clone(), ok["block_table"], ok["start"])
    with pytest.raises(TypeError):
        lidx.lidx_rope_cache_append(k, k, freqs, ok["k_cache"], c8, sc, sc.clone(), ok["block_table"], ok["start"])
