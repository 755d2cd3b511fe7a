"""Writing into the paged 8-bit cache (lidx_cache_append) against its definition: codes and scales are
whole results, so they must be equal bit for bit."""

import ctypes as C

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


def test_refusals_without_gpu():
    L = lidx.lib()
    P = lambda v: None if v is None else C.c_void_p(v)
    st = (C.c_int64 * 3)(64, 64, 64)
    odd = (C.c_int64 * 3)(64, 4, 64)

    def call(k=16, v=16, ks=st, vs=st, table=16, start=16, count=None, B=1, S=1, H=1, D=64, page=16, MP=1, NP=1, kc=16,
             vc=16, ksc=16, vsc=16):
        return L.lidx_cache_append(P(k), P(v), ks, vs, P(table), P(start), P(count), B, S, H, D, page, MP, NP, P(kc),
                                   P(vc), P(ksc), P(vsc), None)

    for name in ("k", "v", "ks", "vs", "table", "start", "kc", "vc", "ksc", "vsc"):
        assert call(**{name: None}) == 1, name
    for bad in (dict(B=0), dict(S=0), dict(H=0), dict(D=8), dict(D=72), dict(D=144), dict(page=8), dict(page=48),
                dict(page=256), dict(MP=0), dict(NP=0), dict(MP=1 << 30), dict(NP=1 << 30),
                dict(B=1 << 20, S=1 << 20)):
        assert call(**bad) == 2, bad
    for bad in (dict(k=24), dict(v=24), dict(kc=8), dict(vc=8), dict(ks=odd), dict(vs=odd), dict(table=18),
                dict(start=18), dict(count=18), dict(ksc=18)):
        assert call(**bad) == 3, bad


def test_plain_rounding_agrees_with_torch():
    """The definition's own rounding, pinned to another implementation."""
    x = torch.cat([torch.linspace(-460, 460, 40001), torch.randn(20000) * 0.01,
                   torch.from_numpy(plain.E4M3[:126] / 2 + plain.E4M3[1:127] / 2).float()])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(plain.e4m3_round(x.numpy().astype(np.float64)), want)


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


@pytest.mark.gpu
@pytest.mark.parametrize("with_spread", [False, True])
@pytest.mark.parametrize("B,S,Hkv,D,page,starts,counts", CASES)
def test_against_the_definition(B, S, Hkv, D, page, starts, counts, with_spread):
    g = np.random.default_rng(S + D + page)
    MP = max(2, (min(max(starts), 400) + S) // page + 1) if max(starts) < 1000 else 4
    NP = B * MP + 3
    table = g.permutation(NP)[:B * MP].reshape(B, MP).astype(np.int32)
    if B > 2:
        table[0, 0] = NP       # an id out of range: its tokens are dropped
        table[2, -1] = -1
    size = np.exp(3 * g.standard_normal((B, S, Hkv, 1))) if with_spread else 1.0
    k = torch.from_numpy(g.standard_normal((B, S, Hkv, D)) * size).to(torch.bfloat16)
    v = torch.from_numpy(g.standard_normal((B, S, Hkv, D)) * size).to(torch.bfloat16)
    # amounts at the borders of a scale: zero, exactly 448, just above it, the smallest scale's reach
    if S * Hkv >= 2:
        v[0, -1] = 0
    if S >= 3:
        k[0, 0, 0, 0], k[0, 1, 0, 0], k[0, 2, 0, 0] = 448.0, -450.0, 2.0 ** -60
    kc, ksc = plain.random_cache(g, NP, Hkv, page, D)
    vc, vsc = plain.random_cache(g, NP, Hkv, page, D, -14, -12)  # most pages outgrow this
    kc[:, :, :, 0] = 0x7F  # NaN codes stay what they are when nothing moves them
    cnt = [S] * B if counts is None else counts
    got = [plain.to_cuda(kc), plain.to_cuda(vc), torch.from_numpy(ksc).to(DEV), torch.from_numpy(vsc).to(DEV)]
    kc[:, :, :, 0] = 0
    got[0].view(torch.uint8)[:, :, :, 0] = 0
    lidx.lidx_cache_append(k.to(DEV), v.to(DEV), *got, torch.from_numpy(table).to(DEV),
                           torch.tensor(starts, dtype=torch.int32, device=DEV),
                           count=None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV))
    plain.append(k, kc, ksc, table, starts, cnt)
    plain.append(v, vc, vsc, table, starts, cnt)
    for t, w, name in zip(got, (kc, vc, ksc, vsc), ("k", "v", "k_scale", "v_scale")):
        t = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).cpu().numpy()
        assert np.array_equal(t, w), f"{name}: {np.argwhere(t != w)[:4]}"


@pytest.mark.gpu
def test_token_by_token_equals_at_once_and_strides():
    """With powers of two a growing scale moves exponents only, so a page filled token by token holds
    what it holds when filled at once (no value here falls among the subnormals of the final scale).
    The token-by-token calls read slices of a fused, transposed projection."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, S, Hkv, D, page = 2, 37, 2, 64, 16
    fused = torch.randn(S, B, 2 * Hkv + 1, D, generator=g, device=DEV)
    fused = (fused.sign() * (fused.abs() + 0.25)).to(torch.bfloat16)
    k, v = fused.transpose(0, 1)[:, :, :Hkv], fused.transpose(0, 1)[:, :, Hkv:2 * Hkv]
    table = torch.arange(B * 3, dtype=torch.int32, device=DEV).view(B, 3)

    def empty():
        return [torch.zeros(B * 3, Hkv, page, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in (0, 1)] \
            + [torch.zeros(B * 3, Hkv, device=DEV) for _ in (0, 1)]

    a, b = empty(), empty()
    lidx.lidx_cache_append(k.contiguous(), v.contiguous(), *a, table, torch.zeros(B, dtype=torch.int32, device=DEV))
    for i in range(S):
        lidx.lidx_cache_append(k[:, i:i + 1], v[:, i:i + 1], *b, table,
                               torch.full((B,), i, dtype=torch.int32, device=DEV))
    for x, y in zip(a, b):
        x, y = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (x, y))
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_binding_refusals():
    kc = torch.zeros(2, 1, 16, 16, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    sc = torch.ones(2, 1, device=DEV)
    k = torch.zeros(1, 1, 1, 16, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    ok = (k, k, kc, kc.clone(), sc, sc.clone(), table, start)

    def but(i, t):
        return ok[:i] + (t,) + ok[i + 1:]

    with pytest.raises(TypeError):
        lidx.lidx_cache_append(*but(0, k.float()))
    with pytest.raises(TypeError):
        lidx.lidx_cache_append(*but(2, kc.view(torch.uint8)))
    with pytest.raises(ValueError):
        lidx.lidx_cache_append(*but(1, k[:, :, :, :8]))
    with pytest.raises(ValueError):
        lidx.lidx_cache_append(*but(4, sc[:1]))
    with pytest.raises(TypeError):
        lidx.lidx_cache_append(*but(6, table.long()))
    with pytest.raises(ValueError):
        lidx.lidx_cache_append(*but(7, torch.zeros(2, dtype=torch.int32, device=DEV)))
    with pytest.raises(ValueError):
        lidx.lidx_cache_append(*ok, count=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(lidx.LidxError):  # a page of 8 slots
        c8 = kc.view(torch.uint8)[:, :, :8].contiguous().view(torch.float8_e4m3fn)
        lidx.lidx_cache_append(k, k, c8, c8.clone(), sc, sc.clone(), table, start)
