"""Attention over the paged 4-bit cache (lidx_cache4_attn) against its 64-bit definition.

code * 2^x * scale is e4m3 code * (32 scale) exactly, so the definition and the derivation of its tolerances are those of the
8-bit cache (plain.attention), on the cache's 8-bit form.  One term is added, since the groups of these caches differ by up
to 2^11: a weight below 2^-14 of its tile's largest, 2^8, lies among the lower half's subnormals, whose step is 2^-9; it is off
by 2^-10, 2^-18 of the largest weight, and the sum of all weights is at least that weight.  plain.attention counts that once, for
the largest value; every key may be off by as much, so a dim by 2^-18 sum_t |v_t|.  The kernels
widen the codes to that form and go on as the 8-bit ones; units of up to 32 rows add the products of a row's two parts
after them, not in them.  Either call is within the tolerance of the definition, so they are within twice that of each other.
On random inputs the error of a whole output stays below 5e-3 of its norm as there."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import plain
import plain4
import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


def _status_ok():
    torch.cuda.synchronize()
    assert lidx.lidx_device_status() == 0


def test_refusals_without_gpu():
    L = lidx.lib()
    P = lambda v: None if v is None else C.c_void_p(v)
    st, odd = (C.c_int64 * 3)(64, 64, 64), (C.c_int64 * 3)(64, 4, 64)

    def call(q=16, qs=st, kc=16, vc=16, ke=16, ve=16, ksc=16, vsc=16, table=16, lens=16, pos=None, idx=None, B=1, S=1, Hq=1,
             Hkv=1, D=64, page=16, MP=1, NP=1, ratio=1, topk=0, scale=1.0, out=16, lse=None, ws=None, wsb=0):
        return L.lidx_cache4_attn(P(q), qs, P(kc), P(vc), P(ke), P(ve), P(ksc), P(vsc), P(table), P(lens), P(pos), P(idx), B,
                                  S, Hq, Hkv, D, page, MP, NP, ratio, topk, scale, P(out), P(lse), P(ws), wsb, None)

    for name in ("q", "qs", "kc", "vc", "ke", "ve", "ksc", "vsc", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
    for bad in (dict(B=0), dict(S=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3, Hkv=2), dict(Hq=129), dict(D=8), dict(D=136),
                dict(D=256), dict(page=24), dict(MP=0), dict(NP=0), dict(NP=1 << 29), dict(ratio=0),
                dict(idx=16, topk=0), dict(idx=16, topk=(1 << 20) + 1), dict(scale=math.nan), dict(B=1 << 16, S=1 << 16)):
        assert call(**bad) == 2, bad
    for bad in (dict(q=24), dict(qs=odd), dict(kc=8), dict(vc=8), dict(out=8), dict(lens=18), dict(table=18), dict(ke=24), dict(ke=24),
                dict(ve=24), dict(pos=18), dict(idx=18, topk=1), dict(lse=18), dict(ksc=18), dict(vsc=18)):
        assert call(**bad) == 3, bad


# ------------------------------------------------------------------ GPU

class Case:
    """A 4-bit cache, its tables and queries on both sides."""

    def __init__(self, seed, B, S, Hq, Hkv, D, page, lens, q_scale=1.0, exps=(-13, -10), poison=True):
        g = np.random.default_rng(seed)
        self.g, self.page, self.D = g, page, D
        MP = max(1, max(-(-max(n, 1) // page) for n in lens))
        NP = B * MP + 2
        self.kc, self.ke, self.ks = plain4.random_cache(g, NP, Hkv, page, D, *exps)
        self.vc, self.ve, self.vs = plain4.random_cache(g, NP, Hkv, page, D, *exps)
        self.table = g.permutation(NP)[:B * MP].reshape(B, MP).astype(np.int32)
        self.lens = np.asarray(lens, np.int32)
        if poison:
            # every slot past a sequence's length reads as NaN, and so do pages of nobody
            used = np.zeros((NP, page), bool)
            for b, n in enumerate(lens):
                for t in range(min(n, MP * page)):
                    used[self.table[b, t // page], t % page] = True
            for e in (self.ke, self.ve):
                e.transpose(0, 2, 1)[~used] = -1
            for s in (self.ks, self.vs):
                s[~used.any(1)] = np.nan
        self.q = torch.from_numpy(g.standard_normal((B, S, Hq, D)) * q_scale).to(torch.bfloat16)

    def args(self):
        t = lambda a: torch.from_numpy(a).to(DEV)
        return (self.q.to(DEV), t(self.kc), t(self.vc), t(self.ke), t(self.ve), t(self.ks), t(self.vs), t(self.table),
                t(self.lens))

    def args8(self):
        q, kc, vc, ke, ve, ks, vs, table, lens = self.args()
        k8, v8 = lidx.lidx_cache4_to_8(kc, vc, ke, ve)
        return q, k8, v8, ks * 32, vs * 32, table, lens

    def value_sizes(self, idx):
        """Sum over a sequence's keys of |v| [B,1,Hq,D], as often as a row lists a key."""
        P, Hkv = self.vs.shape
        out = np.zeros((len(self.lens), 1, Hkv, self.D))
        for b, n in enumerate(np.clip(self.lens, 0, self.table.shape[1] * self.page)):
            t = np.arange(n)
            pid = self.table[b, t // self.page]
            t, pid = t[(pid >= 0) & (pid < P)], pid[(pid >= 0) & (pid < P)]
            v = plain4.numbers(self.vc[pid, :, t % self.page], self.ve[pid, :, t % self.page]) * self.vs[pid][..., None]
            out[b, 0] = np.abs(v).sum(0)
        times = 1 if idx is None else max(np.unique(r, return_counts=True)[1].max() for r in np.asarray(idx).reshape(-1, np.shape(idx)[-1]))
        return np.repeat(out, self.q.shape[2] // Hkv, 2) * times

    def check(self, q_pos=None, ratio=1, idx=None, scale=None, whole=True):
        t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
        kw = dict(q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx), softmax_scale=scale)
        o, lse = lidx.lidx_cache4_attn(*self.args(), want_lse=True, **kw)
        o2, none = lidx.lidx_cache4_attn(*self.args(), **kw)
        _status_ok()
        assert none is None and torch.equal(o, o2)  # and twice the same bits
        ro, rl, so, sl = plain.attention(self.q, plain4.as_8(self.kc, self.ke), plain4.as_8(self.vc, self.ve), self.ks * 32,
                                         self.vs * 32, self.table, self.lens, q_pos, ratio, idx, scale)
        od, lse_d = o.double().cpu().numpy(), lse.double().cpu().numpy()
        seen = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse_d), ~seen)
        assert (od[~seen] == 0).all()
        so = so + 2.0 ** -18 * self.value_sizes(idx)
        err = np.abs(od - ro)
        assert (err <= so).all(), f"out: {np.max(err - so):.3e} over, at {np.argwhere(~(err <= so))[:3]}"
        el = np.abs(lse_d[seen] - rl[seen])
        assert (el <= sl[seen]).all(), f"lse: {np.max(el - sl[seen]):.3e} over"
        if whole and seen.any():
            assert np.linalg.norm(od - ro) <= 5e-3 * np.linalg.norm(ro)
        o8, l8 = lidx.lidx_cache_attn(*self.args8(), want_lse=True, **kw)
        assert (np.abs(od - o8.double().cpu().numpy()) <= 2 * so).all()
        assert (np.abs(lse_d[seen] - l8.double().cpu().numpy()[seen]) <= 2 * sl[seen]).all()
        return od, lse_d


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,page", [
    (1, 1, 128, 64), (8, 1, 64, 16), (8, 8, 128, 128), (10, 2, 80, 16), (21, 3, 16, 32), (34, 2, 112, 64), (9, 1, 96, 64),
    (16, 1, 32, 32), (64, 1, 128, 128), (96, 1, 96, 32), (128, 1, 128, 64), (130, 2, 48, 128), (32, 1, 80, 16),
])
def test_single_tokens(Hq, Hkv, D, page):
    Case(Hq + D, 4, 1, Hq, Hkv, D, page, [1, 0, 257, 130]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_lengths_around_tiles(n):
    Case(n, 1, 1, 8, 2, 64, 16, [n]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("S,Hq,Hkv,D,page,lens,ratio", [
    (2, 8, 2, 64, 16, [40, 1], 1),          # the second sequence holds fewer keys than it has queries
    (5, 20, 4, 80, 32, [77, 300, 0], 1),
    (33, 4, 4, 128, 64, [200], 1),
    (40, 12, 4, 32, 16, [300, 41], 1),      # 3 heads a group: tokens of a tile do not fill it
    (70, 8, 1, 64, 128, [150], 1),
    (37, 16, 1, 128, 64, [9], 4),           # compressed keys: the first rows see nothing
    (9, 128, 1, 64, 64, [200], 1),
    (130, 1, 1, 16, 16, [130], 1),
    (2, 4, 1, 128, 64, [260], 1),           # eight rows of two tokens
])
def test_causal_chunks(S, Hq, Hkv, D, page, lens, ratio):
    c = Case(S + Hq, len(lens), S, Hq, Hkv, D, page, lens)
    c.check(q_pos=[n * ratio - S for n in lens], ratio=ratio)


@pytest.mark.gpu
def test_queries_before_and_behind_the_cache():
    c = Case(5, 3, 4, 8, 2, 64, 16, [50, 50, 50])
    o, lse = c.check(q_pos=[-10, 48, 2 ** 31 - 5], ratio=1)
    assert np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("S,Hq,Hkv,D,page,lens,topk,ratio", [
    (1, 64, 1, 128, 64, [500, 3, 0], 130, 1),
    (1, 8, 2, 80, 16, [300], 1, 1),
    (3, 20, 4, 64, 32, [200, 40], 37, 1),
    (50, 16, 1, 128, 64, [100], 64, 4),
    (4, 128, 1, 128, 128, [400], 256, 1),
    (6, 100, 1, 48, 16, [90, 60], 129, 1),
    (3, 30, 1, 16, 16, [500], 300, 1),
])
def test_selected_keys(S, Hq, Hkv, D, page, lens, topk, ratio):
    B = len(lens)
    c = Case(S * 7 + topk, B, S, Hq, Hkv, D, page, lens)
    idx = c.g.integers(-3, max(lens) + 40, (B, S, topk))          # many out of range, some twice
    idx[0, 0, topk // 2:] = -1
    idx[0, -1] = 2 ** 31 - 1 if S > 1 else idx[0, -1]
    c.check(idx=idx)
    pos = [n * ratio - S for n in lens]
    c.check(idx=idx, q_pos=pos, ratio=ratio)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("Hq", [4, 16, 64])
def test_softmax_scales(scale, Hq):
    Case(7, 1, 3, Hq, 2, 64, 16, [100]).check(scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [8, 16, 40, 100])
def test_groups_that_read_as_nan(Hq):
    """A key with such a group makes its rows NaN, a value makes the group's dims NaN in the rows that see it, with the other
    dims and the log-sum-exp as they are; what no row sees does not reach the output."""
    c = Case(Hq, 3, 1, Hq, 1, 64, 32, [200, 150, 90])
    want, wl = lidx.lidx_cache4_attn(*c.args(), want_lse=True)
    pid = c.table[0, 1]
    c.ke[pid, 0, 5] = (c.ke[pid, 0, 5] & ~0xF0) | 0xC0          # key 37 of sequence 0, dims 16 .. 31
    pid = c.table[1, 0]
    c.ve[pid, 0, 31] = (c.ve[pid, 0, 31] & ~0xF00) | 0xF00      # value 31 of sequence 1, dims 32 .. 47
    o, lse = lidx.lidx_cache4_attn(*c.args(), want_lse=True)
    _status_ok()
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert o[1, ..., 32:48].isnan().all() and torch.equal(o[1, ..., :32], want[1, ..., :32])
    assert torch.equal(o[1, ..., 48:], want[1, ..., 48:]) and torch.equal(lse[1], wl[1])
    assert torch.equal(o[2], want[2]) and torch.equal(lse[2], wl[2])


@pytest.mark.gpu
def test_queries_that_are_not_finite_and_tiny_ones():
    c = Case(9, 1, 4, 8, 1, 128, 64, [200])
    c.q[0, 0] = 0.0
    c.q[0, 1] *= 2.0 ** -100
    c.q[0, 2] *= 2.0 ** 40
    c.ks *= np.float32(2.0) ** -36
    c.check(whole=False)
    c.q[0, 3, 2, 5] = float("inf")
    o, lse = lidx.lidx_cache4_attn(*c.args(), want_lse=True)
    bad = torch.zeros(4, 8, dtype=torch.bool, device=DEV)
    bad[3, 2] = True
    assert torch.equal(o[0].isnan().all(-1), bad) and torch.equal(lse[0].isnan(), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [8, 16, 48])
@pytest.mark.parametrize("k_exp,v_exp", [(-85, -85), (60, 95), (-40, 95)])
def test_scales_at_their_limits(Hq, k_exp, v_exp):
    """The scores stay what they are: queries are scaled against the keys' scale.  (bf16 outputs reach 2^127: values are below 6
    2^11 2^95 = 2^109.)"""
    c = Case(Hq, 2, 1, Hq, 1, 64, 32, [200, 77], poison=False)
    c.ks *= np.float32(2.0) ** k_exp
    c.q *= 2.0 ** -k_exp if abs(k_exp) < 100 else 1
    c.vs *= np.float32(2.0) ** (v_exp + (13 if v_exp < 0 else 10))
    c.check()


@pytest.mark.gpu
def test_page_ids_out_of_range_are_not_seen():
    c = Case(10, 2, 2, 8, 2, 64, 16, [100, 90])
    c.table[0, 2], c.table[0, 4], c.table[1, 0] = -1, 10 ** 6, 2 ** 31 - 1
    c.table[1, 1:] = -5
    o, lse = c.check()
    assert np.isneginf(lse[1]).all()
    c.check(idx=c.g.integers(0, 100, (2, 2, 50)))


@pytest.mark.gpu
def test_lengths_beyond_the_table_and_negative():
    c = Case(11, 3, 1, 4, 1, 32, 16, [64, 64, 64])
    c.lens[:] = [10 ** 9, -4, 64]
    o, lse = c.check()
    assert np.isneginf(lse[1]).all()


@pytest.mark.gpu
def test_strided_queries_streams_and_preallocated_outputs():
    c = Case(12, 3, 5, 8, 2, 64, 16, [100, 7, 55])
    pos = torch.tensor([95, 2, 50], dtype=torch.int32, device=DEV)
    args = c.args()
    want, wl = lidx.lidx_cache4_attn(*args, q_pos=pos, want_lse=True)
    big = torch.full((5, 3, 11, 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    q = big.transpose(0, 1)[:, :, 2:10, :64]
    q.copy_(args[0])
    st = torch.cuda.Stream()
    out = (torch.full_like(want, 7.0), torch.full_like(wl, 7.0))
    ws = torch.empty(lidx.lidx_cache4_attn_workspace_bytes(3, 5, 8, 2, 64, 16, 7) + 256, dtype=torch.uint8, device=DEV)
    st.wait_stream(torch.cuda.current_stream())
    got, gl = lidx.lidx_cache4_attn(q, *args[1:], q_pos=pos, stream=st, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    assert got is out[0] and torch.equal(got, want) and torch.equal(gl, wl)
    _status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("selected", [False, True])
def test_many_rows_with_pages_out_of_range_nan_and_an_own_workspace(selected):
    """Calls of many rows a key widen pages into the workspace: pages that are not seen, NaN groups, an empty sequence and
    slots behind the last stay what they are, and a workspace that another call has left is as good as a new one."""
    B, S, Hq, Hkv, D, page = 3, 90, 8, 2, 80, 16
    c = Case(21, B, S, Hq, Hkv, D, page, [200, 0, 70])
    c.table[0, 3], c.table[2, 1] = -7, 10 ** 6
    idx = c.g.integers(-3, 230, (B, S, 40)) if selected else None
    pos = [200 - S, 5, 0]
    c.check(q_pos=pos, idx=idx)
    need = lidx.lidx_cache4_attn_workspace_bytes(B, S, Hq, Hkv, D, page, c.table.shape[1], 40 if selected else 0)
    assert need > 2 * B * c.table.shape[1] * page * Hkv * D  # the copy is in it
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
    kw = dict(q_pos=t(pos), topk_indices=t(idx))
    want, _ = lidx.lidx_cache4_attn(*c.args(), **kw)
    for _ in range(2):
        got, _ = lidx.lidx_cache4_attn(*c.args(), workspace=ws, **kw)
        assert torch.equal(got, want)
    with pytest.raises(lidx.LidxError) as e:
        lidx.lidx_cache4_attn(*c.args(), workspace=ws[:lidx.lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, 40)], **kw)
    assert e.value.status == 5
    _status_ok()


@pytest.mark.gpu
def test_many_short_and_one_long_sequence():
    lens = [1, 2, 3000, 5, 0, 129] + [7] * 40
    Case(13, len(lens), 1, 8, 2, 64, 16, lens).check()


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,D,page,L,topk,ratio", [
    (8, 1, 64, 8, 128, 64, 20000, 0, 1),       # several units a CTA, tens of tiles each
    (8, 1, 128, 8, 128, 32, 9000, 0, 1),
    (3, 1, 24, 1, 80, 16, 30000, 0, 1),
    (5, 1, 48, 1, 128, 128, 20000, 0, 1),
    (2, 1, 128, 1, 112, 32, 20000, 0, 1),
    (2, 700, 32, 4, 128, 64, 3000, 0, 1),      # chunks over many tiles of rows
    (1, 900, 20, 4, 64, 16, 2000, 0, 2),
    (1, 1500, 64, 1, 128, 64, 1024, 512, 4),   # selected prompts
    (1, 300, 128, 1, 128, 32, 900, 300, 1),
    (2, 500, 16, 2, 48, 16, 700, 200, 1),
    (24, 1, 40, 1, 128, 64, 9000, 1500, 1),
])
def test_large(B, S, Hq, Hkv, D, page, L, topk, ratio):
    g = torch.Generator(device=DEV).manual_seed(B + S)
    MP = -(-L // page)
    NP = B * MP
    i32 = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device=DEV).to(torch.int32)
    side = lambda: (i32(0, 256, NP, Hkv, page, D // 2).to(torch.uint8),
                    sum(i32(6, 12, NP, Hkv, page) << (4 * i) for i in range(D // 16)),
                    torch.exp2(i32(-14, -11, NP, Hkv).float()))
    (kc, ke, ks), (vc, ve, vs) = side(), side()
    table = torch.randperm(NP, generator=g, device=DEV).to(torch.int32).view(B, MP)
    lens = torch.tensor([L] + [1 + (i * 7919) % L for i in range(1, B)], dtype=torch.int32, device=DEV)
    q = torch.randn(B, S, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    kw = dict(q_pos=lens * ratio - S if S > 1 else None, compress_ratio=ratio,
              topk_indices=i32(-20, L, B, S, topk) if topk else None)
    got, _ = lidx.lidx_cache4_attn(q, kc, vc, ke, ve, ks, vs, table, lens, **kw)
    for _ in range(5):  # roles that hand work to each other: a race would show as other bits
        again, _ = lidx.lidx_cache4_attn(q, kc, vc, ke, ve, ks, vs, table, lens, **kw)
        assert torch.equal(got, again)
    _status_ok()
    k8, v8 = lidx.lidx_cache4_to_8(kc, vc, ke, ve)
    as8, _ = lidx.lidx_cache_attn(q, k8, v8, ks * 32, vs * 32, table, lens, **kw)
    assert ((got.double() - as8.double()).norm() <= 1e-2 * as8.double().norm()).item()
    want = plain.attention_cuda(q, k8, v8, ks * 32, vs * 32, table, lens, q_pos=kw["q_pos"], ratio=ratio,
                                idx=kw["topk_indices"])
    assert ((got.double() - want).norm() <= 5e-3 * want.norm()).item()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of codes whose sequence lies at its end."""
    Hkv, page, D, n = 8, 128, 128, 300
    NP = (1 << 33) // (Hkv * page * D) + 40
    c = Case(14, 1, 1, 16, Hkv, D, page, [n])
    small = c.args()
    m = small[1].shape[0]
    big = [torch.zeros((NP,) + t.shape[1:], dtype=t.dtype, device=DEV) for t in small[1:7]]
    for b, s in zip(big, small[1:7]):
        b[-m:] = s
    table = small[7] + (NP - m)
    want, _ = lidx.lidx_cache4_attn(*small)
    got, _ = lidx.lidx_cache4_attn(small[0], *big, table, small[8])
    idx = torch.arange(n, dtype=torch.int32, device=DEV).view(1, 1, n)
    sel, _ = lidx.lidx_cache4_attn(small[0], *big, table, small[8], topk_indices=idx)
    ref, _ = lidx.lidx_cache4_attn(*small, topk_indices=idx)
    assert torch.equal(got, want) and torch.equal(sel, ref)
    # and the writer reaches the same page
    k = torch.randn(1, 3, Hkv, D, device=DEV).to(torch.bfloat16)
    start = torch.tensor([n - 3], dtype=torch.int32, device=DEV)
    lidx.lidx_cache4_append(k, k, *small[1:7], small[7], start)
    lidx.lidx_cache4_append(k, k, *big, table, start)
    for b, s in zip(big, small[1:7]):
        as_bits = (lambda t: t.view(torch.int32)) if s.dtype == torch.float32 else (lambda t: t)  # unused scales are NaN
        assert torch.equal(as_bits(b[-m:].contiguous()), as_bits(s))
    _status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,selected", [(8, False), (16, False), (64, False), (80, False), (80, True), (256, False), (24, True),
                                         (160, True)])
def test_stall_times_out_and_the_next_call_is_correct(Hq, selected):
    """The producers load nothing, every wait runs out, the launch ends by itself and says so."""
    c = Case(17, 3, 1, Hq, 2, 64, 32, [500, 0, 90])
    idx = c.g.integers(0, 500, (3, 1, 200)) if selected else None
    given = None if idx is None else torch.from_numpy(idx.astype(np.int32)).to(DEV)
    assert lidx.lidx_device_status() == 0
    old = lidx.lidx_set_wait_limit_ns(2_000_000)
    lidx.lidx_debug_stall_producer(True)
    try:
        lidx.lidx_cache4_attn(*c.args(), topk_indices=given)
        assert lidx.lidx_device_status() == 7
    finally:
        lidx.lidx_debug_stall_producer(False)
        lidx.lidx_set_wait_limit_ns(old)
    c.check(idx=idx)


@pytest.mark.gpu
def test_captured_and_replayed_with_new_lengths():
    """Append with the norm and rotation on the way, then attention, in one graph: replayed with new tokens, places and
    lengths, as a server's step is."""
    B, Hq, Hkv, D, page, MP = 3, 16, 2, 64, 16, 8
    g = torch.Generator(device=DEV).manual_seed(6)
    rnd = lambda *n: torch.randn(*n, generator=g, device=DEV).to(torch.bfloat16)
    z = lambda *n, dt=torch.uint8: torch.zeros(*n, dtype=dt, device=DEV)
    cache = [z(B * MP, Hkv, page, D // 2), z(B * MP, Hkv, page, D // 2), z(B * MP, Hkv, page, dt=torch.int32),
             z(B * MP, Hkv, page, dt=torch.int32), z(B * MP, Hkv, dt=torch.float32), z(B * MP, Hkv, dt=torch.float32)]
    table = torch.arange(B * MP, dtype=torch.int32, device=DEV).view(B, MP)
    freqs, w = lidx.lidx_rope_freqs(D), torch.rand(D, generator=g, device=DEV) + 0.5
    q, k, v = rnd(B, 1, Hq, D), rnd(B, 1, Hkv, D), rnd(B, 1, Hkv, D)
    start = z(B, dt=torch.int32)

    def step():
        lidx.lidx_cache4_append(k, v, *cache, table, start, freqs=freqs, weight=w, layout="half")
        turned = lidx.lidx_norm_rope(q, w, start[:, None], freqs, layout="half")
        return lidx.lidx_cache4_attn(turned, *cache, table, start + 1)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in cache:
        t.zero_()
    start.zero_()
    outs, steps = [], []
    for i in range(40):
        for t in (q, k, v):
            t.copy_(rnd(*t.shape))
        steps.append((q.clone(), k.clone(), v.clone(), start.clone()))
        graph.replay()
        outs.append(out.clone())
        start += torch.tensor([1, 1 + i % 2, 1 if i % 3 else 2], dtype=torch.int32, device=DEV)
    held = [t.clone() for t in cache]
    for t in cache:
        t.zero_()
    for (qi, ki, vi, si), want in zip(steps, outs):
        q.copy_(qi), k.copy_(ki), v.copy_(vi), start.copy_(si)
        assert torch.equal(step(), want)
    assert all(torch.equal(a, b) for a, b in zip(cache, held))
    _status_ok()


@pytest.mark.gpu
def test_binding_refusals():
    c = Case(15, 2, 1, 4, 2, 32, 16, [20, 30])
    ok = c.args()
    lidx.lidx_cache4_attn(*ok)

    def but(i, t):
        return ok[:i] + (t,) + ok[i + 1:]

    for bad in (but(0, ok[0].float()), but(1, ok[1].view(torch.int8)), but(3, ok[3].float()), but(8, ok[8].long())):
        with pytest.raises(TypeError):
            lidx.lidx_cache4_attn(*bad)
    for bad in (but(0, ok[0][..., :16]), but(8, ok[8][:1]), but(7, ok[7][:1]), but(3, ok[3][:1]), but(5, ok[5][:1]),
                but(2, ok[2][..., :8].contiguous()), but(4, ok[4].cpu())):
        with pytest.raises(ValueError):
            lidx.lidx_cache4_attn(*bad)
    with pytest.raises(ValueError):
        lidx.lidx_cache4_attn(*ok, topk_indices=torch.zeros(1, 1, 4, dtype=torch.int32, device=DEV))
    for kw in (dict(out=(ok[0][:1], None)),):
        with pytest.raises(ValueError):
            lidx.lidx_cache4_attn(*ok, **kw)
    with pytest.raises(lidx.LidxError):
        lidx.lidx_cache4_attn(ok[0][:, :, :3].contiguous(), *ok[1:])  # 3 heads over 2
    shifted = torch.zeros(ok[3].numel() + 1, dtype=torch.int32, device=DEV)[1:].view(ok[3].shape)  # 4 bytes off
    with pytest.raises(lidx.LidxError) as e:
        lidx.lidx_cache4_attn(*but(3, shifted))
    assert e.value.status == 3
    with pytest.raises(lidx.LidxError) as e:
        lidx.lidx_cache4_attn(*ok, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
