"""Attention over the paged 8-bit cache (lidx_cache_attn) against its 64-bit definition.

Element tolerances come from plain.attention's derivation.  On random inputs the error of a whole output
is held too: independent roundings of the weights (2^-8 uniform: rms below 2^-8 / sqrt(3)) and of the
output to bf16 (rms below 2^-9) stay below 5e-3 of its norm."""

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


def _status_ok():
    torch.cuda.synchronize()
    assert lidx.lidx_device_status() == 0


def test_refusals_without_gpu():
    L = lidx.lib()
    P = lambda v: None if v is None else C.c_void_p(v)
    st, odd = (C.c_int64 * 3)(64, 64, 64), (C.c_int64 * 3)(64, 4, 64)

    def call(q=16, qs=st, kc=16, vc=16, ksc=16, vsc=16, table=16, lens=16, pos=None, idx=None, B=1, S=1, Hq=1, Hkv=1,
             D=64, page=16, MP=1, NP=1, ratio=1, topk=0, scale=1.0, out=16, lse=None, ws=None, wsb=0):
        return L.lidx_cache_attn(P(q), qs, P(kc), P(vc), P(ksc), P(vsc), P(table), P(lens), P(pos), P(idx), B, S, Hq,
                                 Hkv, D, page, MP, NP, ratio, topk, scale, P(out), P(lse), P(ws), wsb, None)

    for name in ("q", "qs", "kc", "vc", "ksc", "vsc", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
    for bad in (dict(B=0), dict(S=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3, Hkv=2), dict(Hq=129), dict(D=8), dict(D=136),
                dict(D=256), dict(page=24), dict(MP=0), dict(NP=0), dict(NP=1 << 29), dict(ratio=0),
                dict(idx=16, topk=0), dict(idx=16, topk=(1 << 20) + 1), dict(scale=math.nan), dict(scale=math.inf),
                dict(B=1 << 16, S=1 << 16)):
        assert call(**bad) == 2, bad
    for bad in (dict(q=24), dict(qs=odd), dict(kc=8), dict(vc=8), dict(out=8), dict(lens=18), dict(table=18),
                dict(pos=18), dict(idx=18, topk=1), dict(lse=18), dict(ksc=18), dict(vsc=18)):
        assert call(**bad) == 3, bad


# ------------------------------------------------------------------ GPU

class Case:
    """A cache, its tables and queries on both sides."""

    def __init__(self, seed, B, S, Hq, Hkv, D, page, lens, q_scale=1.0, exps=(-8, -5), poison=True):
        g = np.random.default_rng(seed)
        self.g, self.page = g, page
        MP = max(1, max(-(-max(n, 1) // page) for n in lens))
        NP = B * MP + 2
        self.kc, self.ks = plain.random_cache(g, NP, Hkv, page, D, *exps)
        self.vc, self.vs = plain.random_cache(g, NP, Hkv, page, D, *exps)
        self.table = g.permutation(NP)[:B * MP].reshape(B, MP).astype(np.int32)
        self.lens = np.asarray(lens, np.int32)
        if poison:
            # every slot past a sequence's length holds NaN codes, and so do pages of nobody
            used = np.zeros((NP, page), bool)
            for b, n in enumerate(lens):
                for t in range(min(n, MP * page)):
                    used[self.table[b, t // page], t % page] = True
            for c in (self.kc, self.vc):
                c.transpose(0, 2, 1, 3)[~used] = 0x7F
            for s in (self.ks, self.vs):
                s[~used.any(1)] = np.nan
        self.q = torch.from_numpy(g.standard_normal((B, S, Hq, D)) * q_scale).to(torch.bfloat16)

    def args(self, q=None):
        t = lambda a: torch.from_numpy(a).to(DEV)
        return ((self.q.to(DEV) if q is None else q), plain.to_cuda(self.kc), plain.to_cuda(self.vc), t(self.ks),
                t(self.vs), t(self.table), t(self.lens))

    def check(self, q_pos=None, ratio=1, idx=None, scale=None, whole=True):
        t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(DEV)
        o, lse = lidx.lidx_cache_attn(*self.args(), q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx),
                                      softmax_scale=scale, want_lse=True)
        o2, none = lidx.lidx_cache_attn(*self.args(), q_pos=t(q_pos), compress_ratio=ratio, topk_indices=t(idx),
                                        softmax_scale=scale)
        _status_ok()
        assert none is None and torch.equal(o, o2)  # and twice the same bits
        ro, rl, so, sl = plain.attention(self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, q_pos, ratio,
                                         idx, scale)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        seen = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse), ~seen)
        assert (o[~seen] == 0).all()
        err = np.abs(o - ro)
        assert (err <= so).all(), f"out: {np.max(err - so):.3e} over, at {np.argwhere(~(err <= so))[:3]}"
        el = np.abs(lse[seen] - rl[seen])
        assert (el <= sl[seen]).all(), f"lse: {np.max(el - sl[seen]):.3e} over"
        if whole and seen.any():
            assert np.linalg.norm(o - ro) <= 5e-3 * np.linalg.norm(ro)
        return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,page", [
    (1, 1, 128, 64), (8, 1, 64, 16), (8, 8, 128, 128), (10, 2, 80, 16), (21, 3, 16, 32), (34, 2, 112, 64),
    (64, 1, 128, 128), (96, 1, 96, 32), (128, 1, 128, 64), (130, 2, 48, 128),
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
])
def test_causal_chunks(S, Hq, Hkv, D, page, lens, ratio):
    c = Case(S + Hq, len(lens), S, Hq, Hkv, D, page, lens)
    c.check(q_pos=[n * ratio - S for n in lens], ratio=ratio)


@pytest.mark.gpu
def test_queries_before_and_behind_the_cache():
    """q_pos is free: rows far before the first key see none, rows far behind see all."""
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
def test_indices_of_the_indexer_drive_the_attention():
    """The indexer's own output, padding and all, selects the keys."""
    import workloads

    S, H, D, n, ratio, topk, page = 48, 8, 64, 24, 4, 10, 16
    wl = workloads.WORKLOADS["tiny"].with_(S=S, H=H, D=32, Skv=n, ratio=ratio, topk=topk)
    qi, ki, w = (t.to(DEV) for t in workloads.v4_inputs(wl, 3))
    idx, _, _ = lidx.lidx_indexer_fwd(qi, ki, w, ratio, topk)
    c = Case(2, 1, S, 16, 2, D, page, [n])
    c.check(idx=idx.cpu().numpy(), q_pos=[0], ratio=ratio)


@pytest.mark.gpu
def test_all_keys_selected_equals_all_keys():
    c = Case(8, 2, 1, 32, 2, 128, 64, [333, 200])
    idx = np.stack([c.g.permutation(400) for _ in range(2)])[:, None]
    a, la = c.check(idx=idx)
    b, lb = c.check()
    assert np.abs(la - lb).max() < 1e-3 and np.linalg.norm(a - b) <= 8e-3 * np.linalg.norm(b)


@pytest.mark.gpu
@pytest.mark.parametrize("selected", [False, True])
def test_peaks_sinks_and_wide_scales(selected):
    """A first key that takes nearly all the weight with a long flat tail that together still counts; score
    ranges far beyond e^88; page scales over 2^20."""
    n, D = 3000, 64
    c = Case(4, 2, 1, 8, 1, D, 64, [n, n], poison=False)
    idx = np.stack([np.arange(n)] * 2)[:, None] if selected else None
    # queries along one dim; key 0 alone is large there: its weight is e^10 times each other's
    c.q[:] = 0.0
    c.q[0, 0, :, 3] = 8.0
    c.kc[:, :, :, 3] = 0
    p0 = c.table[0, 0]
    c.ks[p0, 0] = 0.03125
    c.kc[p0, 0, 0, 3] = plain.e4m3_round(320.0)        # 8 * 10 / sqrt(64) = 10
    c.q[1, 0, :, 5] = 300.0                             # scores to thousands: the weights are 0 and 1
    o, lse = c.check(idx=idx, whole=False)
    assert abs(lse[0, 0, 0] - math.log(math.exp(10) + n - 1)) < 1e-2
    c = Case(6, 2, 1, 16, 2, D, 32, [n, 777], exps=(-20, 0), q_scale=0.02)
    c.check(idx=None if not selected else np.stack([c.g.permutation(n) for _ in range(2)])[:, None], whole=False)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_softmax_scales(scale):
    Case(7, 1, 3, 8, 2, 64, 16, [100]).check(scale=scale)


@pytest.mark.gpu
def test_zero_and_tiny_queries():
    """A query of zeros weighs all keys alike; tiny and huge queries keep their scores."""
    c = Case(9, 1, 4, 8, 1, 128, 64, [200])
    c.q[0, 0] = 0.0
    c.q[0, 1] *= 2.0 ** -100
    c.q[0, 2] *= 2.0 ** 40
    c.ks *= np.float32(2.0) ** -36
    c.check(whole=False)


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
    want, wl = lidx.lidx_cache_attn(*args, q_pos=pos, want_lse=True)
    big = torch.full((5, 3, 11, 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    q = big.transpose(0, 1)[:, :, 2:10, :64]
    q.copy_(args[0])
    st = torch.cuda.Stream()
    out = (torch.full_like(want, 7.0), torch.full_like(wl, 7.0))
    ws = torch.empty(lidx.lidx_cache_attn_workspace_bytes(3, 5, 8, 2, 64) + 256, dtype=torch.uint8, device=DEV)
    st.wait_stream(torch.cuda.current_stream())
    got, gl = lidx.lidx_cache_attn(q, *args[1:], q_pos=pos, stream=st, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    assert got is out[0] and torch.equal(got, want) and torch.equal(gl, wl)
    _status_ok()


@pytest.mark.gpu
def test_many_short_and_one_long_sequence():
    lens = [1, 2, 3000, 5, 0, 129] + [7] * 40
    Case(13, len(lens), 1, 8, 2, 64, 16, lens).check()


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,page,L,topk,ratio", [
    (8, 1, 64, 8, 64, 20000, 0, 1),       # several units a CTA, tens of tiles each
    (3, 1, 24, 1, 16, 30000, 0, 1),
    (5, 1, 48, 1, 128, 20000, 0, 1),
    (2, 1, 128, 1, 32, 20000, 0, 1),
    (2, 700, 32, 4, 64, 3000, 0, 1),      # chunks over many tiles of rows
    (1, 900, 20, 4, 16, 2000, 0, 2),
    (1, 1500, 64, 1, 64, 1024, 512, 4),   # selected prompts
    (1, 300, 128, 1, 32, 900, 300, 1),
    (2, 500, 16, 2, 16, 700, 200, 1),
    (24, 1, 40, 1, 64, 9000, 1500, 1),
])
def test_large(B, S, Hq, Hkv, page, L, topk, ratio):
    g = torch.Generator(device=DEV).manual_seed(B + S)
    D, MP = 128, -(-L // page)
    NP = B * MP
    rnd = lambda *n: torch.randn(*n, generator=g, device=DEV)
    kc, vc = ((rnd(NP, Hkv, page, D) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in (0, 1))
    ks, vs = (torch.exp2(torch.randint(-9, -5, (NP, Hkv), generator=g, device=DEV).float()) for _ in (0, 1))
    table = torch.randperm(NP, generator=g, device=DEV).to(torch.int32).view(B, MP)
    lens = torch.tensor([L] + [1 + (i * 7919) % L for i in range(1, B)], dtype=torch.int32, device=DEV)
    q = rnd(B, S, Hq, D).to(torch.bfloat16)
    q_pos = lens * ratio - S if S > 1 else None
    idx = torch.randint(-20, L, (B, S, topk), generator=g, device=DEV).to(torch.int32) if topk else None
    args = (q, kc, vc, ks, vs, table, lens)
    got, _ = lidx.lidx_cache_attn(*args, q_pos=q_pos, compress_ratio=ratio, topk_indices=idx)
    for _ in range(5):  # roles that hand work to each other: a race would show as other bits
        again, _ = lidx.lidx_cache_attn(*args, q_pos=q_pos, compress_ratio=ratio, topk_indices=idx)
        assert torch.equal(got, again)
    _status_ok()
    want = plain.attention_cuda(*args, q_pos=q_pos, ratio=ratio, idx=idx)
    assert ((got.double() - want).norm() <= 5e-3 * want.norm()).item()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes whose sequence lies at its end."""
    Hkv, page, D, n = 8, 128, 128, 300
    NP = (1 << 32) // (Hkv * page * D) + 40
    c = Case(14, 1, 1, 16, Hkv, D, page, [n])
    kc = torch.zeros(NP, Hkv, page, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros(NP, Hkv, page, D, dtype=torch.uint8, device=DEV)
    ks, vs = torch.ones(NP, Hkv, device=DEV), torch.ones(NP, Hkv, device=DEV)
    small = c.args()
    m = small[1].shape[0]
    kc[-m:], vc[-m:] = small[1].view(torch.uint8), small[2].view(torch.uint8)
    ks[-m:], vs[-m:] = small[3], small[4]
    f8 = torch.float8_e4m3fn
    want, _ = lidx.lidx_cache_attn(*small)
    got, _ = lidx.lidx_cache_attn(small[0], kc.view(f8), vc.view(f8), ks, vs, small[5] + (NP - m), small[6])
    idx = torch.arange(n, dtype=torch.int32, device=DEV).view(1, 1, n)
    sel, _ = lidx.lidx_cache_attn(small[0], kc.view(f8), vc.view(f8), ks, vs, small[5] + (NP - m), small[6],
                                  topk_indices=idx)
    ref, _ = lidx.lidx_cache_attn(*small, topk_indices=idx)
    assert torch.equal(got, want) and torch.equal(sel, ref)
    # and the writer reaches the same page
    k = torch.randn(1, 3, Hkv, D, device=DEV).to(torch.bfloat16)
    start = torch.tensor([n - 3], dtype=torch.int32, device=DEV)
    lidx.lidx_cache_append(k, k, *(t for t in small[1:5]), small[5], start)
    lidx.lidx_cache_append(k, k, kc.view(f8), vc.view(f8), ks, vs, small[5] + (NP - m), start)
    assert torch.equal(kc[-m:], small[1].view(torch.uint8))
    assert torch.equal(vs[-m:].view(torch.int32), small[4].view(torch.int32))  # as bits: unused scales are NaN
    _status_ok()


@pytest.mark.gpu
def test_workspace_refusals():
    c = Case(16, 1, 1, 8, 1, 64, 16, [40])
    need = lidx.lidx_cache_attn_workspace_bytes(1, 1, 8, 1, 64)
    assert need > 0
    for ws in (torch.empty(need + 512, dtype=torch.uint8, device=DEV)[16:], torch.empty(64, dtype=torch.uint8, device=DEV)):
        with pytest.raises(lidx.LidxError) as e:
            lidx.lidx_cache_attn(*c.args(), workspace=ws)
        assert e.value.status == 5
    _status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,selected", [(16, False), (80, False), (80, True), (256, False), (24, True), (160, True)])
def test_stall_times_out_and_the_next_call_is_correct(Hq, selected):
    """The producer loads nothing, every wait runs out, the launch ends by itself and says so."""
    c = Case(17, 3, 1, Hq, 2, 64, 32, [500, 0, 90])
    idx = c.g.integers(0, 500, (3, 1, 200)) if selected else None
    given = None if idx is None else torch.from_numpy(idx.astype(np.int32)).to(DEV)
    assert lidx.lidx_device_status() == 0
    old = lidx.lidx_set_wait_limit_ns(2_000_000)
    lidx.lidx_debug_stall_producer(True)
    try:
        lidx.lidx_cache_attn(*c.args(), topk_indices=given)
        assert lidx.lidx_device_status() == 7
    finally:
        lidx.lidx_debug_stall_producer(False)
        lidx.lidx_set_wait_limit_ns(old)
    c.check(idx=idx)


@pytest.mark.gpu
def test_binding_refusals():
    c = Case(15, 2, 1, 4, 2, 32, 16, [20, 30])
    ok = c.args()

    def but(i, t):
        return ok[:i] + (t,) + ok[i + 1:]

    with pytest.raises(TypeError):
        lidx.lidx_cache_attn(*but(0, ok[0].float()))
    with pytest.raises(TypeError):
        lidx.lidx_cache_attn(*but(1, ok[1].view(torch.uint8)))
    with pytest.raises(ValueError):
        lidx.lidx_cache_attn(*but(0, ok[0][..., :16]))
    with pytest.raises(ValueError):
        lidx.lidx_cache_attn(*but(6, ok[6][:1]))
    with pytest.raises(ValueError):
        lidx.lidx_cache_attn(*but(5, ok[5][:1]))
    with pytest.raises(ValueError):
        lidx.lidx_cache_attn(*ok, topk_indices=torch.zeros(1, 1, 4, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        lidx.lidx_cache_attn(*ok, topk_indices=torch.zeros(2, 1, 4, device=DEV))
    with pytest.raises(ValueError):
        lidx.lidx_cache_attn(*ok, out=(ok[0][:1], None))
    with pytest.raises(lidx.LidxError):
        lidx.lidx_cache_attn(ok[0][:, :, :3].contiguous(), *ok[1:])  # 3 heads over 2


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,scale", [(16, 1e5), (64, 1e5), (128, 1e5), (16, -0.07), (64, -0.07), (128, -0.07), (64, 0.0),
                                      (128, 0.0)])
def test_scores_beyond_fp32_and_other_signs_of_the_scale(Hq, scale):
    """|score| up to 2^24 and more, the largest ahead by 2^12 or more: the row is that key's value.  Negative and zero scales."""
    c = Case(Hq, 2, 1, Hq, 1, 128, 64, [300, 129])
    if scale <= 0:
        c.check(scale=scale)
        return
    # keys are one-hot in a dim each with an own integer code, queries one-hot: the scores are exact products
    kc = np.zeros((2 * 5 + 2, 1, 64, 128), np.uint8)
    g = c.g
    for b, n in enumerate(c.lens):
        for t in range(int(n)):
            # 0x40 .. 0x7e are e4m3 codes of 2 .. 448 in order; key t of dim d: one code lies above the others
            kc[c.table[b, t // 64], 0, t % 64, :] = g.integers(0x38, 0x70, 128)
    best = g.integers(0, 129, 128)
    for b in range(2):
        for d in range(128):
            t = int(best[d])
            kc[c.table[b, t // 64], 0, t % 64, d] = 0x7E  # 448
    c.kc = kc
    c.ks = np.ones_like(c.ks)
    q = torch.zeros(2, 1, Hq, 128)
    for h in range(Hq):
        q[:, 0, h, h] = 1.0
    c.q = q.to(torch.bfloat16)
    o, lse = lidx.lidx_cache_attn(*c.args(), softmax_scale=scale, want_lse=True)
    _status_ok()
    o, lse = o.float().cpu(), lse.double().cpu().numpy()
    e4m3 = torch.from_numpy(c.vc).view(torch.float8_e4m3fn).float()
    for b in range(2):
        for h in range(Hq):
            t = int(best[h])
            pg = int(c.table[b, t // 64])
            want = (e4m3[pg, 0, t % 64] * float(c.vs[pg, 0])).to(torch.bfloat16).float()
            # hi + lo weights: 2^-8 at most, and one bf16 rounding
            assert ((o[b, 0, h] - want).abs() <= 2.0 ** -7 * want.abs()).all()
    assert np.allclose(lse, 448 * scale, rtol=2.0 ** -20)
