"""More operators that stand next to the lightning indexer in a sparse-attention model, as cases.

Four operators that are used together, from a projection's output to the attention's:

  norm    norms of queries and keys for each head, with the rotary positions in the same pass, forward
          and backward (gradients of the inputs and of the norms' weights)
  axes    rotary positions with several axes (time, height, width), forward and backward
  append  writing new keys and values into a paged cache, 8 or 4 bits a number, with the norm and the
          rotation of the keys on the way
  attn4   attention over a paged cache of 4-bit numbers: all keys of a sequence, causal chunks of
          queries, or the keys that the indexer selected for each query row

Layouts: queries, keys and values [batch, token, head, dim].  The 8-bit cache is [page, head, slot, dim] in
float8_e4m3fn with scales [page, head] in float32.  The 4-bit cache has codes uint8 [page, head, slot, dim / 2] (the
even dim in the low half; sign, two exponent bits, one fraction bit: 0 .5 1 1.5 2 3 4 6), exponents int32 [page,
head, slot] (four bits for each 16 dims, the first dims in the lowest bits) and scales [page, head]: a number is code *
2^exponent * scale.

A case is a dict of plain values; ``prepare`` makes what a caller holds before the call, ``run``
makes one call, in plain torch operations or, where ``own`` is set, through the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def _turn(name, op, B, S, H, H2, D, R, off, layout, dtype, back, axes=1, mix=False, factor=1.0, top=8192):
    # axes: of a position; mix: the axes' pairs alternate, else they follow each other in sections;
    # top: positions lie below it; factor: long-context scaling of the frequencies
    return dict(name=name, op=op, B=B, S=S, H=H, H2=H2, D=D, R=R, off=off, layout=layout, dtype=dtype, back=back,
                axes=axes, mix=mix, factor=factor, top=top)


def _append(name, bits, B, S, Hkv, D, R, off, layout, norm, axes, mix, PS, top):
    # top: the longest sequence already holds about this many tokens
    return dict(name=name, op="append", bits=bits, B=B, S=S, Hkv=Hkv, D=D, R=R, off=off, layout=layout, norm=norm,
                axes=axes, mix=mix, PS=PS, top=top, factor=1.0)


def _attn(name, B, S, Hq, Hkv, D, PS, L, ragged=False, causal=False, ratio=1, topk=0, hole=False):
    # L: longest sequence in the cache; topk: selected keys a row (0: all visible keys);
    # hole: the last sequence of a batch is empty
    return dict(name=name, op="attn4", B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, PS=PS, L=L, ragged=ragged, causal=causal,
                ratio=ratio, topk=topk, hole=hole)


def listed():
    return [
        # one decode step of 16 sequences, grouped heads, both sides normed; latency counts
        _turn("norm decode 16", "norm", 16, 1, 64, 8, 128, 128, 0, "half", "bf16", False, factor=32.0, top=131072),
        # the prompt of two sequences, sizes of the backward workload's rows
        _turn("norm prompt 2x8192", "norm", 2, 8192, 64, 8, 128, 128, 0, "half", "bf16", False, factor=32.0, top=16384),
        # a training step's gradients in 32 bits, part of each head rotated, an odd number of tokens
        _turn("norm backward 4095 fp32", "norm", 1, 4095, 32, 8, 128, 64, 64, "interleaved", "fp32", True),
        # a prompt of text and video: time, height and width in sections of the pairs
        _turn("axes prompt 8191", "axes", 1, 8191, 64, 8, 128, 128, 0, "half", "bf16", False, axes=3),
        # gradients of an image tower: height and width, four images of 37 x 37 patches, narrow heads
        _turn("axes backward 4x1369", "axes", 4, 1369, 20, 20, 80, 80, 0, "half", "fp32", True, axes=2, mix=True),
        # one new token for each of 64 sequences, keys normed and turned; latency counts
        _append("append decode 64", 8, 64, 1, 8, 128, 128, 0, "half", True, 1, False, 64, 8191),
        # ragged prompts of four sequences behind some tokens that are there already, the shared key's part rotated
        _append("append prompt 4x4097", 8, 4, 4097, 8, 128, 64, 64, "interleaved", False, 1, False, 128, 777),
        # the same into four bits, keys normed and turned by three axes
        _append("append prompt 4x4097 4-bit", 4, 4, 4097, 8, 128, 128, 0, "half", True, 3, True, 64, 777),
        # one sequence with a short cache: latency counts
        _attn("attn decode 1x1024", 1, 1, 64, 8, 128, 64, 1024),
        # a serving batch of ragged lengths, grouped heads: bandwidth counts
        _attn("attn decode 64x32768 ragged", 64, 1, 64, 8, 128, 64, 32768, ragged=True),
        # a chunk of a long prompt, causal over what the cache holds: tensor rate counts
        _attn("attn chunk 2048 of 16384", 1, 2048, 64, 8, 128, 64, 16384, causal=True),
        # decode over the keys that the indexer selected, one selection a sequence
        _attn("attn selected decode 32", 32, 1, 64, 1, 128, 64, 65536, ragged=True, topk=2048),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def _draw_one(rng):
    kind = rng.choice(["norm", "norm", "axes", "append", "append", "decode", "decode", "chunk", "selected"])
    if kind in ("norm", "axes"):
        D = rng.choice([32, 64, 80, 128, 256])
        R = rng.choice([D, D, D // 2])
        return dict(op=kind, B=rng.choice([1, 1, 2, 5, 16]), S=_log(rng, 1, 8192), H=rng.choice([1, 8, 20, 32, 64]),
                    H2=rng.choice([0, 1, 8]), D=D, R=R, off=rng.choice([0, D - R]),
                    layout=rng.choice(["interleaved", "half"]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    back=rng.random() < 0.4, axes=rng.choice([2, 3]) if kind == "axes" else rng.choice([1, 1, 3]),
                    mix=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 32.0]), top=_log(rng, 2048, 262144))
    if kind == "append":
        D = rng.choice([64, 80, 128])
        R = rng.choice([D, D // 2])
        return dict(op="append", bits=rng.choice([4, 8]), B=_log(rng, 1, 128), S=_log(rng, 1, 8192),
                    Hkv=rng.choice([1, 2, 4, 8]), D=D, R=R, off=rng.choice([0, D - R]),
                    layout=rng.choice(["interleaved", "half"]), norm=rng.random() < 0.5, axes=rng.choice([1, 1, 2, 3]),
                    mix=rng.random() < 0.5, PS=rng.choice([16, 32, 64, 128]), top=_log(rng, 2, 8192), factor=1.0)
    Hkv = rng.choice([1, 1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 8, 12, 16]) if Hkv > 1 else rng.choice([8, 32, 48, 64, 128])
    c = dict(op="attn4", B=_log(rng, 1, 64), S=1, Hq=G * Hkv, Hkv=Hkv, D=rng.choice([64, 80, 112, 128, 128]),
             PS=rng.choice([16, 32, 64, 128]), L=_log(rng, 64, 131072), ragged=rng.random() < 0.7,
             causal=False, ratio=1, topk=0, hole=rng.random() < 0.2)
    if kind == "decode" and rng.random() < 0.3:
        c.update(S=rng.choice([2, 3, 5]), causal=True)
    if kind == "chunk":
        c.update(B=rng.choice([1, 1, 2, 3]), S=_log(rng, 16, 4096), L=_log(rng, 64, 16384), causal=True)
    if kind == "selected":
        c.update(topk=_log(rng, 16, 2048))
        if rng.random() < 0.5:
            c.update(B=rng.choice([1, 1, 2]), S=_log(rng, 2, 4096), L=_log(rng, 64, 8192), causal=True,
                     ratio=rng.choice([1, 4]))
    return c


def draw(rng):
    big = [work(c) for c in listed()]
    bytes_, flops = max(w["bytes"] for w in big), max(w["flops"] for w in big)
    while True:
        c = _draw_one(rng)
        w = work(c)
        if w["bytes"] > bytes_ or w["flops"] > flops:
            continue
        if c["op"] == "attn4":
            # what the plain form holds in 32 bits stays within a few tens of gigabytes
            keys = c["topk"] * c["S"] * c["B"] if c["topk"] else c["B"] * _longest(c)
            if keys * c["Hkv"] * c["D"] * 4 > 9e9 or (not c["topk"] and c["B"] * c["S"] * c["Hq"] * _longest(c) * 4 > 9e9):
                continue
            if c["topk"] and c["B"] * c["S"] * c["L"] * 4 > 9e9:
                continue
        return c


# ------------------------------------------------------------------ sizes of a case

def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], the same for every seed, the first of them hi."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _lens(c):
    lens = _spread(c["B"], 1, c["L"]) if c["ragged"] else [c["L"]] * c["B"]
    if c["hole"] and c["B"] > 1:
        lens[-1] = 0
    return lens


def _longest(c):
    return -(-c["L"] // c["PS"]) * c["PS"]


def _starts(c):
    return _spread(c["B"], 0, c["top"])


def _counts(c):
    return _spread(c["B"], max(1, c["S"] // 2), c["S"])


def _q_pos(c, n):
    """Position of a sequence's first query, so that its last one is the newest token."""
    return n * c["ratio"] - c["S"]


def _end(c, n, s):
    """Row s of a sequence with n keys sees keys [0, end)."""
    return max(0, min(n, (_q_pos(c, n) + s + 1) // c["ratio"])) if c["causal"] else n


def _pairs(c, n, cap):
    """Sum over a sequence's rows of min(end, cap)."""
    s = np.arange(c["S"], dtype=np.int64)
    end = np.clip((_q_pos(c, n) + s + 1) // c["ratio"], 0, n) if c["causal"] else np.full(c["S"], n)
    return int(np.minimum(end, cap).sum())


def work(c):
    if c["op"] in ("norm", "axes"):
        n = c["B"] * c["S"] * (c["H"] + c["H2"])
        size = 2 if c["dtype"] == "bf16" else 4
        norm = c["op"] == "norm"
        passes = 3 if norm and c["back"] else 2  # the backward of a norm reads its input, too
        flops = 3.0 * n * c["R"] + (n * c["D"] * (9.0 if c["back"] else 4.0) if norm else 0.0)
        return {"bytes": float(passes) * n * c["D"] * size + 4.0 * c["axes"] * c["B"] * c["S"], "flops": flops}
    if c["op"] == "append":
        n = sum(_counts(c)) * c["Hkv"] * c["D"]
        held = 1.0 if c["bits"] == 8 else 0.5 + 4.0 / c["D"]
        return {"bytes": 2.0 * n * (2 + held), "flops": n * (4.0 + (4.0 if c["norm"] else 0.0) + 3.0 * c["R"] / c["D"])}
    lens = _lens(c)
    cap = c["topk"] or (1 << 62)
    pairs = sum(_pairs(c, n, cap) for n in lens)
    if c["topk"]:
        keys = sum(min(n, c["S"] * c["topk"]) for n in lens)
    else:
        keys = sum(_end(c, n, c["S"] - 1) for n in lens)
    rows = c["B"] * c["S"]
    nbytes = 2.0 * keys * c["Hkv"] * (c["D"] / 2 + 4.0 + 4.0 / c["PS"]) + 2.0 * 2 * rows * c["Hq"] * c["D"] + 4.0 * rows * c["topk"]
    return {"bytes": nbytes, "flops": 4.0 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _omega(c):
    """Radians per position of each rotated pair: base 10000, stretched for long contexts by the
    ramp between pairs that turn less than once and more than 32 times in 4096 positions."""
    R, f = c["R"], c["factor"]
    w = 10000.0 ** (-2.0 * np.arange(R // 2, dtype=np.float64) / R)
    if f != 1.0:
        g = np.clip((4096.0 * w / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        w = w * ((1.0 - g) / f + g)
    return w


def _mscale(c):
    return 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0


def _freqs(c):
    turns = np.rint(_omega(c) / (2 * math.pi) * 2.0 ** 64).astype(np.uint64).view(np.int64)
    return torch.from_numpy(turns).to(DEV)


def _axis_list(c):
    """Axis of each pair: alternating, or in sections of which the first is the shortest."""
    n, A = c["R"] // 2, c["axes"]
    if c["mix"]:
        return [i % A for i in range(n)]
    first = n // 4 if A == 3 else n // A
    rest = (n - first + A - 2) // max(1, A - 1)
    return [0 if i < first else 1 + (i - first) // rest for i in range(n)] if A > 1 else [0] * n


def _axis_map(c):
    return torch.tensor(_axis_list(c), dtype=torch.uint8, device=DEV) if c["axes"] > 1 else None


def _positions(g, c, first):
    """[axes, B, S] int32 (or [B, S] with one axis): a token's place; with several axes frames of 24 x 37 patches."""
    i = first + torch.arange(c["S"], device=DEV)
    if c["axes"] == 1:
        return i.to(torch.int32)
    t = torch.arange(c["S"], device=DEV).expand(c["B"], -1)
    yx = [first + t // 37 % 24, first + t % 37]
    return torch.stack(yx if c["axes"] == 2 else [first + t // (24 * 37)] + yx).to(torch.int32)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(g, B, MP):
    return torch.randperm(B * MP, generator=g, device=DEV).to(torch.int32).view(B, MP)


def _cache8(g, pages, c):
    """A cache as it is found: every slot holds numbers, used or not."""
    shape = (pages, c["Hkv"], c["PS"], c["D"])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(100.0).clamp_(-448.0, 448.0)
    scale = torch.exp2(torch.randint(-8, -5, shape[:2], generator=g, device=DEV).float())
    return x.to(torch.float8_e4m3fn), None, scale


def _cache4(g, pages, c):
    """The same in four bits: codes of normally distributed numbers whose group's largest is in (3, 6]."""
    z = np.abs(_normal_quantiles(256)) * 2.2
    nearest = np.abs(z[:, None] - np.array(E2M1)).argmin(1)
    code = (nearest | np.where(np.arange(256) < 128, 8, 0)).astype(np.uint8)
    byte = torch.from_numpy((code[None, :] | (code[:, None] << 4)).reshape(-1)).to(DEV)
    shape = (pages, c["Hkv"], c["PS"])
    codes = byte[torch.randint(0, 65536, shape + (c["D"] // 2,), generator=g, device=DEV, dtype=torch.int32)]
    exps = (torch.randint(7, 12, shape + (c["D"] // 16,), generator=g, device=DEV, dtype=torch.int32) << _shifts(c)).sum(-1)
    scale = torch.exp2(torch.randint(-13, -10, shape[:2], generator=g, device=DEV).float())
    return codes, exps.to(torch.int32), scale


def _shifts(c):
    """Place of each group's bits in a slot's exponents."""
    return 4 * torch.arange(c["D"] // 16, device=DEV, dtype=torch.int32)


def _normal_quantiles(n):
    p = torch.from_numpy((np.arange(n) + 0.5) / n)
    return torch.erfinv(2 * p - 1).numpy() * math.sqrt(2.0)


def prepare(c, seed):
    g = _gen(seed)
    B, S = c["B"], c["S"]
    if c["op"] in ("norm", "axes"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

        def rows(H):
            return torch.randn(B, S, H, c["D"], generator=g, device=DEV).to(dt) if H else None

        def weight(H):
            return (1.0 + 0.2 * torch.randn(c["D"], generator=g, device=DEV)).to(dt) if H else None

        first = torch.randint(0, max(1, c["top"] - S), (B, 1), generator=g, device=DEV)
        st = dict(c=c, x=rows(c["H"]), x2=rows(c["H2"]), pos=_positions(g, c, first), freqs=_freqs(c), axes=_axis_map(c))
        if c["op"] == "norm":
            st.update(w=weight(c["H"]), w2=weight(c["H2"]))
            if c["back"]:
                st.update(g=rows(c["H"]), g2=rows(c["H2"]))
        return st
    if c["op"] == "append":
        Hkv, D, PS = c["Hkv"], c["D"], c["PS"]
        MP = (max(_starts(c)) + S) // PS + 3
        cache = _cache8 if c["bits"] == 8 else _cache4
        kc, ke, ks = cache(g, B * MP, c)
        vc, ve, vs = cache(g, B * MP, c)
        # the size of a token's values varies, so that some tokens outgrow their page's scale
        size = torch.exp(torch.randn(B, S, Hkv, 1, generator=g, device=DEV))
        k = (torch.randn(B, S, Hkv, D, generator=g, device=DEV) * size).to(torch.bfloat16)
        v = (torch.randn(B, S, Hkv, D, generator=g, device=DEV) * size).to(torch.bfloat16)
        w = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
        start = _int32(_starts(c))
        # with one axis a key's position is its place in the cache
        pos = _positions(g, c, start.long()[:, None]) if c["axes"] > 1 else None
        return dict(c=c, k=k, v=v, kc=kc, vc=vc, ke=ke, ve=ve, ks=ks, vs=vs, w=w, pos=pos, freqs=_freqs(c),
                    axes=_axis_map(c), table=_table(g, B, MP), start=start, count=_int32(_counts(c)))
    MP = _longest(c) // c["PS"]
    kc, ke, ks = _cache4(g, B * MP, c)
    vc, ve, vs = _cache4(g, B * MP, c)
    q = torch.randn(B, S, c["Hq"], c["D"], generator=g, device=DEV).to(torch.bfloat16)
    lens = _lens(c)
    q_pos = _int32([_q_pos(c, n) for n in lens]) if c["causal"] else None
    idx = None
    if c["topk"]:
        # distinct visible keys in random order, -1 behind them
        key = torch.rand(B, S, c["L"], generator=g, device=DEV)
        end = _ends_plain(c, _int32(lens), q_pos)
        key = torch.where(torch.arange(c["L"], device=DEV) < end[:, :, None], key, -1.0)
        n = min(c["topk"], c["L"])
        val, at = torch.topk(key, n, dim=2)
        idx = torch.full((B, S, c["topk"]), -1, dtype=torch.int32, device=DEV)
        idx[:, :, :n] = torch.where(val >= 0, at, -1).to(torch.int32)
    return dict(c=c, q=q, kc=kc, vc=vc, ke=ke, ve=ve, ks=ks, vs=vs, table=_table(g, B, MP), lens=_int32(lens),
                q_pos=q_pos, idx=idx)


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["c"]
    if own:
        import sparse_attention_top_tcgen05_gb300 as lidx

        turn = dict(layout=c["layout"], rot_off=c["off"], mscale=_mscale(c), axes=st["axes"]) if "layout" in c else {}
        if c["op"] == "axes":
            call = lidx.lidx_rope_bwd if c["back"] else lidx.lidx_rope
            return call(st["x"], st["pos"], st["freqs"], x2=st["x2"], **turn)
        if c["op"] == "norm":
            if c["back"]:
                return lidx.lidx_norm_rope_bwd(st["g"], st["x"], st["w"], st["pos"], st["freqs"], g2=st["g2"], x2=st["x2"],
                                               weight2=st["w2"], eps=EPS, **turn)
            return lidx.lidx_norm_rope(st["x"], st["w"], st["pos"], st["freqs"], x2=st["x2"], weight2=st["w2"], eps=EPS,
                                       **turn)
        if c["op"] == "append":
            kw = dict(count=st["count"], pos=st["pos"], weight=st["w"], eps=EPS, **turn)
            if c["bits"] == 8:
                lidx.lidx_rope_cache_append(st["k"], st["v"], st["freqs"], st["kc"], st["vc"], st["ks"], st["vs"],
                                            st["table"], st["start"], **kw)
                return st["kc"], st["vc"], st["ks"], st["vs"]
            lidx.lidx_cache4_append(st["k"], st["v"], st["kc"], st["vc"], st["ke"], st["ve"], st["ks"], st["vs"],
                                    st["table"], st["start"], freqs=st["freqs"], **kw)
            # the numbers that the codes stand for, in units of 32 scales: an 8-bit cache's
            return lidx.lidx_cache4_to_8(st["kc"], st["vc"], st["ke"], st["ve"]) + (st["ks"], st["vs"])
        return lidx.lidx_cache4_attn(st["q"], st["kc"], st["vc"], st["ke"], st["ve"], st["ks"], st["vs"], st["table"],
                                     st["lens"], q_pos=st["q_pos"], compress_ratio=c["ratio"], topk_indices=st["idx"])[0]
    if c["op"] == "axes":
        cos, sin = _angles_plain(st, c)
        y = _rotate(st["x"].float(), cos, sin, c).to(st["x"].dtype)
        return y if st["x2"] is None else (y, _rotate(st["x2"].float(), cos, sin, c).to(y.dtype))
    if c["op"] == "norm":
        cos, sin = _angles_plain(st, c)
        if c["back"]:
            out = _norm_bwd_plain(st["g"], st["x"], st["w"], cos, sin, c)
            return out if st["x2"] is None else out + _norm_bwd_plain(st["g2"], st["x2"], st["w2"], cos, sin, c)
        y = _rotate(_norm_plain(st["x"].float(), st["w"]), cos, sin, c).to(st["x"].dtype)
        if st["x2"] is None:
            return y
        return y, _rotate(_norm_plain(st["x2"].float(), st["w2"]), cos, sin, c).to(y.dtype)
    if c["op"] == "append":
        k = _norm_plain(st["k"].float(), st["w"]) if c["norm"] else st["k"].float()
        _append_plain(st, _rotate(k, *_angles_plain(st, c), c), st["kc"], st["ke"], st["ks"])
        _append_plain(st, st["v"].float(), st["vc"], st["ve"], st["vs"])
        if c["bits"] == 8:
            return st["kc"], st["vc"], st["ks"], st["vs"]
        return tuple((_unpack4(*h) / 32.0).to(torch.float8_e4m3fn) for h in ((st["kc"], st["ke"]), (st["vc"], st["ve"]))) + (
            st["ks"], st["vs"])
    return _selected_plain(st, c) if c["topk"] else _attn_plain(st, c)


def _angles_plain(st, c):
    """Scaled cosine and sine [B, S, 1, pairs]."""
    pos = st["pos"]
    if pos is None:
        pos = st["start"][:, None] + torch.arange(c["S"], device=DEV)
    pos = pos.long() if c["axes"] == 1 else pos.long()[st["axes"].long()].permute(1, 2, 0)
    # the product wraps at whole turns; its upper half is the angle, from half a turn back to half a turn
    turn = ((pos[..., None] if c["axes"] == 1 else pos) * st["freqs"]) >> 32
    angle = turn.float() * (2.0 * math.pi / 2.0 ** 32)
    m = _mscale(c)
    return (angle.cos() * m)[:, :, None], (angle.sin() * (-m if c.get("back") else m))[:, :, None]


def _rotate(y, cos, sin, c):
    R, o = c["R"], c["off"]
    rot = y[..., o:o + R]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if c["layout"] == "interleaved" else (rot[..., :R // 2], rot[..., R // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    new = torch.stack((p, q), -1).flatten(-2) if c["layout"] == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((y[..., :o], new, y[..., o + R:]), -1)


def _norm_plain(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)


def _norm_bwd_plain(g, x, w, cos, sin, c):
    u = _rotate(g.float(), cos, sin, c)  # the sine's sign is turned: the gradient before the rotation
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    xh, t = xf * r, u * w.float()
    dx = r * (t - xh * (t * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (u * xh).sum((0, 1, 2))


def _unpack4(codes, exps):
    """Codes and exponents -> numbers of their page's scale, float32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    G = both.shape[-1] // 16
    x = (exps[..., None] >> (4 * torch.arange(G, device=DEV, dtype=torch.int32))) & 15
    return (table[both.int()].unflatten(-1, (G, 16)) * torch.exp2(x.float())[..., None]).flatten(-2)


def _held4(codes, exps, scale):
    return _unpack4(codes, exps) * scale[..., None, None]


def _pow2_over(amax, top):
    """Exponent e of the smallest 2^e with amax <= top 2^e, top = 2^k times 7/8 or 3/4."""
    mt, et = math.frexp(top)
    m, ex = torch.frexp(amax)
    return ex - et + (m > mt).int()


def _code4(x):
    """Nearest 4-bit codes, ties to the even one: the borders lie half way between neighbours."""
    a = x.abs().contiguous()
    # a border with an even code below it belongs to that code, the others to the code above
    below = torch.bucketize(a, torch.tensor([0.25, 1.25, 2.5, 5.0], device=DEV), out_int32=True)
    above = torch.bucketize(a, torch.tensor([0.75, 1.75, 3.5], device=DEV), out_int32=True, right=True)
    return (below + above).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)


def _append_plain(st, x, cache, exps, scale):
    """Pages are worked on whole: the first J pages from the one that holds position start."""
    c, start, count, table = st["c"], st["start"].long(), st["count"].long(), st["table"].long()
    B, S, PS, D = c["B"], c["S"], c["PS"], c["D"]
    top = 448.0 if c["bits"] == 8 else 6.0 * 2.0 ** 11
    J = (S + PS - 2) // PS + 1
    first = start // PS
    p = (first[:, None, None] + torch.arange(J, device=DEV)[None, :, None]) * PS + torch.arange(PS, device=DEV)
    i = p - start[:, None, None]                                              # [B,J,PS] token of the call
    new = (i >= 0) & (i < count[:, None, None])
    at = i.clamp(0, S - 1).view(B, J * PS, 1, 1).expand(-1, -1, x.shape[2], x.shape[3])
    val = x.gather(1, at).view(B, J, PS, x.shape[2], x.shape[3]).transpose(2, 3)
    new5 = new[:, :, None, :, None]
    amax = torch.where(new5, val, 0.0).abs().amax((3, 4))                     # [B,J,Hkv]
    e = torch.where(amax > 0, _pow2_over(amax, top), -40).clamp(min=-40)
    want = torch.exp2(e.float())
    ids = table.gather(1, first[:, None] + torch.arange(J, device=DEV))
    old = scale[ids]
    kept = (p[:, :, 0] < start[:, None])[:, :, None]
    touched = new.any(2)[:, :, None]
    now = torch.where(touched, torch.where(kept, torch.maximum(old, want), want), old)
    held = (p < start[:, None, None])[:, :, None, :, None] & touched[..., None, None]
    val = val / now[..., None, None]
    if c["bits"] == 8:
        was = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()      # [B,J,Hkv,PS,D]
        out = torch.where(new5, val, torch.where(held, was * (old / now)[..., None, None], was))
        cache.view(torch.uint8)[ids] = out.to(torch.float8_e4m3fn).view(torch.uint8)
        scale[ids] = now
        return
    codes, ex = cache[ids], exps[ids]
    shift = _shifts(c)
    was = _unpack4(codes, ex) * (old / now)[..., None, None]
    was_x = (ex[..., None] >> shift) & 15                                     # [B,J,Hkv,PS,groups]
    fall = torch.round(torch.log2(now / old)).int()[..., None, None]
    gmax = val.abs().unflatten(-1, (D // 16, 16)).amax(-1)
    x_new = torch.where(gmax > 0, _pow2_over(gmax, 6.0), 0).clamp(0, 11)
    x_out = torch.where(new5, x_new, torch.where(held, (was_x - fall).clamp(min=0), was_x))
    num = torch.where(new5, val, was) / torch.exp2(x_out.repeat_interleave(16, -1).float())
    code = _code4(num).unflatten(-1, (D // 2, 2))
    write = (new5 | held)
    cache[ids] = torch.where(write, code[..., 0] | (code[..., 1] << 4), codes)
    exps[ids] = torch.where(write[..., 0], (x_out << shift).sum(-1).to(torch.int32), ex)
    scale[ids] = now


def _ends_plain(c, lens, q_pos):
    """[B,S]: row s of a sequence sees keys [0, end)."""
    s = torch.arange(c["S"], device=DEV)
    end = lens.long()[:, None].expand(-1, c["S"])
    if q_pos is not None:
        seen = torch.div(q_pos.long()[:, None] + s + 1, c["ratio"], rounding_mode="floor")
        end = torch.minimum(end, seen).clamp(min=0)
    return end


def _softmax_times(score, ok, v):
    """Rows of score over the keys where ok, times v; a row with none gives zeros."""
    score = torch.where(ok, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total > 0, total, 1.0)


def _dense4(codes, exps, scale, table):
    """[B,Hkv,keys,D] float32 of the sequences' pages."""
    return _held4(codes[table], exps[table], scale[table]).transpose(1, 2).flatten(2, 3)


def _attn_plain(st, c):
    B, S, Hkv, D = c["B"], c["S"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    table = st["table"].long()
    k = _dense4(st["kc"], st["ke"], st["ks"], table)
    q = st["q"].float().view(B, S, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, D)
    score = torch.matmul(q * D ** -0.5, k.transpose(2, 3))                        # [B,Hkv,S*G,keys]
    del k
    end = _ends_plain(c, st["lens"], st["q_pos"]).repeat_interleave(G, 1)[:, None, :, None]
    ok = torch.arange(score.shape[-1], device=DEV) < end
    o = _softmax_times(score, ok, _dense4(st["vc"], st["ve"], st["vs"], table)).view(B, Hkv, S, G, D)
    return o.permute(0, 2, 1, 3, 4).reshape(B, S, c["Hq"], D).to(torch.bfloat16)


def _selected_plain(st, c):
    B, S, Hkv, D, PS, K = c["B"], c["S"], c["Hkv"], c["D"], c["PS"], c["topk"]
    G = c["Hq"] // Hkv
    idx = st["idx"].long()
    ok = (idx >= 0) & (idx < _ends_plain(c, st["lens"], st["q_pos"])[:, :, None])
    t = torch.where(ok, idx, 0)
    page = st["table"].long().gather(1, (t // PS).view(B, S * K)).view(B, S, K)
    head = torch.arange(Hkv, device=DEV)[:, None]
    cell = page[:, :, None] * Hkv + head                                          # [B,S,Hkv,K]
    row = cell * PS + (t % PS)[:, :, None]

    def dense(codes, exps, scale):
        return _unpack4(codes.view(-1, D // 2)[row], exps.view(-1)[row]) * scale.view(-1)[cell][..., None]

    q = st["q"].float().view(B, S, Hkv, G, D)
    score = torch.matmul(q * D ** -0.5, dense(st["kc"], st["ke"], st["ks"]).transpose(3, 4))
    o = _softmax_times(score, ok[:, :, None, None], dense(st["vc"], st["ve"], st["vs"]))
    return o.reshape(B, S, c["Hq"], D).to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    if c["op"] == "attn4" and work(c)["flops"] > 6e12:
        return None
    if c["op"] == "append" and c["B"] * c["S"] > 10000 * c["PS"]:  # it goes page by page
        return None
    st = prepare(c, seed)
    return {"axes": _axes_exact, "norm": _norm_exact, "append": _append_exact, "attn4": _attn_exact}[c["op"]](st, c)


def _pairs_of(c):
    half, o = c["R"] // 2, c["off"]
    i = torch.arange(half, device=DEV)
    return (o + 2 * i, o + 2 * i + 1) if c["layout"] == "interleaved" else (o + i, o + i + half)


def _units(st, c, inverse=False):
    """Unit complex numbers times the scale [B, S, 1, pairs]: pair (a, b) times exp(i angle)."""
    w = torch.from_numpy(_omega(c)).to(DEV)
    if st["pos"] is None:
        place = (st["start"].double()[:, None] + torch.arange(c["S"], device=DEV))[..., None]
    elif c["axes"] == 1:
        place = st["pos"].double()[..., None]
    else:
        place = torch.stack([st["pos"][a] for a in _axis_list(c)], -1).double()
    angle = place * w * (-1.0 if inverse else 1.0)
    return torch.polar(torch.full_like(angle, _mscale(c)), angle)[:, :, None]


def _turn_exact(y, unit, c):
    ia, ib = _pairs_of(c)
    z = torch.complex(y[..., ia], y[..., ib]) * unit
    y = y.clone()
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _axes_exact(st, c):
    unit = _units(st, c, c["back"])
    y = _turn_exact(st["x"].double(), unit, c)
    return y if st["x2"] is None else (y, _turn_exact(st["x2"].double(), unit, c))


def _normed(x):
    """x over its root mean square, and that root."""
    root = torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / x.shape[-1] + EPS)
    return x / root, root


def _norm_exact(st, c):
    unit = _units(st, c, c["back"])
    res = ()
    for name in ("", "2"):
        if st["x" + name] is None:
            continue
        n, root = _normed(st["x" + name].double())
        w = st["w" + name].double()
        if not c["back"]:
            res += (_turn_exact(n * w, unit, c),)
            continue
        u = _turn_exact(st["g" + name].double(), unit, c)
        t = w * u
        along = torch.linalg.vecdot(t, n)[..., None] / c["D"]
        res += ((t - n * along) / root, torch.einsum("bshd,bshd->d", u, n))
    return res if len(res) > 1 else res[0]


def _round_e4m3(x):
    """Nearest number of 1 + 4 + 3 bits (exponents from -6, steps of 2^-9 below), ties to even."""
    mag = x.abs().clamp(min=2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(mag)).clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _round_e2m1(x):
    """Nearest of 0 .5 1 1.5 2 3 4 6: steps of 1/2 to 2, of 1 to 4, of 2 above; ties to even."""
    a = x.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.round(x / step) * step


def _smallest_pow2(top, limit, least):
    """Smallest 2^e >= 2^least with top <= limit 2^e."""
    e = torch.ceil(torch.log2(top.clamp(min=limit * 2.0 ** least) / limit))
    e = torch.where(torch.exp2(e - 1) * limit >= top, e - 1, e)
    e = torch.where(torch.exp2(e) * limit < top, e + 1, e)
    return torch.exp2(e.clamp(min=least))


def _append_exact(st, c):
    PS, G = c["PS"], c["D"] // 16
    k = st["k"].double()
    if c["norm"]:
        k = _normed(k)[0] * st["w"].double()
    k = _turn_exact(k, _units(st, c), c)
    table, starts, counts = st["table"].tolist(), _starts(c), _counts(c)
    res, scales = [], []
    for x, cache, exps, scale in ((k, st["kc"], st["ke"], st["ks"]), (st["v"].double(), st["vc"], st["ve"], st["vs"])):
        scale = scale.double()
        if c["bits"] == 8:
            held = cache.double()
        else:
            held = _unpack4(cache, exps).double()
            unit = torch.exp2(((exps[..., None] >> (4 * torch.arange(G, device=DEV))) & 15).double())
        for b in range(c["B"]):
            lo, hi = starts[b], starts[b] + counts[b]
            for j in range(lo // PS, (hi - 1) // PS + 1):
                a, z = max(lo, j * PS), min(hi, j * PS + PS)
                t = x[b, a - lo:z - lo].transpose(0, 1)                           # [Hkv, tokens, D]
                s = _smallest_pow2(t.abs().amax((1, 2)), 448.0 if c["bits"] == 8 else 6.0 * 2.0 ** 11, -40)
                pid, n = table[b][j], max(0, lo - j * PS)
                if n:
                    s = torch.maximum(s, scale[pid])
                    fall = (scale[pid] / s)[:, None, None]
                    if c["bits"] == 8:
                        held[pid, :, :n] = _round_e4m3(held[pid, :, :n] * fall)
                    else:
                        m = (unit[pid, :, :n] * fall).clamp(min=1.0).repeat_interleave(16, -1)
                        held[pid, :, :n] = _round_e2m1(held[pid, :, :n] * fall / m) * m
                t = t / s[:, None, None]
                if c["bits"] == 8:
                    t = _round_e4m3(t)
                else:
                    m = _smallest_pow2(t.abs().unflatten(-1, (G, 16)).amax(-1), 6.0, 0).repeat_interleave(16, -1)
                    t = _round_e2m1(t / m) * m
                held[pid, :, a - j * PS:z - j * PS] = t
                scale[pid] = s
        res.append(held if c["bits"] == 8 else held / 32.0)
        scales.append(scale)
    return tuple(res + scales)


def _attn_exact(st, c):
    S, Hkv, D, PS = c["S"], c["Hkv"], c["D"], c["PS"]
    G = c["Hq"] // Hkv
    out = torch.zeros(c["B"], S, c["Hq"], D, dtype=torch.float64, device=DEV)
    number = torch.tensor([(-1.0 if n & 8 else 1.0) * (n % 2 * 0.5 if n & 7 < 2 else (1 + n % 2 * 0.5) * 2.0 ** ((n & 7) // 2 - 1))
                           for n in range(16)], dtype=torch.float64, device=DEV)

    def dense(codes, exps, scale, ids, n):
        x = torch.empty(codes[ids].shape[:-1] + (D,), dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = number[(codes[ids] % 16).int()], number[(codes[ids] // 16).int()]
        for i in range(D // 16):
            x[..., 16 * i:16 * i + 16] *= torch.exp2(((exps[ids] >> (4 * i)) & 15).double())[..., None]
        return (x * scale[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :n]

    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // PS)].long()
        kb, vb = dense(st["kc"], st["ke"], st["ks"], ids, n), dense(st["vc"], st["ve"], st["vs"], ids, n)
        ends = torch.tensor([_end(c, n, s) for s in range(S)], device=DEV)
        step = 64 if c["topk"] else 256
        for a in range(0, S, step):
            z = min(S, a + step)
            end = ends[a:z, None]
            for h in range(Hkv):
                q = st["q"][b, a:z, h * G:(h + 1) * G].double()                   # [rows, G, D]
                if c["topk"]:
                    t = st["idx"][b, a:z].long()
                    ok = (t >= 0) & (t < end)
                    t = t.clamp(0, n - 1)
                    score = torch.einsum("rgd,rkd->rgk", q, kb[h][t])
                else:
                    ok = torch.arange(n, device=DEV)[None] < end
                    score = torch.einsum("rgd,kd->rgk", q, kb[h])
                score = (score / math.sqrt(D)).masked_fill(~ok[:, None], float("-inf"))
                p = torch.nan_to_num(torch.softmax(score, -1), nan=0.0)
                eq, val = ("rgk,rkd->rgd", vb[h][t]) if c["topk"] else ("rgk,kd->rgd", vb[h])
                out[b, a:z, h * G:(h + 1) * G] = torch.einsum(eq, p, val)
    return out
