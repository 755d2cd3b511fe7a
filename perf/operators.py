"""Operators that stand next to the lightning indexer in a sparse-attention model, as cases.

Three operators that are used together when a model with a selected-key attention is served or
trained:

  rope    rotary positions of queries and keys, forward and backward
  append  writing new keys and values into a paged cache of 8-bit floating-point numbers that has
          one power-of-two scale for each page (block of tokens) and head
  attn    attention over that cache: all keys of a sequence, causal chunks of queries, or the keys
          that the indexer selected for each query row

Layouts: queries, keys and values [batch, token, head, dim]; the cache [page, head, slot, dim] in
float8_e4m3fn with scales [page, head] in float32; block_table int32 [batch, pages of a sequence].

A case is a dict of plain values; ``prepare`` makes what a caller holds before the call, ``run``
makes one call, in plain torch operations or, where ``own`` is set, through the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _rope(name, B, S, H, H2, D, R, off, layout, dtype, back, factor=1.0, top=8192):
    # top: positions lie below it; factor: long-context scaling of the frequencies
    return dict(name=name, op="rope", B=B, S=S, H=H, H2=H2, D=D, R=R, off=off, layout=layout,
                dtype=dtype, back=back, factor=factor, top=top)


def _append(name, B, S, Hkv, D, PS, top):
    # top: the longest sequence already holds about this many tokens
    return dict(name=name, op="append", B=B, S=S, Hkv=Hkv, D=D, PS=PS, top=top)


def _attn(name, B, S, Hq, Hkv, D, PS, L, ragged=False, causal=False, ratio=1, topk=0, hole=False):
    # L: longest sequence in the cache; topk: selected keys a row (0: all visible keys);
    # hole: the last sequence of a batch is empty
    return dict(name=name, op="attn", B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, PS=PS, L=L, ragged=ragged,
                causal=causal, ratio=ratio, topk=topk, hole=hole)


def listed():
    return [
        # one decode step of 16 sequences: 64 query heads and the one shared key, the last 64 of
        # 128 dims rotated, frequencies stretched for a long context; latency counts
        _rope("rope decode 16", 16, 1, 64, 1, 128, 64, 64, "interleaved", "bf16", False, 32.0, 131072),
        # the prompt of two sequences, sizes of the backward workload's rows
        _rope("rope prompt 2x8192", 2, 8192, 64, 1, 128, 64, 64, "interleaved", "bf16", False, 32.0, 16384),
        # gradients of a training step in 32 bits, whole heads in the half layout, grouped keys,
        # an odd number of tokens
        _rope("rope backward 4095 fp32", 1, 4095, 32, 8, 128, 128, 0, "half", "fp32", True),
        # one new token for each of 64 sequences; latency counts
        _append("append decode 64", 64, 1, 8, 128, 64, 8191),
        # ragged prompts of four sequences behind some tokens that are there already
        _append("append prompt 4x4097", 4, 4097, 8, 128, 128, 777),
        # one sequence with a short cache: latency counts
        _attn("attn decode 1x1024", 1, 1, 64, 8, 128, 64, 1024),
        # a serving batch of ragged lengths, grouped heads: bandwidth counts
        _attn("attn decode 64x32768 ragged", 64, 1, 64, 8, 128, 64, 32768, ragged=True),
        # few long sequences, all heads on one shared key head
        _attn("attn decode 4x131072 shared", 4, 1, 64, 1, 128, 128, 131072),
        # a chunk of a long prompt, causal over what the cache holds: tensor rate counts
        _attn("attn chunk 2048 of 16384", 1, 2048, 64, 8, 128, 64, 16384, causal=True),
        # small odd sizes: speculative tokens, heads that are no power of two, a narrow head
        # dimension, short pages, an empty sequence, rows with nothing to see
        _attn("attn odd 7x3", 7, 3, 20, 4, 80, 16, 1037, ragged=True, causal=True, hole=True),
        # decode over the keys that the indexer selected, one selection a sequence
        _attn("attn selected decode 32", 32, 1, 64, 1, 128, 64, 65536, ragged=True, topk=2048),
        # a prompt over selected compressed keys, sizes of the C4 layer workload
        _attn("attn selected prompt 4096", 1, 4096, 64, 1, 128, 64, 1024, causal=True, ratio=4, topk=512),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n + 1 if n == 3072 else n


def _draw_one(rng):
    kind = rng.choice(["rope", "append", "decode", "decode", "chunk", "selected", "selected"])
    if kind == "rope":
        B, S, D = rng.choice([1, 1, 2, 5, 16]), _log(rng, 1, 8192), rng.choice([32, 64, 80, 128])
        R = rng.choice([D, D // 2, max(2, D // 4)])
        return dict(op="rope", B=B, S=S, H=rng.choice([1, 8, 20, 32, 64]), H2=rng.choice([0, 1, 8]), D=D, R=R,
                    off=rng.choice([0, D - R]), layout=rng.choice(["interleaved", "half"]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), back=rng.random() < 0.4,
                    factor=rng.choice([1.0, 4.0, 32.0]), top=_log(rng, 2048, 262144))
    if kind == "append":
        return dict(op="append", B=_log(rng, 1, 128), S=_log(rng, 1, 8192), Hkv=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 80, 128]), PS=rng.choice([16, 32, 64, 128]), top=_log(rng, 2, 8192))
    Hkv = rng.choice([1, 1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 8, 12, 16]) if Hkv > 1 else rng.choice([8, 32, 48, 64, 128])
    c = dict(op="attn", B=_log(rng, 1, 64), S=1, Hq=G * Hkv, Hkv=Hkv, D=rng.choice([64, 80, 112, 128, 128]),
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
        if c["op"] == "attn":
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
    if c["op"] == "rope":
        n = c["B"] * c["S"] * (c["H"] + c["H2"])
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * n * c["D"] * size + 4.0 * c["B"] * c["S"], "flops": 3.0 * n * c["R"]}
    if c["op"] == "append":
        n = sum(_counts(c)) * c["Hkv"] * c["D"]
        return {"bytes": 2.0 * n * (2 + 1), "flops": 2.0 * 2 * n}
    lens = _lens(c)
    cap = c["topk"] or (1 << 62)
    pairs = sum(_pairs(c, n, cap) for n in lens)
    if c["topk"]:
        keys = sum(min(n, c["S"] * c["topk"]) for n in lens)
    else:
        keys = sum(_end(c, n, c["S"] - 1) for n in lens)
    rows = c["B"] * c["S"]
    nbytes = 2.0 * keys * c["Hkv"] * (c["D"] + 4.0 / c["PS"]) + 2.0 * 2 * rows * c["Hq"] * c["D"] + 4.0 * rows * c["topk"]
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


def _cache(g, pages, c):
    """A cache as it is found: every slot holds numbers, used or not."""
    shape = (pages, c["Hkv"], c["PS"], c["D"])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(100.0).clamp_(-448.0, 448.0)
    scale = torch.exp2(torch.randint(-8, -5, shape[:2], generator=g, device=DEV).float())
    return x.to(torch.float8_e4m3fn), scale


def _table(g, B, MP):
    return torch.randperm(B * MP, generator=g, device=DEV).to(torch.int32).view(B, MP)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, S = c["B"], c["S"]
        x = torch.randn(B, S, c["H"], c["D"], generator=g, device=DEV).to(dt)
        x2 = torch.randn(B, S, c["H2"], c["D"], generator=g, device=DEV).to(dt) if c["H2"] else None
        first = torch.randint(0, max(1, c["top"] - S), (B, 1), generator=g, device=DEV)
        pos = (first + torch.arange(S, device=DEV)).to(torch.int32)
        turns = np.rint(_omega(c) / (2 * math.pi) * 2.0 ** 64).astype(np.uint64).view(np.int64)
        return dict(c=c, x=x, x2=x2, pos=pos, freqs=torch.from_numpy(turns).to(DEV))
    if c["op"] == "append":
        B, S, Hkv, D, PS = c["B"], c["S"], c["Hkv"], c["D"], c["PS"]
        MP = (max(_starts(c)) + S) // PS + 3
        kc, ks = _cache(g, B * MP, c)
        vc, vs = _cache(g, B * MP, c)
        # the size of a token's values varies, so that some tokens outgrow their page's scale
        size = torch.exp(torch.randn(B, S, Hkv, 1, generator=g, device=DEV))
        k = (torch.randn(B, S, Hkv, D, generator=g, device=DEV) * size).to(torch.bfloat16)
        v = (torch.randn(B, S, Hkv, D, generator=g, device=DEV) * size).to(torch.bfloat16)
        return dict(c=c, k=k, v=v, kc=kc, vc=vc, ks=ks, vs=vs, table=_table(g, B, MP),
                    start=_int32(_starts(c)), count=_int32(_counts(c)))
    B, S = c["B"], c["S"]
    MP = _longest(c) // c["PS"]
    kc, ks = _cache(g, B * MP, c)
    vc, vs = _cache(g, B * MP, c)
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
    return dict(c=c, q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=_table(g, B, MP), lens=_int32(lens),
                q_pos=q_pos, idx=idx)


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["c"]
    if own:
        import sparse_attention_top_tcgen05_gb300 as lidx

        if c["op"] == "rope":
            call = lidx.lidx_rope_bwd if c["back"] else lidx.lidx_rope
            return call(st["x"], st["pos"], st["freqs"], x2=st["x2"], layout=c["layout"], rot_off=c["off"],
                        mscale=_mscale(c))
        if c["op"] == "append":
            lidx.lidx_cache_append(st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"],
                                   st["start"], count=st["count"])
            return st["kc"], st["vc"], st["ks"], st["vs"]
        return lidx.lidx_cache_attn(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["lens"],
                                    q_pos=st["q_pos"], compress_ratio=c["ratio"], topk_indices=st["idx"])[0]
    if c["op"] == "rope":
        return _rope_plain(st, c)
    if c["op"] == "append":
        _append_plain(st, st["k"], st["kc"], st["ks"])
        _append_plain(st, st["v"], st["vc"], st["vs"])
        return st["kc"], st["vc"], st["ks"], st["vs"]
    return _selected_plain(st, c) if c["topk"] else _attn_plain(st, c)


def _rotate(x, cos, sin, c):
    R, o = c["R"], c["off"]
    y = x.float()
    rot = y[..., o:o + R]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if c["layout"] == "interleaved" else (rot[..., :R // 2], rot[..., R // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    new = torch.stack((p, q), -1).flatten(-2) if c["layout"] == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((y[..., :o], new, y[..., o + R:]), -1).to(x.dtype)


def _rope_plain(st, c):
    # the product wraps at whole turns; its upper half is the angle, from half a turn back to half a turn
    turn = (st["pos"].long()[..., None] * st["freqs"]) >> 32
    angle = turn.float() * (2.0 * math.pi / 2.0 ** 32)
    m = _mscale(c)
    cos, sin = (angle.cos() * m)[:, :, None], (angle.sin() * (-m if c["back"] else m))[:, :, None]
    y = _rotate(st["x"], cos, sin, c)
    return y if st["x2"] is None else (y, _rotate(st["x2"], cos, sin, c))


def _append_plain(st, x, cache, scale):
    """Pages are worked on whole: the first J pages from the one that holds position start."""
    c, start, count, table = st["c"], st["start"].long(), st["count"].long(), st["table"].long()
    B, S, PS = c["B"], c["S"], c["PS"]
    J = (S + PS - 2) // PS + 1
    first = start // PS
    p = (first[:, None, None] + torch.arange(J, device=DEV)[None, :, None]) * PS + torch.arange(PS, device=DEV)
    i = p - start[:, None, None]                                              # [B,J,PS] token of the call
    new = (i >= 0) & (i < count[:, None, None])
    at = i.clamp(0, S - 1).view(B, J * PS, 1, 1).expand(-1, -1, x.shape[2], x.shape[3])
    val = x.float().gather(1, at).view(B, J, PS, x.shape[2], x.shape[3]).transpose(2, 3)
    new5 = new[:, :, None, :, None]
    amax = torch.where(new5, val, 0.0).abs().amax((3, 4))                     # [B,J,Hkv]
    # amax = m 2^x with m in [1/2, 1), and 448 = 7/8 2^9: the smallest e with amax <= 448 2^e
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - 9 + (m > 0.875).int(), -40).clamp(min=-40)
    want = torch.exp2(e.float())
    ids = table.gather(1, first[:, None] + torch.arange(J, device=DEV))
    old = scale[ids]
    kept = (p[:, :, 0] < start[:, None])[:, :, None]
    touched = new.any(2)[:, :, None]
    now = torch.where(touched, torch.where(kept, torch.maximum(old, want), want), old)
    was = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()      # [B,J,Hkv,PS,D]
    moved = (was * (old / now)[..., None, None])
    held = (p < start[:, None, None])[:, :, None, :, None] & touched[..., None, None]
    out = torch.where(new5, val / now[..., None, None], torch.where(held, moved, was))
    cache.view(torch.uint8)[ids] = out.to(torch.float8_e4m3fn).view(torch.uint8)
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


def _attn_plain(st, c):
    B, S, Hkv, D = c["B"], c["S"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    table = st["table"].long()

    def dense(cache, scale):
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    k = dense(st["kc"], st["ks"])
    q = st["q"].float().view(B, S, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, D)
    score = torch.matmul(q * D ** -0.5, k.transpose(2, 3))                        # [B,Hkv,S*G,keys]
    del k
    end = _ends_plain(c, st["lens"], st["q_pos"]).repeat_interleave(G, 1)[:, None, :, None]
    ok = torch.arange(score.shape[-1], device=DEV) < end
    o = _softmax_times(score, ok, dense(st["vc"], st["vs"])).view(B, Hkv, S, G, D)
    return o.permute(0, 2, 1, 3, 4).reshape(B, S, c["Hq"], D).to(torch.bfloat16)


def _selected_plain(st, c):
    B, S, Hkv, D, PS, K = c["B"], c["S"], c["Hkv"], c["D"], c["PS"], c["topk"]
    G = c["Hq"] // Hkv
    idx = st["idx"].long()
    ok = (idx >= 0) & (idx < _ends_plain(c, st["lens"], st["q_pos"])[:, :, None])
    t = torch.where(ok, idx, 0)
    page = st["table"].long().gather(1, (t // PS).view(B, S * K)).view(B, S, K)
    head = torch.arange(Hkv, device=DEV)[:, None]
    row = (page[:, :, None] * Hkv + head) * PS + (t % PS)[:, :, None]             # [B,S,Hkv,K]

    def dense(cache, scale):
        x = cache.view(torch.uint8).view(-1, D)[row].view(torch.float8_e4m3fn).float()
        return x * scale.view(-1)[page[:, :, None] * Hkv + head][..., None]

    q = st["q"].float().view(B, S, Hkv, G, D)
    score = torch.matmul(q * D ** -0.5, dense(st["kc"], st["ks"]).transpose(3, 4))
    o = _softmax_times(score, ok[:, :, None, None], dense(st["vc"], st["vs"]))
    return o.reshape(B, S, c["Hq"], D).to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    if c["op"] == "attn" and work(c)["flops"] > 6e12:
        return None
    st = prepare(c, seed)
    return {"rope": _rope_exact, "append": _append_exact, "attn": _attn_exact}[c["op"]](st, c)


def _rope_exact(st, c):
    w = torch.from_numpy(_omega(c)).to(DEV)
    sign = -1.0 if c["back"] else 1.0
    half, o = c["R"] // 2, c["off"]
    i = torch.arange(half, device=DEV)
    ia, ib = (o + 2 * i, o + 2 * i + 1) if c["layout"] == "interleaved" else (o + i, o + i + half)
    # unit complex numbers: pair (a, b) times exp(i angle)
    unit = torch.polar(torch.full_like(st["pos"], _mscale(c), dtype=torch.float64)[..., None].expand(-1, -1, half).contiguous(),
                       sign * st["pos"].double()[..., None] * w)[:, :, None]

    def turn(x):
        y = x.double()
        z = torch.complex(y[..., ia], y[..., ib]) * unit
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    y = turn(st["x"])
    return y if st["x2"] is None else (y, turn(st["x2"]))


def _round_e4m3(x):
    """Nearest number of 1 + 4 + 3 bits (exponents from -6, steps of 2^-9 below), ties to even."""
    mag = x.abs().clamp(min=2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(mag)).clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _append_exact(st, c):
    PS = c["PS"]
    table, starts, counts = st["table"].tolist(), _starts(c), _counts(c)
    res = []
    for x, cache, scale in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        cache, scale = cache.double(), scale.double()
        for b in range(c["B"]):
            lo, hi = starts[b], starts[b] + counts[b]
            for j in range(lo // PS, (hi - 1) // PS + 1):
                a, z = max(lo, j * PS), min(hi, j * PS + PS)
                t = x[b, a - lo:z - lo].double().transpose(0, 1)                  # [Hkv, tokens, D]
                top = t.abs().amax((1, 2)).clamp(min=448.0 * 2.0 ** -40)
                e = torch.ceil(torch.log2(top / 448.0))
                e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)
                s = torch.exp2(torch.where(torch.exp2(e) * 448.0 < top, e + 1, e)).clamp(min=2.0 ** -40)
                pid = table[b][j]
                if j * PS < lo:
                    s = torch.maximum(s, scale[pid])
                    n = lo - j * PS
                    cache[pid, :, :n] = _round_e4m3(cache[pid, :, :n] * (scale[pid] / s)[:, None, None])
                cache[pid, :, a - j * PS:z - j * PS] = _round_e4m3(t / s[:, None, None])
                scale[pid] = s
        res.append((cache, scale))
    return res[0][0], res[1][0], res[0][1], res[1][1]


def _attn_exact(st, c):
    S, Hkv, D, PS = c["S"], c["Hkv"], c["D"], c["PS"]
    G = c["Hq"] // Hkv
    out = torch.zeros(c["B"], S, c["Hq"], D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // PS)].long()
        kb, vb = ((cache[ids].double() * scale[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
                  for cache, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
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
