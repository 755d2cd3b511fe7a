"""Plain 64-bit definitions of the 4-bit paged cache, for the tests: numbers, rounding, writing."""

import numpy as np

import plain

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def code4(x):
    """Codes (uint8) of the nearest 4-bit numbers, ties to the even code, saturating at +-6."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 6.0)
    hi = np.searchsorted(E2M1, a, side="left").clip(0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def pack(code):
    """[..., D] codes -> [..., D/2] bytes, the even dim low."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    out = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def exps_of(words, D):
    """int32 [...] -> [..., D/16]."""
    return (words.astype(np.int64)[..., None] >> (4 * np.arange(D // 16))) & 15


def pack_exps(x):
    w = (x.astype(np.int64) << (4 * np.arange(x.shape[-1]))).sum(-1)
    return np.where(w >= 2 ** 31, w - 2 ** 32, w).astype(np.int32)


def numbers(codes, words):
    """code * 2^x, NaN where x is not an exponent."""
    c = unpack(codes)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    x = np.repeat(exps_of(words, c.shape[-1]), 16, -1)
    return np.where(x < 12, v * 2.0 ** x, np.nan)


def smallest(amax, limit, least):
    """Smallest e >= least with amax <= limit * 2^e."""
    e = least
    while amax > limit * 2.0 ** e:
        e += 1
    return e


def encode(x, scale):
    """Rows x [..., D] at a scale -> codes [..., D/2], exponents [..., D/16] (15: not finite)."""
    g = x.reshape(x.shape[:-1] + (-1, 16)) / scale
    ok = np.isfinite(g).all(-1)
    top = np.where(ok, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0.0)
    e = np.zeros(top.shape, np.int64)
    for k in range(1, 12):
        e[top > 6.0 * 2.0 ** (k - 1)] = k
    code = code4(np.where(ok[..., None], g / 2.0 ** e[..., None], 0.0))
    return pack(code.reshape(x.shape)), np.where(ok, e, 15)


def append(x, codes, words, scale, table, start, count):
    """x [B,S,Hkv,D] float64; codes [P,Hkv,page,D/2], words int32 [P,Hkv,page], scale [P,Hkv]: updated in place."""
    P, Hkv, page, half = codes.shape
    B, S = x.shape[:2]
    for b in range(B):
        by_slot = {}
        for i in range(min(max(int(count[b]), 0), S)):
            p = int(start[b]) + i
            if p >= 0 and p // page < table.shape[1] and 0 <= table[b, p // page] < P:
                by_slot.setdefault(p // page, []).append((p % page, i))
        for slot, toks in by_slot.items():
            pid = int(table[b, slot])
            for h in range(Hkv):
                new = np.stack([x[b, i, h] for _, i in toks])
                fin = np.abs(new[np.isfinite(new)])
                s = 2.0 ** smallest(fin.max() if fin.size else 0.0, 6.0 * 2.0 ** 11, -40)
                if slot * page < start[b]:
                    old = float(scale[pid, h])
                    s = max(s, old)
                    if s > old:
                        n = int(start[b]) - slot * page
                        rise = smallest(old / s, 1.0, -200)
                        e = exps_of(words[pid, h, :n], 2 * half)
                        to = np.where(e < 12, np.maximum(e + rise, 0), e)
                        c = unpack(codes[pid, h, :n])
                        v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
                        f = np.repeat(np.where(e < 12, old / s * 2.0 ** (e - to), 1.0), 16, -1)
                        codes[pid, h, :n] = pack(code4(v * f))
                        words[pid, h, :n] = pack_exps(to)
                at = [a for a, _ in toks]
                c, e = encode(new, s)
                codes[pid, h, at], words[pid, h, at] = c, pack_exps(e)
                scale[pid, h] = s


def random_cache(g, pages, Hkv, page, D, lo_exp=-13, hi_exp=-10):
    """Codes, exponents and scales of a cache whose every slot holds finite numbers."""
    codes = pack(code4(g.standard_normal((pages, Hkv, page, D)) * 2.2))
    words = pack_exps(g.integers(0, 12, (pages, Hkv, page, D // 16)))
    scale = np.exp2(g.integers(lo_exp, hi_exp + 1, (pages, Hkv))).astype(np.float32)
    return codes, words, scale


def as_8(codes, words):
    """e4m3 codes (uint8) of code * 2^x / 32: an 8-bit cache of 32 times the scale."""
    v = numbers(codes, words) / 32.0
    out = plain.e4m3_round(np.where(np.isnan(v), 0.0, v))
    back = plain.E4M3[out]
    assert (back[~np.isnan(v)] == v[~np.isnan(v)]).all()
    c = unpack(codes)
    return np.where(np.isnan(v), 0x7F | np.where(c & 8, 128, 0), out).astype(np.uint8)
