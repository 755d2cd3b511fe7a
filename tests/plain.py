"""Plain 64-bit definitions of the rotary, cache and attention operators, for the tests.

Written from the formulas on numpy arrays and CPU tensors, one sequence, page and row at a time."""

import math

import numpy as np
import torch

TWO_PI = 2.0 * math.pi


# ------------------------------------------------------------------ rotary

def rope_omega(R, theta=10000.0, scaling=None, factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "ntk" and R > 2:
        theta = theta * factor ** (R / (R - 2.0))
    w = theta ** (-2.0 * i / R)
    if scaling == "linear" or (scaling == "ntk" and R == 2):
        w = w / factor
    if scaling == "yarn":
        g = np.clip((original_len * w / TWO_PI - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        w = w * ((1.0 - g) / factor + g)
    return w


def rope(x, pos, omega, layout, off, mscale=1.0, inverse=False):
    """x [T0,T1,H,D] any float tensor, pos int [T0,T1]; returns float64 numpy."""
    x = x.double().cpu().numpy()
    y = x.copy()
    R = 2 * len(omega)
    ang = np.asarray(pos, np.float64)[:, :, None] * omega
    c, s = mscale * np.cos(ang), mscale * np.sin(ang) * (-1.0 if inverse else 1.0)
    for i in range(R // 2):
        ia, ib = (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + i + R // 2)
        ci, si = c[:, :, None, i], s[:, :, None, i]
        y[..., ia] = x[..., ia] * ci - x[..., ib] * si
        y[..., ib] = x[..., ib] * ci + x[..., ia] * si
    return y


# ------------------------------------------------------------------ cache

def e4m3_values():
    """The 256 numbers of e4m3 codes (1 sign, 4 exponent bits of bias 7, 3 fraction bits)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = f * 2.0 ** -9 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else m
        if c & 128:
            v[c] = -v[c]
    return v


E4M3 = e4m3_values()


def e4m3_round(x):
    """Codes (uint8) of the nearest e4m3 numbers, ties to the even code, saturating at +-448."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:127]  # 0 .. 448, increasing with the code
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(pos, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def pow2_scale(amax):
    """Smallest 2^e, e >= -40, with amax <= 448 * 2^e."""
    e = -40
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, cache, scale, table, start, count):
    """x [B,S,Hkv,D]; cache uint8 [P,Hkv,page,D], scale [P,Hkv]: numpy, updated in place."""
    x = x.double().cpu().numpy()
    P, Hkv, page, _ = cache.shape
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
                s = pow2_scale(max(np.abs(x[b, i, h]).max() for _, i in toks))
                if slot * page < start[b]:
                    s = max(s, scale[pid, h])
                    if s > scale[pid, h]:
                        n = int(start[b]) - slot * page
                        cache[pid, h, :n] = e4m3_round(E4M3[cache[pid, h, :n]] * (scale[pid, h] / s))
                for at, i in toks:
                    cache[pid, h, at] = e4m3_round(x[b, i, h] / s)
                scale[pid, h] = s


# ------------------------------------------------------------------ attention

def row_end(n, s, q_pos, ratio):
    if q_pos is None:
        return n
    return max(0, min(n, (q_pos + s + 1) // ratio))


def attention(q, kc, vc, ks, vs, table, kv_len, q_pos=None, ratio=1, idx=None, scale=None):
    """float64 (out [B,S,Hq,D], lse [B,S,Hq], slack [B,S,Hq,D], lse slack [B,S,Hq]).

    Derivation of the slack, what a correct kernel of 8-bit operands may be off by:
      * a score is an fp32 sum of D exact products that the tensor cores may add with as few as 13
        bits behind the largest partial sum, and a query element below 2^-11 of its row's largest
        keeps an error of 2^-17 of that: ds <= scale (2^-13 sum |q k| + 2^-17 max|q| sum |k|)
      * a weight is held as two 4-bit halves: relative error 2^-8
      * the output is rounded to bf16: 2^-8 of it
    so |do| <= 2^-8 |o| + sum p |v| (2^-8 + 2 max ds) + 2^-18 max|v| and |dlse| <= max ds + 2^-18 |lse| + 2^-18."""
    B, S, Hq, D = q.shape
    P, Hkv, page, _ = kc.shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((B, S, Hq, D)), np.full((B, S, Hq), -np.inf)
    slack, lslack = np.zeros((B, S, Hq, D)), np.zeros((B, S, Hq))
    qd = q.double().cpu().numpy()
    for b in range(B):
        n = int(min(max(int(kv_len[b]), 0), table.shape[1] * page))
        for s in range(S):
            end = row_end(n, s, None if q_pos is None else int(q_pos[b]), ratio)
            t = np.arange(end) if idx is None else np.asarray(idx[b, s], np.int64)
            t = t[(t >= 0) & (t < end)]
            pid = table[b, t // page].astype(np.int64)
            t, pid = t[(pid >= 0) & (pid < P)], pid[(pid >= 0) & (pid < P)]
            if len(t) == 0:
                continue
            for h in range(Hkv):
                k = E4M3[kc[pid, h, t % page]] * ks[pid, h].astype(np.float64)[:, None]
                v = E4M3[vc[pid, h, t % page]] * vs[pid, h].astype(np.float64)[:, None]
                rows = slice(h * G, (h + 1) * G)
                qq = qd[b, s, rows]
                sc = scale * (qq @ k.T)
                ds = abs(scale) * (2.0 ** -13 * (np.abs(qq) @ np.abs(k).T)
                                   + 2.0 ** -17 * np.abs(qq).max(1)[:, None] * np.abs(k).sum(1)).max(1)
                m = sc.max(1, keepdims=True)
                w = np.exp(sc - m)
                l = w.sum(1, keepdims=True)
                p = w / l
                out[b, s, rows] = p @ v
                lse[b, s, rows] = (m + np.log(l))[:, 0]
                slack[b, s, rows] = (2.0 ** -8 * np.abs(p @ v) + (p @ np.abs(v)) * (2.0 ** -8 + 2 * ds[:, None])
                                     + 2.0 ** -18 * np.abs(v).max())
                lslack[b, s, rows] = ds + 2.0 ** -18 * (np.abs(lse[b, s, rows]) + 1)
    return out, lse, slack, lslack


def random_cache(g, pages, Hkv, page, D, lo_exp=-8, hi_exp=-5):
    """Codes (uint8) and scales of a cache whose every slot holds a finite number."""
    codes = e4m3_round(g.standard_normal((pages, Hkv, page, D)) * 100.0)
    scale = np.exp2(g.integers(lo_exp, hi_exp + 1, (pages, Hkv))).astype(np.float32)
    return codes, scale


def to_cuda(codes):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)


def attention_cuda(q, kc, vc, ks, vs, table, kv_len, q_pos=None, ratio=1, idx=None):
    """attention()'s output in float64 torch operations on the GPU, for sizes the loops above are too slow for."""
    B, S, Hq, D = q.shape
    _, Hkv, page, _ = kc.shape
    G = Hq // Hkv
    out = torch.zeros(B, S, Hq, D, dtype=torch.float64, device=q.device)
    s = torch.arange(S, device=q.device)
    for b in range(B):
        n = int(kv_len[b])
        if n == 0:
            continue
        ids = table[b, :-(-n // page)].long()
        k, v = ((c[ids].double() * sc[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
                for c, sc in ((kc, ks), (vc, vs)))
        end = torch.full_like(s, n) if q_pos is None else ((int(q_pos[b]) + s + 1) // ratio).clamp(0, n)
        for a in range(0, S, 128):
            rows = slice(a, min(S, a + 128))
            qq = q[b, rows].double().view(-1, Hkv, G, D)
            if idx is None:
                sc = torch.einsum("rhgd,hkd->rhgk", qq, k)
                ok = (torch.arange(n, device=q.device) < end[rows, None])[:, None, None]
            else:
                t = idx[b, rows].long()
                ok = ((t >= 0) & (t < end[rows, None]))[:, None, None]
                t = t.clamp(0, n - 1)
                sc = torch.einsum("rhgd,hrkd->rhgk", qq, k[:, t])
            p = torch.nan_to_num(torch.softmax((sc * D ** -0.5).masked_fill(~ok, float("-inf")), -1))
            o = torch.einsum("rhgk,hkd->rhgd", p, v) if idx is None else torch.einsum("rhgk,hrkd->rhgd", p, v[:, t])
            out[b, rows] = o.reshape(-1, Hq, D)
    return out
