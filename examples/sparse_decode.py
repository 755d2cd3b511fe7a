"""A layer of sparse attention served with the library: prompt, then decode steps.

For each new token the path is
  rotary positions of the indexer's and the attention's queries and keys   lidx_rope
  selection of the compressed keys each query row reads                     lidx_indexer_fwd_ranges
  the new keys and values into the paged 8-bit cache                        lidx_cache_append
  attention over exactly the selected keys of that cache                    lidx_cache_attn

Inputs are random (there are no weights here); compressed keys come one for every `ratio` tokens, as they
would from a compressor.  The last step's output is checked against the same path in plain torch.

Run on a GB300:  python examples/sparse_decode.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_top_tcgen05_gb300 as lidx  # noqa: E402


class Layer:
    """Indexer keys and the paged 8-bit cache of a batch of sequences."""

    def __init__(self, B, heads, D, idx_heads, idx_D, ratio, topk, max_tokens, page=64, device="cuda"):
        self.B, self.H, self.D, self.HI, self.DI = B, heads, D, idx_heads, idx_D
        self.ratio, self.topk, self.page = ratio, topk, page
        pages = -(-(max_tokens // ratio) // page) + 1
        self.table = torch.randperm(B * pages, device=device).to(torch.int32).view(B, pages)
        f8 = lambda: torch.zeros(B * pages, 1, page, D, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.k8, self.v8 = f8(), f8()
        self.ks, self.vs = (torch.ones(B * pages, 1, device=device) for _ in (0, 1))
        self.idx_keys = torch.zeros(max_tokens // ratio + 1, B, idx_D, dtype=torch.bfloat16, device=device)
        # long-context frequencies: half of each head turns, in its last dims
        self.freqs = lidx.lidx_rope_freqs(D // 2, scaling="yarn", factor=8.0, device=device)
        self.idx_freqs = lidx.lidx_rope_freqs(idx_D // 2, scaling="yarn", factor=8.0, device=device)
        self.tokens = 0  # tokens so far; tokens // ratio of them have a compressed key

    def step(self, q, qi, w, k, v, ki):
        """S new tokens.  q [B,S,H,D], qi [S,B,HI,DI], w [S,B,HI] fp32; k, v [B,C,1,D] and ki [C,B,DI] for the C
        compressed keys that these tokens complete.  Returns the attention output [B,S,H,D] and the selection."""
        S, C, dev = q.shape[1], k.shape[1], q.device
        held, n = self.tokens // self.ratio, (self.tokens + S) // self.ratio
        assert C == n - held
        pos = torch.arange(self.tokens, self.tokens + S, dtype=torch.int32, device=dev)
        if C:
            kpos = torch.arange(held, n, dtype=torch.int32, device=dev) * self.ratio
            k = lidx.lidx_rope(k, kpos, self.freqs, rot_off=self.D // 2)
            ki = lidx.lidx_rope(ki[:, :, None], kpos[:, None], self.idx_freqs, rot_off=self.DI // 2)[:, :, 0]
            self.idx_keys[held:n] = ki
            start = torch.full((self.B,), held, dtype=torch.int32, device=dev)
            lidx.lidx_cache_append(k, v, self.k8, self.v8, self.ks, self.vs, self.table, start)
        q = lidx.lidx_rope(q, pos, self.freqs, rot_off=self.D // 2)
        qi = lidx.lidx_rope(qi, pos[:, None], self.idx_freqs, rot_off=self.DI // 2)
        # row s sees the compressed keys that are complete at its token
        ke = ((pos + 1) // self.ratio).to(torch.int32)
        idx, _, _ = lidx.lidx_indexer_fwd_ranges(qi, self.idx_keys, w, torch.zeros_like(ke), ke, self.topk)
        kv_len = torch.full((self.B,), n, dtype=torch.int32, device=dev)
        q_pos = torch.full((self.B,), self.tokens, dtype=torch.int32, device=dev)
        out, _ = lidx.lidx_cache_attn(q, self.k8, self.v8, self.ks, self.vs, self.table, kv_len, q_pos=q_pos,
                                      compress_ratio=self.ratio, topk_indices=idx)
        self.tokens += S
        return out, idx, q

    def plain(self, q, idx):
        """Attention of turned queries q over the selected cache entries, in plain torch."""
        n = self.tokens // self.ratio
        slot = torch.arange(n, device=q.device)
        page = self.table[:, slot // self.page].long()
        get = lambda c, s: c.float()[page, 0, slot % self.page] * s[page, 0][..., None]      # [B,n,D]
        k, v = get(self.k8, self.ks), get(self.v8, self.vs)
        ok = torch.zeros(q.shape[0], q.shape[1], n + 1, dtype=torch.bool, device=q.device)
        ok.scatter_(2, torch.where(idx < 0, n, idx).long(), True)
        s = torch.einsum("bshd,bnd->bshn", q.float(), k) * self.D ** -0.5
        s = s.masked_fill(~ok[:, :, None, :n], float("-inf"))
        return torch.einsum("bshn,bnd->bshd", torch.nan_to_num(torch.softmax(s, -1)), v)


def main(prompt=512, steps=9, verbose=True):
    B, H, D, HI, DI, ratio, topk = 2, 64, 128, 16, 64, 4, 48
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *n: torch.randn(*n, generator=g, device="cuda").to(torch.bfloat16)
    layer = Layer(B, H, D, HI, DI, ratio, topk, max_tokens=prompt + steps + ratio)
    worst = 0.0
    for S in [prompt] + [1] * steps:
        C = (layer.tokens + S) // ratio - layer.tokens // ratio
        w = torch.randn(S, B, HI, generator=g, device="cuda") / HI ** 0.5
        out, idx, q = layer.step(rnd(B, S, H, D), rnd(S, B, HI, DI), w, rnd(B, C, 1, D), rnd(B, C, 1, D), rnd(C, B, DI))
        want = layer.plain(q, idx)
        err = ((out.float() - want).norm() / want.norm()).item()
        worst = max(worst, err)
        if verbose:
            print(f"{S:4d} token(s), {layer.tokens // ratio:4d} compressed keys, relative difference {err:.2e}")
    assert lidx.lidx_device_status() == 0
    return worst


if __name__ == "__main__":
    from sparse_attention_top_tcgen05_gb300 import build

    build.build()
    main()
