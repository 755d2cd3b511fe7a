"""Capture of the rotary, cache and attention calls in a CUDA graph, whose replays read new inputs and lengths."""

import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


@pytest.mark.parametrize("S,Hq,Hkv,topk", [(1, 16, 2, 0), (1, 32, 1, 0), (3, 64, 1, 0), (40, 16, 4, 0), (1, 64, 1, 200),
                                           (2, 128, 1, 130), (1, 8, 1, 40)])
def test_step_in_a_graph(S, Hq, Hkv, topk):
    """rope, append and attention of a step, replayed with other queries, keys, positions, lengths and selections: the
    bits of the same calls made directly."""
    B, D, page, MP = 3, 128, 64, 64
    g = torch.Generator(device=DEV).manual_seed(Hq + S)
    rnd = lambda *n: torch.randn(*n, generator=g, device=DEV).to(torch.bfloat16)
    f8 = lambda: (torch.randn(B * MP, Hkv, page, D, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = lambda: torch.exp2(torch.randint(-9, -5, (B * MP, Hkv), generator=g, device=DEV).float())
    first = [f8(), f8(), scale(), scale()]
    table = torch.randperm(B * MP, generator=g, device=DEV).to(torch.int32).view(B, MP)
    freqs = lidx.lidx_rope_freqs(64)
    q, k, v = rnd(B, S, Hq, D), rnd(B, S, Hkv, D), rnd(B, S, Hkv, D)
    start = torch.zeros(B, dtype=torch.int32, device=DEV)
    idx = torch.zeros(B, S, topk, dtype=torch.int32, device=DEV) if topk else None

    def step(cache):
        pos = start[:, None] + torch.arange(S, dtype=torch.int32, device=DEV)
        qr, kr = lidx.lidx_rope(q, pos, freqs, x2=k, rot_off=64)
        lidx.lidx_cache_append(kr, v, *cache, table, start)
        return lidx.lidx_cache_attn(qr, *cache, table, start + S, q_pos=start, topk_indices=idx, want_lse=True)

    kept = [t.clone() for t in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kept)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(kept)
    for lens in ([0, 5, 100], [700, 3000, 64], [MP * page - S, 1, 129]):
        q.copy_(rnd(B, S, Hq, D)), k.copy_(rnd(B, S, Hkv, D)), v.copy_(rnd(B, S, Hkv, D))
        start.copy_(torch.tensor(lens, dtype=torch.int32))
        if topk:
            idx.copy_(torch.randint(-5, max(lens) + S, idx.shape, generator=g, device=DEV))
        direct = [t.clone() for t in first]
        want, wl = step(direct)
        for t, f in zip(kept, first):
            t.copy_(f)
        graph.replay()
        graph.replay()  # (the same tokens once more: the cache holds them already)
        assert torch.equal(out, want) and torch.equal(lse, wl)
        for a, b in zip(kept, direct):
            a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
            assert torch.equal(a, b)
    assert lidx.lidx_device_status() == 0
