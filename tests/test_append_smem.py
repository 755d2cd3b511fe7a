"""Appends whose shared memory is just what a kernel may have without asking for more (48 KB), or a few bytes less or more: 95
tokens of 128 dims, all turned, in a page of 128, have angles and weights of 48 KB exactly, and the block's maxima beside
them.  The limit stays raised once a larger call has raised it, so the sizes are met in a process of their own, in order."""

import os
import subprocess
import sys

import pytest

from sparse_attention_top_tcgen05_gb300 import build as lidx_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUN = r"""
import sys
sys.path.insert(0, "tests")
import test_rope_append as t

for S in (94, 95, 96):
    t.CASES = [(1, S, 2, 128, 128, [0], None)] * 3
    for bits in (4, 8):
        for layout in ("interleaved", "half"):
            t.test_turned_keys_against_the_definition(0, bits, True, 1, True, layout)

import torch
import sparse_attention_top_tcgen05_gb300 as lidx

# pairs that lie anyhow: 64 tokens of 126 turned dims
g = torch.Generator(device="cuda").manual_seed(1)
k = torch.randn(1, 65, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
z = lambda *n, dt=torch.uint8: torch.zeros(*n, dtype=dt, device="cuda")
freqs, zero = lidx.lidx_rope_freqs(126), z(1, dt=torch.int32)


def append(S):
    c4 = [z(1, 2, 128, 64), z(1, 2, 128, 64), z(1, 2, 128, dt=torch.int32), z(1, 2, 128, dt=torch.int32)]
    c8 = [z(1, 2, 128, 128).view(torch.float8_e4m3fn) for _ in range(2)]
    s4, s8 = ([z(1, 2, dt=torch.float32) for _ in range(2)] for _ in range(2))
    lidx.lidx_cache4_append(k[:, :S], k[:, :S], *c4, *s4, zero[None], zero, freqs=freqs, rot_off=1, layout="half")
    lidx.lidx_rope_cache_append(k[:, :S], k[:, :S], freqs, *c8, *s8, zero[None], zero, rot_off=1, layout="half")
    torch.cuda.synchronize()
    return [t.view(torch.uint8) for t in c4 + c8 + s4 + s8]


first = {S: append(S) for S in (63, 64, 65)}
for S, got in first.items():
    assert all(torch.equal(a, b) for a, b in zip(got, append(S))), S
print("all sizes")
"""


@pytest.mark.gpu
def test_sizes_around_the_limit():
    lidx_build.build()
    r = subprocess.run([sys.executable, "-c", RUN], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all sizes" in r.stdout, r.stdout + r.stderr
