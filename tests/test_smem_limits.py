"""A kernel's limit of dynamic shared memory, where calls of one kernel ask for different sizes (appends: by the tokens of a
call) from several threads: it is never set below what has been recorded for the kernel."""

import os
import shutil
import subprocess
import sys

import pytest

from sparse_attention_top_tcgen05_gb300 import build as lidx_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The limit is a variable; setting the smaller size takes longer, so that it would come last were it not for the lock.
HOST = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_attr.h"

static lidx::SmemLimits<2, 2> limits;
static std::atomic<int> limit[2][3];
static std::atomic<int> calls;

int main() {
    const char fn[3] = {};
    auto want = [&](int dev, int k, int bytes) {
        return limits.ensure(dev, fn + k, bytes, [&](int b) {
            ++calls;
            if (b < 60000) std::this_thread::sleep_for(std::chrono::milliseconds(50));
            if (b == 77) return 1;
            limit[dev][k] = b;
            return 0;
        });
    };
    std::thread a([&] { want(0, 0, 51712); }), b([&] { want(0, 0, 66048); });
    a.join();
    b.join();
    if (want(0, 0, 66048) || limit[0][0] != 66048) return 1;
    const int before = calls;
    if (want(0, 0, 50000) || calls != before || limit[0][0] != 66048) return 2;  // covered
    if (want(1, 0, 50000) || limit[1][0] != 50000 || limit[0][0] != 66048) return 3;  // devices by themselves
    if (want(0, 1, 77) != 1 || want(0, 1, 70000) || limit[0][1] != 70000) return 4;  // a failure is no record
    if (want(0, 2, 70000) != -1 || limit[0][2] != 0) return 5;  // a full table
    if (want(0, 1, 80000) || limit[0][1] != 80000) return 6;
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_limits_on_the_host(tmp_path):
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(HOST)
    subprocess.run(["g++", "-O2", "-std=c++17", "-pthread", "-I", lidx_build.CSRC, str(src), "-o", str(exe)], check=True)
    for _ in range(5):
        assert subprocess.run([str(exe)], timeout=60).returncode == 0


# In a process of its own: the first calls of each kernel are what matters.
GPU = r"""
import threading
import torch
import sparse_attention_top_tcgen05_gb300 as lidx

DEV, Hkv, D, page = "cuda", 2, 128, 128
g = torch.Generator(device=DEV).manual_seed(1)
k = torch.randn(1, 128, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
start = torch.zeros(1, dtype=torch.int32, device=DEV)


def append(bits, S, R, off, layout):
    z = lambda *n, dt=torch.uint8: torch.zeros(*n, dtype=dt, device=DEV)
    f = lidx.lidx_rope_freqs(R)
    scales = [z(1, Hkv, dt=torch.float32) for _ in range(2)]
    if bits == 4:
        cache = [z(1, Hkv, page, D // 2) for _ in range(2)] + [z(1, Hkv, page, dt=torch.int32) for _ in range(2)] + scales
        lidx.lidx_cache4_append(k[:, :S], k[:, :S], *cache, table, start, freqs=f, rot_off=off, layout=layout)
    else:
        cache = [z(1, Hkv, page, D).view(torch.float8_e4m3fn) for _ in range(2)] + scales
        lidx.lidx_rope_cache_append(k[:, :S], k[:, :S], f, *cache, table, start, rot_off=off, layout=layout)
    torch.cuda.synchronize()
    return [t.view(torch.uint8) for t in cache]


for bits in (8, 4):
    for R, off, layout in ((128, 0, "half"), (128, 0, "interleaved"), (126, 1, "half")):
        got, gate = {}, threading.Barrier(2)

        def one(S):
            torch.cuda.set_device(0)
            gate.wait()
            got[S] = append(bits, S, R, off, layout)

        threads = [threading.Thread(target=one, args=(S,)) for S in (100, 128)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        for S in (128, 100):
            assert all(torch.equal(a, b) for a, b in zip(got[S], append(bits, S, R, off, layout))), (bits, R, S)
print("both sizes")
"""


@pytest.mark.gpu
def test_first_calls_of_two_sizes_from_two_threads():
    lidx_build.build()
    r = subprocess.run([sys.executable, "-c", GPU], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "both sizes" in r.stdout, r.stdout + r.stderr
