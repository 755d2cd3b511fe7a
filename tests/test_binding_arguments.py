"""Arguments of the rotary and norm calls in Python: numbers that do not fit what goes to C, and outputs that are given."""

import math

import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_streams import fake

f32, i32 = torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(lidx, "_raw_stream", lambda s, dev: 0)


def args(H2=0):
    x = fake(1, 3, 2, 32, dtype=f32)
    return x, fake(1, 3, dtype=i32), fake(8, dtype=torch.int64), fake(1, 3, H2, 32, dtype=f32) if H2 else None


CALLS = {
    "rope": lambda x, pos, fr, **kw: lidx.lidx_rope(x, pos, fr, **kw),
    "rope_bwd": lambda x, pos, fr, **kw: lidx.lidx_rope_bwd(x, pos, fr, **kw),
    "norm": lambda x, pos, fr, **kw: lidx.lidx_norm_rope(x, None, pos, fr, **kw),
    "norm_bwd": lambda x, pos, fr, **kw: lidx.lidx_norm_rope_bwd(x, x, None, pos, fr, **kw),
    "append": lambda x, pos, fr, **kw: append(fr, pos=pos, **kw),
    "append, own positions": lambda x, pos, fr, **kw: append(fr, **kw),
}


def append(freqs, **kw):
    k, u8 = fake(1, 3, 2, 32), torch.uint8
    lidx.lidx_cache4_append(k, k, fake(2, 2, 16, 16, dtype=u8), fake(2, 2, 16, 16, dtype=u8), fake(2, 2, 16, dtype=i32),
                            fake(2, 2, 16, dtype=i32), fake(2, 2, dtype=f32), fake(2, 2, dtype=f32), fake(1, 2, dtype=i32),
                            fake(1, dtype=i32), freqs=freqs, **kw)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("mscale", [1e40, -1e300, math.inf, math.nan])
def test_a_scale_beyond_fp32_is_the_librarys_error(on_cpu, call, mscale):
    x, pos, freqs, _ = args()
    with pytest.raises(lidx.LidxError) as e:
        CALLS[call](x, pos, freqs, mscale=mscale)
    assert e.value.status == 2


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [dict(rot_off=2 ** 32), dict(rot_off=-2 ** 40), dict(rot_off=1.5), dict(mscale="1"), dict(mscale=10 ** 400)])
def test_numbers_that_are_none_of_c(on_cpu, call, kw):
    x, pos, freqs, _ = args()
    with pytest.raises(ValueError):
        CALLS[call](x, pos, freqs, **kw)


@pytest.fixture
def told(monkeypatch):
    """The norm tensors that go to C, as (y, dw) pointers of each."""
    seen = []

    class FakeLib:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096

            def call(arr, nt, *a):
                t = (lidx._NormTensor * nt).from_buffer_copy(arr)
                seen.append([(s.y, s.dw) for s in t])
                return 0
            return call

    monkeypatch.setattr(lidx, "_raw_stream", lambda s, dev: 0)
    monkeypatch.setattr(lidx, "_lib", FakeLib())
    return seen


def test_outputs_that_are_given_in_part(told):
    """What is given is written, what is None is made."""
    x, pos, freqs, x2 = args(H2=1)
    w, dx, dw, dx2, dw2 = (fake(*s, dtype=f32) for s in ((32,), x.shape, (32,), x2.shape, (32,)))
    given = (dx, dw, dx2, dw2)
    for mask in range(16):
        out = tuple(t if mask >> i & 1 else None for i, t in enumerate(given))
        got = lidx.lidx_norm_rope_bwd(x, x, w, pos, freqs, g2=x2, x2=x2, weight2=w, out=out)
        flat = [p for pair in told[-1] for p in pair]
        assert len(got) == 4
        for i, (o, t) in enumerate(zip(out, got)):
            assert t.shape == given[i].shape and t.dtype == f32 and flat[i] == t.data_ptr()
            assert o is None or t is o
    y = fake(*x2.shape, dtype=f32)
    got = lidx.lidx_norm_rope(x, w, pos, freqs, x2=x2, weight2=w, out=(None, y))
    assert got[1] is y and got[0].shape == x.shape and told[-1] == [(got[0].data_ptr(), None), (y.data_ptr(), None)]
    # without a weight its gradient is written where it is asked for
    assert lidx.lidx_norm_rope_bwd(x, x, None, pos, freqs)[1] is None and told[-1][0][1] is None
    assert lidx.lidx_norm_rope_bwd(x, x, None, pos, freqs, out=(None, dw))[1] is dw and told[-1][0][1] == dw.data_ptr()


@pytest.mark.parametrize("count,n,call", [
    (2, 1, lambda o, x, p, f, x2: lidx.lidx_norm_rope(x, None, p, f, x2=x2, out=o)),
    (2, 3, lambda o, x, p, f, x2: lidx.lidx_norm_rope(x, None, p, f, x2=x2, out=o)),
    (2, 1, lambda o, x, p, f, x2: lidx.lidx_norm_rope_bwd(x, x, None, p, f, out=o)),
    (2, 4, lambda o, x, p, f, x2: lidx.lidx_norm_rope_bwd(x, x, None, p, f, out=o)),
    (4, 2, lambda o, x, p, f, x2: lidx.lidx_norm_rope_bwd(x, x, None, p, f, g2=x2, x2=x2, out=o)),
])
def test_another_number_of_outputs(told, count, n, call):
    x, pos, freqs, x2 = args(H2=2)
    with pytest.raises(ValueError, match=f"out has {n} tensors, not {count}"):
        call((x,) * n, x, pos, freqs, x2)
