"""Calls on a stream of the caller's choice: what they allocate themselves must belong to that stream.

torch's allocator hands a freed block out again at once to the stream it was allocated on.  A call that takes its
scratch from the current stream's pool and works on another stream would give a block back that its kernels still use,
and could be given one that the current stream's kernels still use."""

import contextlib
import types

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


# ------------------------------------------------------------------ CPU: whose pool an allocation comes from

class FakeCuda(torch.Tensor):
    """A CPU tensor that the binding's checks take for a CUDA tensor."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(FakeCuda)


@pytest.fixture
def pools(monkeypatch):
    """Runs the binding without a GPU; the list gets the name of the current stream at each allocation."""
    log, current = [], ["main"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.name)
        yield
        current.pop()

    def logged(make):
        def wrap(*a, **kw):
            log.append(current[-1])
            return make(*a, **kw)
        return wrap

    class FakeLib:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("workspace_bytes") else (lambda *a: 0)

    monkeypatch.setattr(torch, "empty", logged(torch.empty))
    monkeypatch.setattr(torch, "empty_like", logged(torch.empty_like))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: types.SimpleNamespace(name=f"raw {raw}"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    monkeypatch.setattr(lidx, "_raw_stream", lambda s, dev: 0)
    monkeypatch.setattr(lidx, "_stream", lambda s: None)
    monkeypatch.setattr(lidx, "_lib", FakeLib())
    monkeypatch.setattr(lidx, "lib", lambda: lidx._lib)
    return log


f8, i32, f32 = torch.float8_e4m3fn, torch.int32, torch.float32


def rope_args():
    return (fake(2, 3, 4, 16), fake(2, 3, dtype=i32), fake(8, dtype=torch.int64))


def attn_args():
    return (fake(1, 2, 4, 16), fake(3, 2, 16, 16, dtype=f8), fake(3, 2, 16, 16, dtype=f8), fake(3, 2, dtype=f32),
            fake(3, 2, dtype=f32), fake(1, 2, dtype=i32), fake(1, dtype=i32))


def v4_args():
    return fake(4, 2, 8, 32), fake(6, 2, 32), fake(4, 2, 8, dtype=f32)


def v41_args():
    return fake(2, 4, 8, 32), fake(2, 6, 32), fake(2, 4, 8), fake(2, 4, 6, dtype=torch.bool)


def ranges():
    return fake(4, dtype=i32), fake(4, dtype=i32)


def bwd_args():
    return (*v4_args(), fake(2, 4, 3, dtype=i32), fake(2, 4, 3, dtype=f32))


CALLS = {
    "fwd": (lambda **kw: lidx.lidx_indexer_fwd(*v4_args(), 1, 3, **kw), 3),
    "fwd logits": (lambda **kw: lidx.lidx_indexer_fwd(*v4_args(), 1, 3, materialise_logits=True, **kw), 4),
    "fwd_ranges": (lambda **kw: lidx.lidx_indexer_fwd_ranges(*v4_args(), *ranges(), 3, **kw), 3),
    "fwd_noalloc": (lambda **kw: lidx.lidx_indexer_fwd_noalloc(*v4_args(), 1, 3, **kw), 2),
    "logits": (lambda **kw: lidx.lidx_indexer_logits(*v4_args(), **kw), 1),
    "extract": (lambda **kw: lidx.lidx_extract_topk_scores(fake(2, 4, 6, dtype=f32), fake(2, 4, 3, dtype=i32), **kw), 1),
    "topk_rows": (lambda **kw: lidx.lidx_topk_rows(fake(2, 4, 6, dtype=f32), 3, **kw), 2),
    "scores_v41": (lambda **kw: lidx.lidx_indexer_scores_v41(*v41_args(), **kw), 2),
    "topk_v41": (lambda **kw: lidx.lidx_indexer_topk_v41(*v41_args(), 3, **kw), 4),
    "topk_v41 no scores": (lambda **kw: lidx.lidx_indexer_topk_v41(*v41_args(), 3, keep_scores=False, **kw), 3),
    "bwd": (lambda **kw: lidx.lidx_indexer_bwd(*bwd_args(), 1, **kw), 4),
    "bwd_ranges": (lambda **kw: lidx.lidx_indexer_bwd_ranges(*bwd_args(), *ranges(), **kw), 4),
    "rope": (lambda **kw: lidx.lidx_rope(*rope_args(), **kw), 1),
    "rope x2": (lambda **kw: lidx.lidx_rope(*rope_args(), x2=fake(2, 3, 1, 16), **kw), 2),
    "rope strided": (lambda **kw: lidx.lidx_rope(fake(3, 2, 4, 16).transpose(0, 1), *rope_args()[1:], **kw), 1),
    "rope_bwd": (lambda **kw: lidx.lidx_rope_bwd(*rope_args(), **kw), 1),
    "cache_attn": (lambda **kw: lidx.lidx_cache_attn(*attn_args(), **kw), 2),
    "cache_attn lse": (lambda **kw: lidx.lidx_cache_attn(*attn_args(), want_lse=True, **kw), 3),
    "cache_attn out, lse wanted": (
        lambda **kw: lidx.lidx_cache_attn(*attn_args(), out=(fake(1, 2, 4, 16), None), want_lse=True, **kw), 2),
    "cache_attn out": (lambda **kw: lidx.lidx_cache_attn(*attn_args(), out=(fake(1, 2, 4, 16), None), **kw), 1),
}


@pytest.mark.parametrize("call", CALLS)
def test_allocations_belong_to_the_stream_of_the_call(pools, call):
    fn, n = CALLS[call]
    fn()
    assert pools == ["main"] * n
    pools.clear()
    fn(stream=types.SimpleNamespace(cuda_stream=7))
    assert pools == ["raw 7"] * n


def test_a_wanted_log_sum_exp_is_returned_beside_a_given_output(pools):
    o = fake(1, 2, 4, 16)
    got, lse = lidx.lidx_cache_attn(*attn_args(), out=(o, None), want_lse=True)
    assert got is o and lse is not None and lse.shape == (1, 2, 4)
    assert lidx.lidx_cache_attn(*attn_args(), out=(o, None))[1] is None


# ------------------------------------------------------------------ GPU

def _case(seed, B, Hq, Hkv, n, page=64, D=128):
    g = torch.Generator(device=DEV).manual_seed(seed)
    MP = -(-n // page)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    kc, vc = ((rnd(B * MP, Hkv, page, D) * 100).clamp(-448, 448).to(f8) for _ in (0, 1))
    ks, vs = (torch.exp2(torch.randint(-9, -5, (B * MP, Hkv), generator=g, device=DEV).float()) for _ in (0, 1))
    table = torch.randperm(B * MP, generator=g, device=DEV).to(i32).view(B, MP)
    lens = torch.full((B,), n, dtype=i32, device=DEV)
    return rnd(B, 1, Hq, D).to(torch.bfloat16), kc, vc, ks, vs, table, lens


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (64, 2), (80, 1)])
def test_scratch_is_not_handed_out_while_the_call_runs(Hq, Hkv):
    """The stream of the call is held up; meanwhile the current stream allocates and fills blocks of the scratch's
    size.  Neither may show in the other."""
    args = _case(Hq, 2, Hq, Hkv, 9000)
    want, wl = lidx.lidx_cache_attn(*args, want_lse=True)
    size = lidx.lidx_cache_attn_workspace_bytes(2, 1, Hq, Hkv, 128)
    st = torch.cuda.Stream()
    for _ in range(3):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got, gl = lidx.lidx_cache_attn(*args, want_lse=True, stream=st)
        mine = [torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        st.synchronize()
        assert all(bool((m == 0xA5).all()) for m in mine)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    assert lidx.lidx_device_status() == 0


@pytest.mark.gpu
def test_scratch_of_the_indexer_calls():
    """The same for the fused forward and its backward, whose scratch holds logits and partial gradients."""
    import workloads

    wl = workloads.WORKLOADS["tiny"]
    q, k, w = (t.to(DEV) for t in workloads.v4_inputs(wl, 5))
    grad = torch.randn(wl.B, wl.S, wl.topk, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)

    def both(stream=None):
        idx, sc, _ = lidx.lidx_indexer_fwd(q, k, w, wl.ratio, wl.topk, stream=stream)
        return (idx, sc, *lidx.lidx_indexer_bwd(q, k, w, idx, grad, wl.ratio, stream=stream))

    want = both()
    D = q.shape[3]
    sizes = [lidx.lidx_workspace_bytes(op, wl.B, wl.S, k.shape[0], wl.H, D, wl.topk)
             for op in (lidx.OP_INDEXER_FWD, lidx.OP_INDEXER_BWD)]
    st = torch.cuda.Stream()
    for _ in range(3):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)
        got = both(st)
        mine = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes * 2 if n]
        torch.cuda.current_stream().synchronize()
        st.synchronize()
        assert all(bool((m == 0xA5).all()) for m in mine)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert lidx.lidx_device_status() == 0


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams, each with its own scratch, while the other runs."""
    a, b = _case(1, 3, 48, 1, 20000), _case(2, 2, 16, 2, 30000)
    want = [lidx.lidx_cache_attn(*x)[0] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, x in enumerate((a, b)):
            got[i].append(lidx.lidx_cache_attn(*x, stream=streams[i])[0])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])
    assert lidx.lidx_device_status() == 0


@pytest.mark.gpu
def test_fresh_outputs_of_another_stream_outlive_their_reader():
    """An output that the caller drops while the current stream still reads it is not overwritten by the next call."""
    g = torch.Generator(device=DEV).manual_seed(3)
    freqs = lidx.lidx_rope_freqs(64)
    pos = torch.arange(512, dtype=i32, device=DEV)
    xs = [torch.randn(1, 512, 16, 64, generator=g, device=DEV) for _ in range(4)]
    want = [lidx.lidx_rope(x, pos, freqs) for x in xs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = []
    for x in xs:
        y = lidx.lidx_rope(x, pos, freqs, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda._sleep(10_000_000)  # the reader comes late
        got.append(y.clone())
        del y
    assert all(torch.equal(a, b) for a, b in zip(got, want))
