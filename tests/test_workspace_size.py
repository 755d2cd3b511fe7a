"""A caller's workspace goes to the library with its own size, so one that is too small is refused before any launch
(LIDX_ERR_WORKSPACE) and not written past its end."""

import pytest
import torch

import sparse_attention_top_tcgen05_gb300 as lidx
from sparse_attention_top_tcgen05_gb300 import build as lidx_build
from test_streams import attn_args, bwd_args, fake, ranges, v4_args, v41_args


@pytest.fixture(scope="module", autouse=True)
def _built():
    lidx_build.build()
    lidx.lib()


NEED = 4096
CALLS = {
    "fwd": lambda ws: lidx.lidx_indexer_fwd(*v4_args(), 1, 3, workspace=ws),
    "fwd_ranges": lambda ws: lidx.lidx_indexer_fwd_ranges(*v4_args(), *ranges(), 3, workspace=ws),
    "scores_v41": lambda ws: lidx.lidx_indexer_scores_v41(*v41_args(), workspace=ws),
    "topk_v41": lambda ws: lidx.lidx_indexer_topk_v41(*v41_args(), 3, workspace=ws),
    "bwd": lambda ws: lidx.lidx_indexer_bwd(*bwd_args(), 1, workspace=ws),
    "bwd_ranges": lambda ws: lidx.lidx_indexer_bwd_ranges(*bwd_args(), *ranges(), workspace=ws),
    "cache_attn": lambda ws: lidx.lidx_cache_attn(*attn_args(), workspace=ws),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("nbytes", [64, NEED, 3 * NEED])
def test_the_size_that_the_library_is_told(monkeypatch, call, nbytes):
    told = []

    class FakeLib:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: NEED
            return lambda *a: told.append(a[-2]) or 0  # the stream comes last, the size before it

    monkeypatch.setattr(lidx, "_lib", FakeLib())
    monkeypatch.setattr(lidx, "lib", lambda: lidx._lib)
    monkeypatch.setattr(lidx, "_stream", lambda s: None)
    monkeypatch.setattr(lidx, "_raw_stream", lambda s, dev: 0)
    CALLS[call](fake(nbytes, dtype=torch.uint8))
    assert told == [nbytes]


@pytest.mark.gpu
def test_too_small_a_workspace_is_refused():
    import workloads

    wl = workloads.WORKLOADS["tiny"]
    q, k, w = (t.cuda() for t in workloads.v4_inputs(wl, 1))
    idx, sc, _ = lidx.lidx_indexer_fwd(q, k, w, wl.ratio, wl.topk)
    need = lidx.lidx_workspace_bytes(lidx.OP_INDEXER_BWD, wl.B, wl.S, k.shape[0], wl.H, q.shape[3], wl.topk)
    assert need > 256
    with pytest.raises(lidx.LidxError) as e:
        lidx.lidx_indexer_bwd(q, k, w, idx, torch.ones_like(sc), wl.ratio,
                              workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    want = lidx.lidx_indexer_bwd(q, k, w, idx, torch.ones_like(sc), wl.ratio)
    got = lidx.lidx_indexer_bwd(q, k, w, idx, torch.ones_like(sc), wl.ratio,
                                workspace=torch.empty(need + 4096, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
