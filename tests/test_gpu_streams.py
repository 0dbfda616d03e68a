"""Calls on a stream other than the current one: the memory of the outputs that
they make.  It has to be the call's stream's own (a buffer that the current
stream has freed may still be in use there), and it must not come back from
the allocator while either stream may still use it."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def outputs(y):
    return [t for t in (y.values() if isinstance(y, dict) else y if isinstance(y, (tuple, list)) else [y])
            for t in (t.values() if isinstance(t, dict) else [t])]


def logit_calls(sv):
    R, V = 6, 1 << 18
    x = torch.randn(R, V, device="cuda")
    off, T = torch.arange(R + 1, dtype=torch.int32, device="cuda")[:4].contiguous(), torch.ones(3, device="cuda")
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    k = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    return {"process": lambda s: sv.spec_logits_process(x, off, tok, stream=s),
            "truncate": lambda s: sv.spec_logits_truncate(x, T, off, top_k=k, stream=s),
            "both": lambda s: sv.spec_logits_process_truncate(x, T, off, tok, top_k=k, stream=s)}


def check(call):
    """(The streams are idle wherever memory is taken from one and used on the other.)"""
    side = torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(None))]
    torch.cuda.synchronize()
    # buffers of the outputs' sizes that the current stream has freed
    freed = [torch.empty_like(t) for t in want for _ in range(4)]
    ptrs = {t.untyped_storage().data_ptr() for t in freed}
    del freed
    got = outputs(call(side))
    torch.cuda.synchronize()
    assert not ptrs & {t.untyped_storage().data_ptr() for t in got}
    for a, b in zip(got, want):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) if a.is_floating_point() else torch.equal(a, b)
    # the current stream reads them for another 20 ms or so: they stay its own until then
    torch.cuda._sleep(40_000_000)
    sizes = [t.shape for t in got]
    types = [t.dtype for t in got]
    ptrs = {t.untyped_storage().data_ptr() for t in got}
    del got
    with torch.cuda.stream(side):
        again = [torch.empty(s, dtype=d, device="cuda") for s, d in zip(sizes, types)]
    assert not ptrs & {t.untyped_storage().data_ptr() for t in again}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["process", "truncate", "both"])
def test_logit_outputs_on_another_stream(sv, name):
    check(logit_calls(sv)[name])


def verify_calls(sv):
    import workloads
    w = workloads.make_config(1)
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    tl, dl, ua, ur, ud, T, ko = (t(a) for a in (w.target_logits, w.draft_logits, w.u_accept, w.u_resample, w.u_draft, w.temperature, w.k_offsets))
    tok, lse = sv.spec_draft_sample_lse(dl, T, ud, ko)
    n = dl.shape[0]
    # a chain of the draft rows as one tree
    node_off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    parent = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
    one, ui = T[:1].clamp(min=0.5), ua.clone()
    B, V = T.numel(), tl.shape[1]
    bounds = [0, V]
    ws = sv.shard_workspace(B, V, 0)
    stats = sv.spec_shard_stats(tl, dl, tok, T, ko, bounds, 0, ws)

    def adapt(s):
        a = sv.AdaptiveK(B, 1, 4, stream=s)
        return a.k_offsets, a.state

    return {"draft": lambda s: sv.spec_draft_sample(dl, T, ud, ko, stream=s),
            "draft_lse": lambda s: sv.spec_draft_sample_lse(dl, T, ud, ko, stream=s),
            "verify": lambda s: sv.spec_verify(tl, dl, tok, ua, ur, T, ko, stream=s),
            "verify_aux": lambda s: sv.spec_verify(tl, dl, tok, ua, ur, T, ko, aux=True, stream=s),
            "verify_lse": lambda s: sv.spec_verify_lse(tl, dl, lse, tok, ua, ur, T, ko, aux=True, stream=s),
            "verify_noalloc": lambda s: sv.spec_verify_noalloc(tl, dl, tok, ua, ur, T, ko, stream=s),
            "round": lambda s: sv.spec_round(tl, dl, ud, ua, ur, T, ko, stream=s),
            "tree_draft": lambda s: sv.spec_tree_draft_sample(dl, node_off, parent, one, ui, stream=s),
            "tree_verify": lambda s: sv.spec_tree_verify(tl[:n].contiguous(), dl, node_off, parent, tok, ui, ui, one, stream=s),
            "shard_stats": lambda s: sv.spec_shard_stats(tl, dl, tok, T, ko, bounds, 0, ws, stream=s),
            "shard_decide": lambda s: sv.spec_shard_decide(tl, dl, stats, tok, ua, T, ko, bounds, 0, ws, stream=s),
            "adapt": adapt}


@pytest.mark.parametrize("name", ["draft", "draft_lse", "verify", "verify_aux", "verify_lse", "verify_noalloc", "round", "tree_draft",
                                  "tree_verify", "shard_stats", "shard_decide", "adapt"])
def test_outputs_on_another_stream(sv, name):
    call = verify_calls(sv)[name]
    torch.cuda.synchronize()  # the inputs are there
    check(call)


@pytest.mark.parametrize("name", ["process", "truncate", "both"])
def test_logit_outputs_on_a_forked_stream_of_a_capture(sv, name):
    """A captured call on a stream that the capture forked: its new output is the graph's, and replays rewrite it."""
    call, side = logit_calls(sv)[name], torch.cuda.Stream()
    want = call(None).clone()
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        other = call(side)
        torch.cuda.current_stream().wait_stream(side)
    assert got.data_ptr() != other.data_ptr()
    for _ in range(2):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want) and torch.equal(other, want)
    del got, other
    torch.cuda.synchronize()
    assert torch.equal(call(None), want)
