"""Beam search as a server runs it, step after step: logits processed with each hypothesis's own counts, the best
continuations selected, counts and cache put in the order of what was kept, the new token counted, its keys and values
written.  A toy model, whose logits and keys depend on the whole history, stands for the real one, and a plain search that keeps its
histories as lists says what has to come out."""
from __future__ import annotations

import numpy as np
import pytest

import states_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
V, W, B, STEPS, END = 1000, 4, 3, 8, 5
L, H, D = 2, 2, 64


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def model(history):
    """A token history's logits [V] and its last token's keys and values [2, L, H, D]."""
    rng = np.random.default_rng([len(history), *history])
    z = rng.standard_normal(V) * 2 - 1.1 * np.log1p(np.arange(V))
    z[END] += 3
    return z.astype(f32), rng.standard_normal((2, L, H, D)).astype(f32)


def test_steps(sv):
    R = B * W
    off = dev((np.arange(B + 1) * W).astype(i32))
    zeros, one_each = dev(np.zeros(R + 1, i32)), dev(np.zeros(R, i32))
    rng = np.random.default_rng(0)
    slots_h = rng.permutation(R + 3)[:R].astype(i32)
    slots = dev(slots_h)
    freq = np.full(R, 0.7, f32)
    st, cache = sv.PenaltyState(R + 3, V), sv.CacheState(L, R + 3, STEPS + 1, H, D)
    # the plain search: (score, history, ended) of every hypothesis
    plain = [[(0.0 if w == 0 else -np.inf, [100 + b], False) for w in range(W)] for b in range(B)]
    scores = dev(np.array([0 if w == 0 else -np.inf for _ in range(B) for w in range(W)], f32))
    ended = torch.zeros(R, dtype=torch.bool, device="cuda")
    histories = [[100 + r // W] for r in range(R)]
    for step in range(STEPS):
        # the model's forward pass on the device's hypotheses: logits, and the last token's keys and values into the cache
        made = [model(h) for h in histories]
        kv = np.stack([m[1] for m in made], 2)  # [2, L, R, H, D]
        cache.write(dev(kv[0]), dev(kv[1]), rows="next", slots=slots)
        z = sv.spec_logits_process(dev(np.stack([m[0] for m in made])), zeros, dev(np.zeros(0, i32)), rows="next", frequency=dev(freq), counts=st.counts,
                                   seen=st.seen, slots=slots)
        s, tokens, rows = sv.spec_beam_select(z, scores, off, W, ended=ended, end_token=END)
        rows, tokens, scores = rows.flatten(), tokens.flatten(), s.flatten().contiguous()
        st.reorder(rows, off, slots=slots)
        cache.reorder(rows, off, slots=slots)
        # tokens of hypotheses that go on are counted (a hypothesis that had ended counts its end once more, here as there)
        st.update(tokens, one_each, zeros, slots=slots)
        ended = tokens == END
        rh, th = rows.cpu().numpy(), tokens.cpu().numpy()
        histories = [histories[rh[r]] + [int(th[r])] for r in range(R)]
        # the same step in plain form
        for b in range(B):
            zs = np.full((W, V), 0, f32)
            for w, (score, h, _) in enumerate(plain[b]):
                c = np.bincount(h[1:], minlength=V).astype(f32)
                z0 = model(h)[0]
                zs[w] = np.where(c > 0, z0 - f32(0.7) * c, z0)
            sc = np.array([p[0] for p in plain[b]]).astype(f32)
            os, ot, orow = ref.beam_select(zs, sc, [0, W], W, np.array([p[2] for p in plain[b]]), END)[:3]
            assert np.diff(os[0]).max() < -1e-5  # no two so close that their order is open
            plain[b] = [(os[0, i], plain[b][orow[0, i]][1] + [int(ot[0, i])], ot[0, i] == END) for i in range(W)]
        assert histories == [h for b in range(B) for _, h, _ in plain[b]]
        # a step adds at most 130 roundings of 2^-24 of a score below 100 to the plain search's
        assert np.abs(scores.cpu().numpy() - [p[0] for b in range(B) for p in plain[b]]).max() <= (step + 1) * 130 * 100 * 2.0 ** -24
    # what the states hold is what the kept histories say
    counts = st.counts.cpu().numpy()
    lengths = np.full(R, STEPS, i32)
    assert (cache.lengths.cpu().numpy()[slots_h] == lengths).all()
    k, v = cache.read(dev((np.arange(R + 1) * STEPS).astype(i32)), R * STEPS, slots=slots, dtype=torch.float32)
    for r, h in enumerate(histories):
        assert (counts[slots_h[r]] == np.bincount(h[1:], minlength=V)).all()
        for step in range(STEPS):
            kv = model(h[: step + 1])[1]
            for got, x in zip((k, v), kv):
                assert (got[:, r * STEPS + step].double().cpu().numpy() == ref.dequantise(*ref.quantise(x))).all()


def test_a_verify_then_the_cache(sv):
    """A chain's and a tree's round: what the verify accepted, and nothing else, is in the cache."""
    import workloads
    rng = np.random.default_rng(1)
    w = workloads.make_config(1)
    t = dev
    draft = sv.spec_draft_sample(t(w.draft_logits), t(w.temperature), t(w.u_draft), t(w.k_offsets))
    tokens, n = sv.spec_verify(t(w.target_logits), t(w.draft_logits), draft, t(w.u_accept), t(w.u_resample), t(w.temperature), t(w.k_offsets))
    R = w.target_logits.shape[0]
    x = rng.standard_normal((L, R, H, D)).astype(f32)
    cache = sv.CacheState(L, w.B, 16, H, D)
    cache.write(dev(x), dev(x), t(w.k_offsets), num_accepted=n)
    nh = n.cpu().numpy()
    assert (cache.lengths.cpu().numpy() == nh + 1).all() and (nh > 0).any()
    off = np.concatenate([[0], np.cumsum(nh + 1)])
    k, _ = cache.read(dev(off.astype(i32)), int(off[-1]), dtype=torch.float32)
    rows = np.concatenate([w.k_offsets[b] + b + np.arange(nh[b] + 1) for b in range(w.B)])
    assert (k.double().cpu().numpy() == ref.dequantise(*ref.quantise(x[:, rows]))).all()
    # the tree of 3, 2 and 1 children, greedy
    parent = np.array([-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9])
    nodes, Bt = len(parent), 4
    node_off = (np.arange(Bt + 1) * nodes).astype(i32)
    par = np.concatenate([np.where(parent < 0, -1, parent + o) for o in node_off[:-1]]).astype(i32)
    N = Bt * nodes
    zt = rng.standard_normal((N, 64)).astype(f32)
    tok = rng.integers(0, 64, N).astype(i32)
    for b in range(Bt):  # some paths are the greedy ones
        node = node_off[b]
        for depth in range(b):
            node = next(c for c in range(N) if par[c] == node)
            tok[node] = zt[par[node]].argmax()
    u = np.zeros(N, f32)
    zero = dev(np.zeros(Bt, f32))
    _, n, last = sv.spec_tree_verify(dev(zt), dev(zt), dev(node_off), dev(par), dev(tok), dev(u), dev(u), zero)[:3]
    x = rng.standard_normal((L, N, H, D)).astype(f32)
    cache = sv.CacheState(L, Bt, 16, H, D)
    cache.write(dev(x), dev(x), dev(node_off), rows="tree", num_accepted=n, parent=dev(par), last_node=last)
    nh, lh = n.cpu().numpy(), last.cpu().numpy()
    assert (cache.lengths.cpu().numpy() == nh + 1).all() and nh.max() >= 3
    off = np.concatenate([[0], np.cumsum(nh + 1)])
    k, _ = cache.read(dev(off.astype(i32)), int(off[-1]), dtype=torch.float32)
    rows = np.concatenate([ref.tree_path(par, node_off[b], nodes, lh[b], nh[b]) for b in range(Bt)])
    assert (k.double().cpu().numpy() == ref.dequantise(*ref.quantise(x[:, rows]))).all()
