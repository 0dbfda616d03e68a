"""GPU: the reordering of states.  Bytes are moved, so every comparison is exact."""
from __future__ import annotations

import numpy as np
import pytest

import states_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

i32 = np.int32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def maps(kind, W, rng):
    if kind == "same":
        return np.arange(W)
    if kind == "one":
        return np.full(W, W - 1)
    if kind == "cycle":
        return np.roll(np.arange(W), 1)
    if kind == "cycles":  # several of them, and rows that hang on them
        m = rng.permutation(W)
        hang = rng.random(W) < 0.3
        return np.where(hang, rng.integers(0, W, W), m)
    if kind == "chain":
        return np.minimum(np.arange(W) + 1, W - 1)
    if kind == "back":
        return np.maximum(np.arange(W) - 1, 0)
    if kind == "swap":
        return np.arange(W) ^ 1 if W % 2 == 0 else np.arange(W)[::-1].copy()
    m = rng.integers(0, W, W)
    m[rng.random(W) < 0.2] = -1
    return m


@pytest.mark.parametrize("W", [1, 2, 3, 8, 9, 17, 64])
@pytest.mark.parametrize("kind", ["same", "one", "cycle", "cycles", "chain", "back", "swap", "any"])
def test_maps(sv, W, kind):
    """Three groups at scattered slots, columns of 16, 4 and 1 bytes, whole slots."""
    rng = np.random.default_rng(W + len(kind))
    off = np.array([0, W, W, 2 * W, 3 * W])
    S = 3 * W + 5
    slots = rng.permutation(S)[: 3 * W].astype(i32)
    rows = np.concatenate([np.where(m < 0, -1, m + g * W) for g, m in enumerate(maps(kind, W, rng) for _ in range(3))]).astype(i32)
    xs = [rng.integers(-9, 9, (S, 40)).astype(np.float32), rng.integers(0, 255, (S, 3, 7)).astype(np.uint8), rng.integers(-9, 9, (S, 3)).astype(i32),
          rng.integers(-9, 9, S).astype(np.int16)]
    ts = [dev(x) for x in xs]
    sv.spec_state_reorder(ts, dev(rows), dev(off.astype(i32)), slots=dev(slots))
    for x, t in zip(xs, ts):
        assert (t.cpu().numpy() == ref.reorder(x, rows, off, slots)).all()
    # without slots: the entries are the slots
    ts = [dev(x) for x in xs]
    sv.spec_state_reorder(ts, dev(rows), dev(off.astype(i32)))
    for x, t in zip(xs, ts):
        assert (t.cpu().numpy() == ref.reorder(x, rows, off)).all()


@pytest.mark.parametrize("W", [4, 12, 40])
@pytest.mark.parametrize("T,unit,runs", [(5, 16, 1), (300, 48, 1), (37, 20, 3), (64, 3, 2), (5000, 32, 1), (5, 8, 1), (1001, 24, 2), (333, 15, 1), (2000, 15, 1), (4096, 5, 1)])
def test_lengths(sv, W, T, unit, runs):
    """Ragged lengths (none, more than there is room for, negative) of states with layers before the slots
    and heads before the positions."""
    rng = np.random.default_rng(T + W)
    B = 3
    S = B * W
    off = np.arange(B + 1) * W
    x = rng.integers(0, 255, (S, 2, runs, T, unit)).astype(np.uint8)
    lengths = rng.integers(0, T + 1, S).astype(i32)
    lengths[::7], lengths[1::9], lengths[3::11], lengths[5::13] = 0, T, T + 100, -1
    slots = rng.permutation(S).astype(i32)
    for _ in range(3):
        rows = np.concatenate([np.where(m < 0, -1, m + g * W) for g, m in enumerate(maps(k, W, rng) for k in ("any", "cycle", "cycles"))]).astype(i32)
        t = dev(np.ascontiguousarray(x.transpose(1, 0, 2, 3, 4)))  # [layers, S, runs, T, unit]
        other = dev(x[:, 0, 0, 0, 0].copy())  # one without positions beside it
        sv.spec_state_reorder([(t, 1, 3), other], dev(rows), dev(off.astype(i32)), slots=dev(slots), lengths=dev(lengths))
        assert (t.cpu().numpy().transpose(1, 0, 2, 3, 4) == ref.reorder(x, rows, off, slots, lengths, 3)).all()
        assert (other.cpu().numpy() == ref.reorder(x[:, 0, 0, 0, 0], rows, off, slots, lengths)).all()


def test_groups_that_cannot_be(sv):
    """A slot out of range or twice, a row of another group: the group stays, the others do not."""
    x = np.arange(24 * 8, dtype=i32).reshape(24, 8)
    off = np.arange(0, 25, 4)
    rows = np.concatenate([np.roll(np.arange(4), 1) + 4 * g for g in range(6)]).astype(i32)
    rows[9], rows[14] = 3, -2
    slots = np.arange(24).astype(i32)
    slots[5], slots[17], slots[22] = 24, 18, -1
    t = dev(x)
    sv.spec_state_reorder([t], dev(rows), dev(off.astype(i32)), slots=dev(slots))
    want = ref.reorder(x, rows, off, slots)
    assert (t.cpu().numpy() == want).all() and (want != x).any()
    assert [(want[g * 4: g * 4 + 4] == x[g * 4: g * 4 + 4]).all() for g in range(6)] == [False, True, True, True, True, True]


@pytest.mark.parametrize("offsets", [[1, 4, 8], [0, 5, 4], [0, 4, 9], [0, 4, 2 ** 31 - 1]])
def test_invalid_offsets(sv, offsets):
    x = np.arange(64, dtype=i32).reshape(8, 8)
    t = dev(x)
    sv.spec_state_reorder([t], dev(np.roll(np.arange(8), 1).astype(i32)), dev(np.array(offsets, i32)))
    assert (t.cpu().numpy() == x).all()


def test_many_states_and_groups(sv):
    """More states than one launch takes, and the most groups."""
    rng = np.random.default_rng(2)
    x = rng.integers(0, 99, (12, 5)).astype(i32)
    ts = [dev(x + i) for i in range(130)]
    rows = np.array([1, 2, 0, 3, 3, 3, 6, 6, 8, 7, 9, -1], i32)
    off = np.array([0, 3, 6, 10, 12], i32)
    sv.spec_state_reorder(ts, dev(rows), dev(off))
    for i, t in enumerate(ts):
        assert (t.cpu().numpy() == ref.reorder(x + i, rows, off)).all()
    B = 4096
    x = rng.integers(0, 1 << 30, (2 * B, 3)).astype(i32)
    rows = (np.arange(2 * B) ^ (rng.random(2 * B) < 0.5)).astype(i32)
    off = np.arange(0, 2 * B + 1, 2)
    t = dev(x)
    sv.spec_state_reorder([t], dev(rows), dev(off.astype(i32)))
    assert (t.cpu().numpy() == ref.reorder(x, rows, off)).all()


def test_slots_past_32_bits(sv):
    """Slots of over 2^31 bytes each."""
    n = (1 << 29) + 4
    t = torch.zeros((4, n), dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 12345, n // 2, n - 5, n - 1], device="cuda")
    t[:, at] = torch.arange(24, device="cuda", dtype=torch.int32).view(4, 6)
    before = t[:, at].clone()
    sv.spec_state_reorder([t], dev(np.array([3, 0, 1, 2], i32)), dev(np.array([0, 4], i32)))
    assert torch.equal(t[:, at], before[[3, 0, 1, 2]])
    assert int(t.count_nonzero()) == 23


def test_penalty_state_follows(sv):
    """The counts and prompts of a group's hypotheses, by the state's own method."""
    st = sv.PenaltyState(6, 1000)
    st.reset(dev(np.arange(4).astype(i32)), dev(np.array([0, 2, 4, 4, 5], i32)), dev(np.array([1, 2, 3, 4, 999], i32)),
             dev(np.array([0, 1, 3, 3, 4], i32)), dev(np.array([7, 8, 8, 9], i32)))
    counts, seen = st.counts.clone(), st.seen.clone()
    st.reorder(dev(np.array([1, 0, 0, -1], i32)), dev(np.array([0, 4], i32)), slots=dev(np.array([0, 1, 2, 3], i32)))
    assert torch.equal(st.counts, counts[[1, 0, 0, 3, 4, 5]]) and torch.equal(st.seen, seen[[1, 0, 0, 3, 4, 5]])


def test_stream_and_capture(sv):
    rng = np.random.default_rng(4)
    x = rng.integers(0, 99, (16, 3000)).astype(i32)
    rows, off = rng.integers(0, 16, 16).astype(i32), np.array([0, 16], i32)
    once, twice = ref.reorder(x, rows, off), ref.reorder(ref.reorder(x, rows, off), rows, off)
    t, r, o = dev(x), dev(rows), dev(off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_state_reorder([t], r, o, stream=side)
    side.synchronize()
    assert (t.cpu().numpy() == once).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_state_reorder([t], r, o)
    assert (t.cpu().numpy() == once).all()
    g.replay()
    torch.cuda.synchronize()
    assert (t.cpu().numpy() == twice).all()


def test_binding_refusals(sv):
    t, r, o = torch.zeros(4, 8, device="cuda"), dev(np.zeros(4, i32)), dev(np.array([0, 4], i32))
    with pytest.raises(ValueError, match="slots"):
        sv.spec_state_reorder([t, torch.zeros(5, 8, device="cuda")], r, o)
    with pytest.raises(ValueError, match="contiguous"):
        sv.spec_state_reorder([torch.zeros(8, 4, device="cuda").t()], r, o)
    with pytest.raises(ValueError, match="dimension"):
        sv.spec_state_reorder([(t, 1, 1)], r, o)
    with pytest.raises(ValueError, match="entries"):
        sv.spec_state_reorder([t], r, o, slots=r[:3])
    with pytest.raises(TypeError):
        sv.spec_state_reorder([t], r.long(), o)
    with pytest.raises(sv.SpecError, match="INVALID"):
        sv.spec_state_reorder([t, t], r, o)
    assert sv.spec_state_reorder([], r, o) == []
