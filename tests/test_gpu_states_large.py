"""GPU: the reordering of states whose slots pass 4 GiB.  Bytes are moved, so every comparison is exact."""
from __future__ import annotations

import numpy as np
import pytest

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


@pytest.mark.parametrize("count", [(1 << 30) + 4, 1_250_000_000, 3_250_000_001])  # 4 GiB + 16 bytes, 5 GB, 13 GB in columns of 4 bytes
@pytest.mark.parametrize("lengths", [None, 1, 2 ** 31 - 1])
def test_whole_slots(sv, count, lengths):
    """Slots without positions, by all kinds of lengths that take the whole."""
    S = 3
    t = torch.zeros((S, count), dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 12345, 1 << 29, 1 << 30, count // 2, count - 5, count - 1], device="cuda")
    t[:, at] = torch.arange(1, S * len(at) + 1, device="cuda", dtype=torch.int32).view(S, len(at))
    before, held = t[:, at].clone(), int(t[0].count_nonzero())
    sv.spec_state_reorder([t], dev(np.array([2, 0, 0], i32)), dev(np.array([0, S], i32)),
                          lengths=None if lengths is None else dev(np.full(S, lengths, i32)))
    assert torch.equal(t[:, at], before[[2, 0, 0]])
    assert all(int(x.count_nonzero()) == held for x in t)


@pytest.mark.parametrize("lengths", [[2, 2, 2], [2 ** 31 - 1, 3, 1], [1, 0, -1]])
def test_positions_of_4_gib(sv, lengths):
    """Two positions of 4 GiB + 16 bytes each to a slot, as many moved as the source holds."""
    S, unit = 3, (1 << 30) + 4
    t = torch.zeros((S, 2, unit), dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 7, 1 << 29, unit - 1], device="cuda")
    t[:, :, at] = torch.arange(1, S * 2 * len(at) + 1, device="cuda", dtype=torch.int32).view(S, 2, len(at))
    want = t[:, :, at].clone()
    rows = [2, 0, 1]
    for s, source in enumerate(rows):
        n = min(2, max(0, lengths[source]))
        want[s, :n] = t[source, :n][:, at]
    sv.spec_state_reorder([(t, 0, 1)], dev(np.array(rows, i32)), dev(np.array([0, S], i32)), lengths=dev(np.array(lengths, i32)))
    assert torch.equal(t[:, :, at], want)
    assert int(t.count_nonzero()) == S * 2 * len(at)


def test_states_of_different_launches_that_overlap(sv):
    """More states than one launch takes, one of them twice (or a part of another): refused before anything is moved."""
    ts = [torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3) for _ in range(70)]
    rows, off = dev(np.array([1, 2, 3, 0], i32)), dev(np.array([0, 4], i32))
    for bad in (ts + ts[:1], ts + [ts[5].flatten()[4:8].view(4, 1)]):
        with pytest.raises(ValueError, match="overlap"):
            sv.spec_state_reorder(bad, rows, off)
    assert all(torch.equal(t, ts[0]) and int(t[0, 0]) == 0 for t in ts)
    sv.spec_state_reorder(ts + [torch.empty((4, 0), device="cuda")] * 2, rows, off)
    assert all(int(t[0, 0]) == 3 for t in ts)
