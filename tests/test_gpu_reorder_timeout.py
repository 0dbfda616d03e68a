"""A reordering whose waits for the copy engine run out: on the GPU waits for an arrival that nothing makes, which
give up, leave the states as they were and are reported; and what the host refuses."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

i32 = np.int32


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_61_gb300 import build
    build.build()
    import speculative_decoding_verification_61_gb300 as m
    return m


def test_refusals(sv):
    from speculative_decoding_verification_61_gb300._binding import _State
    assert sv.lib().spec_state_reorder_status(None, 0) == -1
    fake = 1 << 20
    state = _State(None, 1, 1, 8, 16)
    assert sv.lib().spec_selfcheck_reorder_timeout(ctypes.byref(state), 1, 4, fake, fake, 1, 4, None, None, None) == -1
    assert sv.lib().spec_selfcheck_reorder_timeout(ctypes.byref(state), 1, 4, fake, fake, 4097, 4, None, None, None) == -1
    with pytest.raises(ValueError, match="CUDA"):
        sv.selfcheck_reorder_timeout(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("count", [64, 1 << 18])  # one chunk of a slot's bytes, and several to a CTA
def test_waits_give_up_and_report(sv, count):
    dev = lambda a: torch.from_numpy(np.asarray(a, i32)).cuda()  # noqa: E731
    assert sv.state_reorder_status() == 0
    t = torch.arange(4 * count, dtype=torch.int32, device="cuda").view(4, count)
    before = t.clone()
    rows, offsets = dev([1, 2, 3, 0]), dev([0, 4])
    sv.selfcheck_reorder_timeout(t, rows, offsets)
    assert sv.state_reorder_status() == -4  # SPEC_ERR_TIMEOUT
    assert torch.equal(t, before)
    assert sv.state_reorder_status(clear=True) == -4 and sv.state_reorder_status() == 0
    # the context is usable, and the next call moves
    sv.spec_state_reorder([t], rows, offsets)
    assert torch.equal(t, before[[1, 2, 3, 0]]) and sv.state_reorder_status() == 0
