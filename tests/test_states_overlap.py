"""CPU: what the state and cache operators refuse: buffers that overlap, and more layers than a position's blocks allow."""
from __future__ import annotations

import ctypes

import pytest

FAKE = 1 << 20  # never read: the checks come first
FAR = 1 << 30


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_61_gb300 import build
    build.build()
    import speculative_decoding_verification_61_gb300 as m
    return m


@pytest.mark.parametrize("which", ["rows", "offsets", "slots", "lengths"])
@pytest.mark.parametrize("at", [0, -4, 508])
def test_a_state_that_says_how_it_is_moved(sv, which, at):
    """4 slots of 128 bytes; an array of 4 entries (2 offsets) that starts in front of it, with it, with its last word."""
    from speculative_decoding_verification_61_gb300._binding import _State
    a = dict(rows=FAR, offsets=FAR + 4096, slots=FAR + 8192, lengths=None)
    a[which] = FAKE + at
    state = _State(FAKE, 1, 1, 8, 16)
    assert sv.lib().spec_state_reorder(ctypes.byref(state), 1, 4, a["rows"], a["offsets"], 1, 4, a["slots"], a["lengths"], None) == -1


@pytest.mark.parametrize("at,B,code", [(4, 2, -1), (-4, 2, -1), (4, 0, -1), (-12, 2, -1), (12, 2, -1), (0, 0, 0)])
def test_lengths_written_beside_themselves(sv, at, B, code):
    """4 lengths, and 4 to be written that start some bytes from them."""
    from speculative_decoding_verification_61_gb300._binding import _Cache, _Rows
    cache = _Cache(FAR, FAR, None, None, 1, 4, 16, 2, 64, None, 4, 1, FAKE)
    rows = _Rows(4, B, 8, FAR, None, None, 0)
    assert sv.lib().spec_cache_write(ctypes.byref(cache), FAR, None, 0, 128, 1, ctypes.byref(rows), None, None, None, FAKE + at, None) == code


@pytest.mark.parametrize("L,H,D,values,fits", [(1023, 4096, 16, True, True), (1024, 4096, 16, True, False), (2047, 4096, 16, False, True),
                                               (2048, 4096, 16, False, False), (2048, 64, 1024, True, False), (2047, 64, 1024, True, True)])
def test_a_positions_blocks(sv, L, H, D, values, fits):
    from speculative_decoding_verification_61_gb300._binding import _Cache
    cache = _Cache(FAR, FAR, FAR if values else None, FAR if values else None, L, 1, 1, H, D, None, 1, 1, FAKE)
    assert sv.lib().spec_cache_read(ctypes.byref(cache), FAR, 0, 8, None, None, 1, FAR, FAR if values else None, None) == (0 if fits else -1)
    if not fits:
        with pytest.raises(ValueError, match="invalid cache"):
            sv.CacheState(L, 1, 1, H, D, values=values, device="cpu")
