"""CPU checks of beam selection, the reordering of states and the 8-bit cache:
what the host refuses, and the restatements that the GPU tests compare with."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

import states_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
vp = ctypes.c_void_p
FAKE = 1 << 20  # never read: the checks come first


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_61_gb300 import build
    build.build()
    import speculative_decoding_verification_61_gb300 as m
    return m


def test_constants_match_the_header(sv):
    src = open(os.path.join(ROOT, "include", "spec_verify.h")).read()
    for name, value in (("SPEC_MAX_BEAMS", sv.MAX_BEAMS), ("SPEC_MAX_CANDIDATES", sv.MAX_CANDIDATES),
                        ("SPEC_MAX_STATES", sv.MAX_STATES), ("SPEC_ROWS_PROMPT", sv.CACHE_ROWS["prompt"])):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == value


def test_beam_workspace(sv):
    L = sv.lib()
    assert sv.beam_workspace_bytes(512, 128256, 1) >= 512 * 126 * 4
    assert sv.beam_workspace_bytes(8, 1001, 1) == 0  # rows that are not multiples of 16 bytes
    assert sv.beam_workspace_bytes(-1, 1000, 1) == 0 and L.spec_beam_workspace_bytes(8, 1000, 7) == 0
    assert sv.beam_workspace_bytes(0, 1000, 0) > 0


@pytest.mark.parametrize("change,code", [
    ({}, -5), (dict(B=-1), -1), (dict(B=4097), -1), (dict(R=-1), -1), (dict(n=0), -1), (dict(n=129), -1), (dict(dtype=2), -1),
    (dict(V=1002), -2), (dict(V=0), -1), (dict(logits=None), -1), (dict(scores=None), -1), (dict(offsets=None), -1),
    (dict(out=None), -1), (dict(ws=None), -1), (dict(logits=FAKE + 4), -2), (dict(ws=FAKE + 16), -2),
    (dict(ended=FAKE, end=-1), -1), (dict(ended=FAKE, end=1000), -1), (dict(B=0), 0)])
def test_beam_select_refusals(sv, change, code):
    a = dict(logits=FAKE, scores=FAKE, ended=None, end=0, offsets=FAKE, B=2, R=8, V=1000, dtype=0, n=8, out=FAKE, ws=FAKE)
    a.update(change)
    rc = sv.lib().spec_beam_select(a["logits"], a["scores"], a["ended"], a["end"], a["offsets"], a["B"], a["R"], a["V"], a["dtype"],
                                   a["n"], a["out"], a["out"], a["out"], None, a["ws"], 16, None)
    assert rc == code


def _state(sv, data=FAKE, planes=1, runs=1, T=8, unit=16):
    from speculative_decoding_verification_61_gb300._binding import _State
    return _State(data, planes, runs, T, unit)


@pytest.mark.parametrize("change,code", [
    (dict(n=65), -1), (dict(n=-1), -1), (dict(S=-1), -1), (dict(B=4097), -1), (dict(B=-1), -1), (dict(R=-1), -1),
    (dict(rows=None), -1), (dict(offsets=None), -1), (dict(states=[dict(data=None)]), -1), (dict(states=[dict(unit=-1)]), -1),
    (dict(states=[dict(T=1 << 32)]), -1), (dict(states=[dict(planes=1 << 40, unit=1 << 40)]), -1),
    (dict(states=[dict(), dict(data=FAKE + 8)]), -1),  # two that overlap
    (dict(states=[dict()], lengths=FAKE + 16), -1),  # the lengths among them
    (dict(B=0), 0), (dict(R=0), 0), (dict(n=0), 0), (dict(states=[dict(T=0)]), 0)])
def test_reorder_refusals(sv, change, code):
    a = dict(states=[dict()], S=4, rows=FAKE, offsets=FAKE, B=1, R=4, lengths=None)
    a.update(change)
    made = [_state(sv, **s) for s in a["states"]]
    arr = (type(made[0]) * len(made))(*made)
    rc = sv.lib().spec_state_reorder(arr, a.get("n", len(made)), a["S"], a["rows"], a["offsets"], a["B"], a["R"], None, a["lengths"], None)
    assert rc == code


def _cache(**change):
    from speculative_decoding_verification_61_gb300._binding import _Cache
    a = dict(k=FAKE, k_scale=FAKE, v=FAKE, v_scale=FAKE, L=1, P=4, T=16, H=2, D=64, pages=None, S=4, M=1, lengths=FAKE)
    a.update(change)
    return _Cache(*a.values())


CACHE_CHANGES = [
    (dict(D=63), -1), (dict(D=24), -1), (dict(D=1040), -1), (dict(H=1025, D=64), -1), (dict(L=-1), -1), (dict(P=-1), -1), (dict(T=0), -1),
    (dict(H=0), -1), (dict(S=3), -1), (dict(k=None), -1), (dict(k_scale=None), -1), (dict(lengths=None), -1), (dict(v_scale=None), -1),
    (dict(k=FAKE + 8), -2), (dict(v=FAKE + 8), -2), (dict(pages=FAKE, M=-1), -1)]


@pytest.mark.parametrize("change,code", CACHE_CHANGES)
def test_cache_refusals(sv, change, code):
    from speculative_decoding_verification_61_gb300._binding import _Rows
    c = ctypes.byref(_cache(**change))
    rows = _Rows(4, 2, 8, FAKE, None, None, 0)
    assert sv.lib().spec_cache_write(c, FAKE, FAKE, 0, 128, 1, ctypes.byref(rows), None, None, None, None, None) == code
    assert sv.lib().spec_cache_read(c, FAKE, 2, 8, None, None, 1, FAKE, FAKE, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(mode=1), -1), (dict(mode=5), -1), (dict(mode=-1), -1), (dict(B=-1), -1), (dict(B=4097), -1), (dict(R=-1), -1), (dict(dtype=2), -1),
    (dict(mode=0), -1), (dict(mode=0, n=FAKE, last=FAKE), -1), (dict(mode=3, n=FAKE), -1), (dict(mode=3, n=FAKE, last=FAKE), -1),
    (dict(n=FAKE), -1), (dict(offsets=None), -1), (dict(keys=None), -1), (dict(values=None), -1), (dict(keys=FAKE + 16), -2),
    (dict(values=FAKE + 16), -2), (dict(row=136), -2), (dict(layer=8), -2), (dict(row=112), -1), (dict(layer=-16), -1), (dict(B=0), 0)])
def test_write_refusals(sv, change, code):
    from speculative_decoding_verification_61_gb300._binding import _Rows
    a = dict(mode=4, B=2, R=8, offsets=FAKE, keys=FAKE, values=FAKE, layer=0, row=128, dtype=1, n=None, last=None)
    a.update(change)
    rows = _Rows(a["mode"], a["B"], a["R"], a["offsets"], None, None, 0)
    rc = sv.lib().spec_cache_write(ctypes.byref(_cache()), a["keys"], a["values"], a["layer"], a["row"], a["dtype"], ctypes.byref(rows),
                                   a["n"], a["last"], None, None, None)
    assert rc == code


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -1), (dict(B=4097), -1), (dict(R=-1), -1), (dict(R=0x7ffffff0), -1), (dict(dtype=5), -1), (dict(offsets=None), -1), (dict(keys=None), -1),
    (dict(values=None), -1), (dict(keys=FAKE + 16), -2), (dict(values=FAKE + 16), -2), (dict(B=0), 0), (dict(R=0), 0)])
def test_read_refusals(sv, change, code):
    a = dict(offsets=FAKE, B=2, R=8, dtype=1, keys=FAKE, values=FAKE)
    a.update(change)
    rc = sv.lib().spec_cache_read(ctypes.byref(_cache()), a["offsets"], a["B"], a["R"], None, None, a["dtype"], a["keys"], a["values"], None)
    assert rc == code


def test_binding_refuses_host_tensors(sv):
    torch = pytest.importorskip("torch")
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_beam_select(torch.zeros(4, 8), torch.zeros(4), i(2), 4)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_state_reorder([torch.zeros(4, 8)], i(4), i(2))
    cache = sv.CacheState(1, 4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        cache.write(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64), i(2), rows="prompt")
    with pytest.raises(ValueError, match="CUDA"):
        cache.read(i(2), 4)
    paged = sv.CacheState(1, 4, 16, 2, 64, pages=10, max_pages=3, device="cpu")
    assert paged.page_table.shape == (4, 3) and bool((paged.page_table == -1).all())
    with pytest.raises(ValueError, match="page table"):
        paged.reorder(i(4), i(2))
    for bad in (dict(D=40), dict(D=0), dict(T=0), dict(H=5000, D=64), dict(pages=3)):
        with pytest.raises(ValueError):
            sv.CacheState(**{**dict(L=1, S=4, T=16, H=2, D=64, device="cpu"), **bad})


# ------------------------------------------------------------ the restatements
def test_e4m3_is_torchs():
    """The grid and its rounding, at every border between neighbours, against torch's conversion."""
    torch = pytest.importorskip("torch")
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    y = np.concatenate([grid, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)]).astype(np.float32)
    y = np.concatenate([y, -y])
    assert (ref.to_e4m3(y.astype(np.float64)) == torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()).all()


def test_scales_are_the_least_that_hold():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 80)) * 2.0 ** rng.integers(-140, 120, (200, 1))).astype(np.float32)
    x[0] = 0
    x[1, 0], x[1, 1:32] = 448, 1
    x[2, 0], x[2, 1:32] = np.nextafter(np.float32(448), np.float32(500)), 1
    q, scale = ref.quantise(x)
    for j in range(3):
        big = np.abs(x[:, 32 * j: 32 * j + 32].astype(np.float64)).max(-1)
        e = scale[:, j].astype(np.int64) - 127
        assert (big <= 448 * 2.0 ** e).all() and ((e == -127) | (big > 448 * 2.0 ** (e - 1))).all()
    assert scale[1, 0] == 127 and scale[2, 0] == 128 and scale[0, 0] == 0
    # half a step of e4m3: 2^-4 of the value, or 2^-10 in units of the scale
    back = ref.dequantise(q, scale)
    unit = np.repeat(2.0 ** (scale.astype(np.int64) - 127), 32, -1)[:, :80]
    assert (np.abs(back - x) <= np.maximum(np.abs(x.astype(np.float64)) * 2.0 ** -4, unit * 2.0 ** -10)).all()


def test_beams_by_enumeration():
    """The restatement against a sort of all candidates of a group."""
    rng = np.random.default_rng(1)
    z = np.round(rng.standard_normal((6, 40)) * 2).astype(np.float32) / 2  # many ties
    s = np.array([0, -1, -1, -np.inf, -3, -0.5], np.float32)
    ended = np.array([0, 0, 1, 0, 0, 0], bool)
    os, ot, orow, lse = ref.beam_select(z, s, [0, 3, 3, 6], 50, ended, 7)[:4]
    p = np.log(np.exp(z.astype(np.float64)) / np.exp(z.astype(np.float64)).sum(1, keepdims=True))
    for b, rows in enumerate(([0, 1, 2], [], [3, 4, 5])):
        every = []
        for r in rows:
            if s[r] > -np.inf:
                every += [(s[r], r, 7)] if ended[r] else [(s[r] + p[r, v], r, v) for v in range(40)]
        every.sort(key=lambda x: (-round(x[0], 9), x[1], x[2]))
        n = min(50, len(every))
        assert np.allclose(os[b, :n], [e[0] for e in every[:n]], atol=1e-12) and (os[b, n:] == -np.inf).all()
        assert list(orow[b, :n]) == [e[1] for e in every[:n]] and list(ot[b, :n]) == [e[2] for e in every[:n]]
    assert np.isnan(lse[2]) and np.isnan(lse[3]) and np.isfinite(lse[[0, 1, 4, 5]]).all()
