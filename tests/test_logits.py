"""Logit operators on the CPU: the plain restatements pinned by hand, and the
refusals that the host makes before any CUDA call."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import logits_ref as ref

f32 = np.float32


# ------------------------------------------------------- the restatement, by hand
def test_process_by_hand():
    z = np.array([[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]], f32)
    rows = ref.Rows("target", np.array([0, 1]), np.array([0]))
    p = dict(repetition=f32([2.0]), frequency=f32([0.25]), presence=f32([1.0]),
             counts=np.array([[0, 3, 0, 0]], np.int32),
             seen=ref.pack(np.array([[[0, 0, 1, 0], [0, 1, 0, 0]]], bool)))
    out, ref64, _ = ref.process(z, rows, p, ref.F32)
    # row 0: token 1 emitted three times, token 2 in the prompt; row 1 also follows the drafted token 0
    assert out[0].tolist() == [2.0, -4.0 - 0.75 - 1.0, 0.5, 0.5]
    assert out[1].tolist() == [1.0 - 0.25 - 1.0, -5.75, 0.5, 0.5]
    assert (out == ref64).all()


def test_process_bias_and_mask_by_hand():
    z = np.array([[1.0, 2.0, np.nan, np.inf]], f32)
    rows = ref.Rows("next", np.array([0, 0]), np.zeros(0, np.int64))
    p = dict(bias_offsets=np.array([0, 3]), bias_tokens=np.array([1, 0, 1]), bias_values=f32([0.5, -np.inf, 0.25]),
             mask=ref.pack(np.array([[1, 1, 0, 0]], bool)))
    out, _, _ = ref.process(z, rows, p, ref.F32)
    assert out[0].tolist() == [-np.inf, 2.75, -np.inf, -np.inf]


def test_tree_rows_by_hand():
    # root 0, children 1 and 2, node 3 under 1
    rows = ref.Rows("tree", np.array([0, 4]), np.array([9, 5, 6, 7]), np.array([-1, 0, 0, 1]))
    assert [sorted(p) for _, p in rows] == [[], [5], [6], [5, 7]]


def test_truncate_by_hand():
    z = np.log(np.array([[1, 4, 2, 1, 2]], f32))  # masses 0.1 0.4 0.2 0.1 0.2: order 1, 2, 4, 0, 3
    one, seq = np.array([1.0]), [0]
    kept = lambda **kw: np.flatnonzero(np.isfinite(ref.truncate(z, seq, one, **kw)[0][0])).tolist()  # noqa: E731
    assert kept(top_k=[2]) == [1, 2]
    assert kept(top_k=[4]) == [0, 1, 2, 4]  # a tie goes to the lowest index
    assert kept(top_p=[0.39]) == [1]
    assert kept(top_p=[0.55]) == [1, 2]
    assert kept(top_p=[0.85]) == [0, 1, 2, 4]
    assert kept(top_k=[2], top_p=[0.6]) == [1]  # of 0.6: 0.36 is reached by the first token
    assert kept(min_p=[0.45]) == [1, 2, 4]
    assert kept(top_p=[1e-30]) == [1]


def test_pack_round_trip():
    bits = np.random.default_rng(0).random((3, 77)) < 0.5
    words = ref.pack(bits)
    assert words.shape == (3, 3) and words.dtype == np.int32
    assert (ref.unpack(words, 77) == bits).all()
    assert words[0, 1] & 1 == bits[0, 32]


# --------------------------------------------------------------- refusals (host)
@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_61_gb300 import build
    build.build()
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


FAKE = 1 << 20  # never read: the checks come first


def structs(sv, **kw):
    from speculative_decoding_verification_61_gb300 import _binding as bd
    rows = dict(rows=0, B=2, R=4, offsets=FAKE, parent=None, draft_tokens=FAKE, n_tokens=2)
    proc = dict(counts=FAKE, seen=FAKE, S=2)
    trunc = dict(temperature=FAKE)
    for k, v in kw.items():
        (rows if k in rows else trunc if k in ("temperature", "top_k", "top_p", "min_p") else proc)[k] = v
    return bd._Rows(**rows), bd._Logits(**proc), bd._Truncate(**trunc)


def call(sv, name, logits=FAKE, out=FAKE + (1 << 24), V=1000, dtype=0, **kw):
    rw, ps, tr = structs(sv, **kw)
    args = {"process": (rw, ps), "truncate": (rw, tr), "process_truncate": (rw, ps, tr)}[name]
    return getattr(sv.lib(), "spec_logits_" + name)(logits, *(ctypes.byref(a) for a in args), V, dtype, out, None)


@pytest.mark.parametrize("name", ["process", "truncate", "process_truncate"])
def test_row_refusals(sv, name):
    assert call(sv, name, dtype=7) == -1
    assert call(sv, name, B=-1) == -1
    assert call(sv, name, B=sv.MAX_B + 1) == -1
    assert call(sv, name, V=0) == -1
    assert call(sv, name, V=sv.MAX_V + 8) == -1
    assert call(sv, name, V=1001) == -2
    assert call(sv, name, V=1004, dtype=1) == -2
    assert call(sv, name, rows=4) == -1
    assert call(sv, name, rows=-1) == -1
    assert call(sv, name, R=-1) == -1
    assert call(sv, name, n_tokens=-1) == -1
    assert call(sv, name, logits=None) == -1
    assert call(sv, name, out=None) == -1
    assert call(sv, name, offsets=None) == -1
    assert call(sv, name, logits=FAKE + 8) == -2
    assert call(sv, name, out=FAKE + (1 << 24) + 4) == -2
    # an output that overlaps the logits but is not the logits
    assert call(sv, name, out=FAKE + 16) == -1
    assert call(sv, name, out=FAKE - 16) == -1
    assert call(sv, name, out=FAKE + 4 * 1000 * 4 - 16) == -1
    # nothing to do
    assert call(sv, name, B=0, logits=None, out=None, offsets=None) == 0
    assert call(sv, name, R=0, logits=None, out=None, offsets=None) == 0


@pytest.mark.parametrize("name", ["process", "process_truncate"])
def test_process_refusals(sv, name):
    assert call(sv, name, seen=None) == -1
    assert call(sv, name, S=-1) == -1
    assert call(sv, name, draft_tokens=None) == -1
    assert call(sv, name, rows=3) == -1  # a tree's penalties without parent
    assert call(sv, name, counts=None) == -1  # seen without counts
    for only in ("repetition", "frequency", "presence", "slots"):
        assert call(sv, name, counts=None, seen=None, **{only: FAKE}) == -1
    assert call(sv, name, bias_tokens=FAKE) == -1
    assert call(sv, name, bias_offsets=FAKE, n_bias=3) == -1
    assert call(sv, name, bias_offsets=FAKE, n_bias=-1) == -1
    assert call(sv, name, mask_rows=FAKE) == -1
    assert call(sv, name, mask=FAKE, M=3) == -1  # fewer masks than rows
    assert call(sv, name, mask=FAKE, mask_rows=FAKE, M=-1) == -1


def test_truncate_refusals(sv):
    assert call(sv, "truncate", temperature=None) == -1
    assert call(sv, "process_truncate", temperature=None) == -1
    assert sv.lib().spec_logits_truncate(FAKE, ctypes.byref(structs(sv)[0]), None, 1000, 0, FAKE, None) == -1
    assert sv.lib().spec_logits_process(FAKE, None, ctypes.byref(structs(sv)[1]), 1000, 0, FAKE, None) == -1


def test_state_refusals(sv):
    L = sv.lib()
    rw = structs(sv)[0]
    up = lambda S=2, V=1000, counts=FAKE, rows=rw, toks=FAKE: L.spec_penalty_update(  # noqa: E731
        counts, FAKE, S, V, None, ctypes.byref(rows), toks, FAKE, None)
    assert up(S=-1) == -1 and up(V=0) == -1 and up(V=sv.MAX_V + 1) == -1
    assert up(counts=None) == -1 and up(toks=None) == -1
    assert up(rows=structs(sv, rows=1)[0]) == -1 and up(rows=structs(sv, rows=2)[0]) == -1
    assert up(rows=structs(sv, offsets=None)[0]) == -1
    assert up(rows=structs(sv, B=0)[0]) == 0
    re = lambda S=2, V=1000, slots=FAKE, n=1, po=FAKE, pt=FAKE, npr=4: L.spec_penalty_reset(  # noqa: E731
        FAKE, FAKE, S, V, slots, n, po, pt, npr, None, None, 0, None)
    assert re(S=-1) == -1 and re(V=0) == -1 and re(n=-1) == -1 and re(n=sv.MAX_B + 1) == -1
    assert re(slots=None) == -1 and re(pt=None) == -1 and re(npr=-1) == -1
    assert re(n=0) == 0


def test_binding_refusals(sv):
    torch = pytest.importorskip("torch")
    z, off = torch.zeros(2, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_logits_process(z, off, off)
    with pytest.raises(ValueError, match="rows"):
        sv.spec_logits_process(z, off, off, rows="all")
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_logits_truncate(z, torch.ones(1), off)
    with pytest.raises(ValueError, match=r"\[rows, V\]"):
        sv.spec_logits_truncate(z[0], torch.ones(1), off)
    with pytest.raises(ValueError):
        sv.PenaltyState(0, 16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        sv.PenaltyState(2, 16, device="cpu").reset(off)
    assert sv.ROWS == {"target": 0, "draft": 1, "next": 2, "tree": 3}


class Sized:
    """A tensor of a given size as the binding's checks see one, without its memory."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda = shape, dtype, True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape, dtype=np.int64))

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return FAKE


def test_binding_refuses_counts_past_31_bits(sv):
    """What the C ABI takes as an int: a larger number would arrive as another one."""
    torch = pytest.importorskip("torch")
    from speculative_decoding_verification_61_gb300 import _binding as bd
    i32, fl = torch.int32, torch.float32
    most = (1 << 31) - 1
    off, z = Sized((3,), i32), Sized((4, 8), fl)
    for n in (most + 1, 1 << 32, (1 << 32) + 4):
        with pytest.raises(ValueError, match="2147483647"):
            bd._rows_arg(Sized((n, 8), fl), off, "target", None, None, i32)
        with pytest.raises(ValueError, match="2147483647"):
            bd._rows_arg(Sized((4, n), fl), off, "target", None, None, i32)
        with pytest.raises(ValueError, match="2147483647"):
            bd._state_arg(Sized((2, n), i32), Sized((2, 2, 1), i32), i32)
        with pytest.raises(ValueError, match="2147483647"):
            bd._rows_arg(z, off, "target", Sized((n,), i32), None, i32)
        rw = bd._rows_arg(z, off, "target", Sized((2,), i32), None, i32)
        lists = dict.fromkeys(("repetition", "frequency", "presence", "counts", "seen", "slots", "bias_offsets", "bias_tokens",
                               "bias_values", "mask", "mask_rows"))
        for big in (dict(counts=Sized((n, 8), i32), seen=Sized((n, 2, 1), i32)),
                    dict(bias_offsets=off, bias_tokens=Sized((n,), i32), bias_values=Sized((n,), fl)),
                    dict(mask=Sized((n, 1), i32), mask_rows=Sized((4,), i32))):
            with pytest.raises(ValueError, match="2147483647"):
                bd._logits_arg(z, rw, "target", Sized((2,), i32), None, **{**lists, **big}, i32=i32, f32=fl)
        with pytest.raises(ValueError, match="2147483647"):
            bd._state_arg(Sized((n, 8), i32), Sized((n, 2, 1), i32), i32)
        st = Sized((2, 8), i32), Sized((2, 2, 1), i32)
        for a, k in ((dict(slots=Sized((2,), i32), prompt_offsets=off, prompt_tokens=Sized((n,), i32)), "prompt_tokens"),
                     (dict(slots=Sized((2,), i32), output_offsets=off, output_tokens=Sized((n,), i32)), "output_tokens")):
            with pytest.raises(ValueError, match=f"{k}.*2147483647"):
                sv.spec_penalty_reset(*st, **a)
        with pytest.raises(ValueError, match="2147483647"):
            sv.spec_penalty_update(*st, Sized((n,), i32), Sized((2,), i32), off)
    rw = bd._rows_arg(Sized((most, 8), fl), off, "target", Sized((most,), i32), None, i32)
    assert rw.R == most and rw.n_tokens == most


def test_biases_of_one_token_are_added_up_first():
    """z = 1 with biases 2^-24 and 2^-24: 1 + 2^-23 by the definition, 1 if they were added one after the other."""
    rows = ref.Rows("next", np.array([0, 0]), np.zeros(0, np.int64))
    p = dict(bias_offsets=np.array([0, 2]), bias_tokens=np.array([1, 1]), bias_values=f32([2.0 ** -24, 2.0 ** -24]))
    out, _, _ = ref.process(f32([[0, 1, 0, 0]]), rows, p, ref.F32)
    assert out[0, 1] == f32(1 + 2.0 ** -23)
