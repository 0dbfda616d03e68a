"""GPU: the 8-bit cache.  An element is rounded once and scales are powers of two, so what is held and what is
read back in fp32 is compared exactly; read back in bf16 it is the fp32 value rounded (exact but for the smallest)."""
from __future__ import annotations

import numpy as np
import pytest

import states_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same(a, b):
    return ((a == b) | (np.isnan(a) & np.isnan(b))).all()


class Case:
    """A cache of some contents on the device, and its restatements for keys and values."""

    def __init__(self, L, S, T, H, D, rng, paged=0, values=True, held=0):
        self.L, self.S, self.T, self.H, self.D, self.rng = L, S, T, H, D, rng
        P = S if not paged else S * paged + 3
        self.pages = rng.permutation(P)[: S * paged].reshape(S, paged).astype(i32) if paged else None
        self.lengths = rng.integers(0, held + 1, S).astype(i32)
        blocks = -(-D // 32)
        self.refs, self.tensors = [], []
        for _ in range(2 if values else 1):
            byte = rng.integers(0, 127, (L, P, T, H, D)).astype(np.uint8) + 128 * rng.integers(0, 2, (L, P, T, H, D)).astype(np.uint8)
            scale = rng.integers(100, 140, (L, P, T, H, blocks)).astype(np.uint8)
            t = dev(byte).view(torch.float8_e4m3fn)
            self.tensors += [t, dev(scale)]
            self.refs.append(ref.Cache(t.double().cpu().numpy(), scale, self.lengths, self.pages))
        if not values:
            self.tensors += [None, None]
        self.d_lengths = dev(self.lengths)
        self.d_pages = None if self.pages is None else dev(self.pages)

    def inputs(self, R, dtype, spread=6):
        shape = (self.L, R, self.H, self.D)
        x = self.rng.standard_normal(shape) * 2.0 ** self.rng.integers(-spread, spread + 1, (*shape[:-1], 1))
        x[self.rng.random(shape) < 0.02] = 0
        t = dev(x.astype(f32)).to(TYPES[dtype])
        return t, t.float().cpu().numpy()

    def check(self, out_lengths=None):
        for i, r in enumerate(self.refs):
            assert same(self.tensors[2 * i].double().cpu().numpy(), r.q)
            assert (self.tensors[2 * i + 1].cpu().numpy() == r.scale).all()
        if out_lengths is not None:
            assert (out_lengths.cpu().numpy() == self.refs[0].after).all()

    def write(self, sv, inputs, paths, slots, offsets=None, out="new", **kw):
        for r, (_, x) in zip(self.refs, inputs):
            r.write(x, paths, slots)
        to = {"new": torch.full_like(self.d_lengths, -77), "in place": self.d_lengths, "none": None}[out]
        sv.spec_cache_write(*self.tensors, self.d_lengths, inputs[0][0], inputs[1][0] if len(inputs) > 1 else None, None if offsets is None else dev(np.asarray(offsets, i32)),
                            slots=dev(np.asarray(slots, i32)), pages=self.d_pages, out_lengths=to, **kw)
        self.check(to)
        if out != "in place":
            assert (self.d_lengths.cpu().numpy() == self.lengths).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L,H,D", [(1, 1, 16), (2, 3, 32), (1, 5, 48), (3, 2, 64), (2, 5, 80), (1, 8, 128), (2, 1, 576), (1, 3, 1008)])
@pytest.mark.parametrize("paged", [0, 6])
def test_a_verifys_rows(sv, dtype, L, H, D, paged):
    rng = np.random.default_rng(D + L)
    k = np.array([4, 0, 3, 10, 1, 7])
    B = len(k)
    c = Case(L, B + 2, 40 if not paged else 7, H, D, rng, paged, held=20)
    off = np.concatenate([[0], np.cumsum(k)])
    n = np.array([4, 0, 1, 6, -1, 8])  # all, none, some, an error, more than there are
    slots = rng.permutation(B + 2)[:B]
    x = [c.inputs(off[-1] + B, dtype) for _ in range(2)]
    paths = [list(range(off[b] + b, off[b] + b + n[b] + 1)) if 0 <= n[b] <= k[b] else None for b in range(B)]
    for out in ("new", "none", "in place"):
        c.write(sv, x, paths, slots, off, out, rows="target", num_accepted=dev(n.astype(i32)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("values", [True, False])
def test_a_trees_path(sv, dtype, values):
    rng = np.random.default_rng(3)
    shapes = [[-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9], [-1], [-1] + list(range(63)), [-1, 0, 0], [-1, 0, 1], [-1, 0, 1], [-1, 0, 1, 2], [-1, 0, 1]]
    last = [11, 0, 63, 2, 2, 1, 3, 5]
    n = np.array([3, 0, 63, 1, 1, -1, 3, 2])  # the fifth is not as deep as its count, the eighth's last node is not its own
    off = np.concatenate([[0], np.cumsum([len(s) for s in shapes])])
    parent = np.concatenate([np.where(np.array(s) < 0, -1, np.array(s) + o) for s, o in zip(shapes, off)]).astype(i32)
    parent[off[6] + 2] = off[6] + 3  # and the seventh's parents do not come before their children
    B = len(shapes)
    c = Case(2, B, 9, 2, 80, rng, 10, values, held=12)
    slots = rng.permutation(B)
    x = [c.inputs(off[-1], dtype) for _ in range(2 if values else 1)]
    paths = [ref.tree_path(parent, off[b], len(shapes[b]), off[b] + last[b], n[b]) for b in range(B)]
    assert [p is None for p in paths] == [False] * 4 + [True] * 4
    c.write(sv, x, paths, slots, off, "new", rows="tree", num_accepted=dev(n.astype(i32)), parent=dev(parent), last_node=dev((off[:-1] + last).astype(i32)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompts_and_single_tokens(sv, dtype):
    rng = np.random.default_rng(4)
    c = Case(2, 5, 16, 2, 64, rng, 20, held=0)
    per = np.array([100, 0, 1, 255])
    off = np.concatenate([[0], np.cumsum(per)])
    slots = rng.permutation(5)[:4]
    x = [c.inputs(off[-1] + 3, dtype) for _ in range(2)]  # rows behind the last sequence's
    paths = [list(range(off[b], off[b + 1])) for b in range(4)]
    c.write(sv, x, paths, slots, off, "in place", rows="prompt")
    for r in c.refs:
        r.lengths = r.after
    x = [c.inputs(4, dtype) for _ in range(2)]
    c.write(sv, x, [[b] for b in range(4)], slots, None, "in place", rows="next")
    for r in c.refs:
        r.lengths = r.after
    # a prompt that goes on where the first part ended
    x = [c.inputs(37, dtype) for _ in range(2)]
    c.write(sv, x, [list(range(37))], slots[:1], [0, 37], "in place", rows="prompt")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_of_every_kind(sv, dtype):
    """Borders between e4m3 values and between scales, zeros, the smallest and largest numbers, infinities and NaN."""
    rng = np.random.default_rng(5)
    c = Case(1, 1, 64, 2, 80, rng)
    c.lengths[:] = 0
    c.d_lengths.zero_()
    x = rng.standard_normal((1, 40, 2, 80)).astype(f32)
    grid = np.unique(ref.to_e4m3(np.linspace(-448, 448, 100000)))
    mid = ((grid[1:] + grid[:-1]) / 2).astype(f32)
    for i in range(4):  # halves between values, under a largest of 448 that makes the scale 1
        x[0, i, :, 1:32] = rng.choice(mid, (2, 31))
        x[0, i, :, 0] = 448
    x[0, 4, :, :32] = 0
    x[0, 5, :, 0], x[0, 6, :, 0] = -0.0, 449
    x[0, 7] = rng.standard_normal((2, 80)) * 1e-38
    x[0, 8] = rng.standard_normal((2, 80)) * 3e37
    x[0, 9] = 2.0 ** -126
    x[0, 10, 0, 3], x[0, 11, 0, 33], x[0, 12, 1, 70], x[0, 13] = np.nan, np.inf, -np.inf, np.nan
    x[0, 14] = np.inf
    x[0, 15, :, ::2], x[0, 16, :, 1::3] = np.inf, np.nan
    x[0, 17] = np.finfo(f32).max if dtype == "fp32" else 3.3895313892515355e38
    if dtype == "fp32":
        x[0, 18] = rng.standard_normal((2, 80)) * 1e-42
        x[0, 19, :, 1] = 448 * (1 + 2.0 ** -23)
    t = dev(x).to(TYPES[dtype])
    x = t.float().cpu().numpy()
    for r in c.refs:
        r.lengths = c.lengths
    c.write(sv, [(t, x), (t, x)], [list(range(40))], [0], [0, 40], "new", rows="prompt")
    c.refs[0].lengths = np.array([40])
    held = c.refs[0].read([0, 40], 40, [0])
    # 255 * 2^120 (the largest bf16 in its block) lies nearer 256 than 240 on e4m3's grid: held is 2^128, past fp32
    assert held[0, 17].max() == 2.0 ** 128
    with np.errstate(over="ignore"):
        held = held.astype(f32).astype(np.float64)
    lengths = torch.tensor([40], dtype=torch.int32, device="cuda")
    keys, values = sv.spec_cache_read(*c.tensors, lengths, dev(np.array([0, 40], i32)), 40, dtype=torch.float32)
    assert same(keys.double().cpu().numpy(), held) and same(values.double().cpu().numpy(), held)
    keys, _ = sv.spec_cache_read(*c.tensors, lengths, dev(np.array([0, 40], i32)), 40)
    want = torch.from_numpy(held).to(torch.float32).to(torch.bfloat16).double().numpy()
    assert keys.dtype == torch.bfloat16 and same(keys.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L,H,D,paged,values", [(1, 1, 16, 0, True), (3, 2, 80, 5, True), (2, 4, 128, 5, True), (2, 1, 576, 3, False), (1, 7, 48, 0, False)])
def test_reading(sv, dtype, L, H, D, paged, values):
    rng = np.random.default_rng(D)
    T = 11 if paged else 40
    c = Case(L, 7, T, H, D, rng, paged, values)
    c.lengths[:] = rng.integers(0, T * max(1, paged), 7)
    c.lengths[2] = -1
    if paged:
        c.pages[1, 1], c.pages[4, 0] = -1, 10 ** 6
    c.d_lengths, c.d_pages = dev(c.lengths), None if not paged else dev(c.pages)
    for r in c.refs:
        r.lengths = c.lengths
    slots = np.array([3, 1, 2, 4, 0, 7, -1, 6, 3])  # two sequences may read one slot
    per = np.array([20, 30, 2, 25, 0, 2, 2, 40, 9])
    off = np.concatenate([[0], np.cumsum(per)])
    first = np.array([0, 5, 0, 3, 0, 0, 0, -2, 1])
    R = off[-1] + 2
    for f in (None, first):
        out = tuple(None if i and not values else torch.full((L, R, H, D), 5.0, dtype=TYPES[dtype], device="cuda") for i in range(2))
        got = sv.spec_cache_read(*c.tensors, c.d_lengths, dev(off.astype(i32)), R, first=None if f is None else dev(f.astype(i32)), slots=dev(slots.astype(i32)),
                                 pages=c.d_pages, out=out)
        for g, r in zip(got, c.refs):
            want = torch.from_numpy(r.read(off, R, slots, f)).to(torch.float32).to(TYPES[dtype]).double().numpy()
            want[:, off[-1]:] = 5.0
            assert same(g.double().cpu().numpy(), want)


def test_no_room_bad_pages_and_slots(sv):
    rng = np.random.default_rng(6)
    B = 8
    c = Case(1, B, 4, 2, 32, rng, 3, held=3)
    c.pages[2, 1], c.pages[3, 2] = -1, c.tensors[0].shape[1]
    c.d_pages = dev(c.pages)
    c.lengths[:] = [3, 10, 3, 3, -1, 12, 0, 2]
    c.d_lengths = dev(c.lengths)
    for r in c.refs:
        r.lengths, r.pages = c.lengths.copy(), c.pages
    per = np.array([9, 4, 2, 9, 3, 1, 12, 13])
    off = np.concatenate([[0], np.cumsum(per)])
    x = [c.inputs(off[-1], "bf16") for _ in range(2)]
    c.write(sv, x, [list(range(off[b], off[b + 1])) for b in range(B)], np.arange(B), off, "new", rows="prompt")
    assert list(c.refs[0].after) == [12, -1, -1, -1, -1, -1, 12, -1]
    slots = np.array([0, B, -1, 6, 2 ** 31 - 1, 5, 1, 7])
    c.write(sv, x, [list(range(off[b], off[b + 1])) for b in range(B)], slots, off, "new", rows="prompt")


@pytest.mark.parametrize("rows,offsets", [("target", [0, 33, 34]), ("target", [1, 2, 3]), ("target", [0, 5, 4]), ("target", [0, 20, 39]), ("tree", [0, 0, 4]),
                                          ("tree", [0, 65, 70]), ("tree", [0, 20, 41]), ("prompt", [0, 5, 4]), ("prompt", [0, 20, 41]), ("prompt", [0, -1, 4]),
                                          ("prompt", [0, 2 ** 31 - 1, 2 ** 31 - 1])])
def test_invalid_offsets(sv, rows, offsets):
    rng = np.random.default_rng(7)
    c = Case(1, 2, 100, 1, 32, rng, held=10)
    x = [c.inputs(40, "bf16") for _ in range(2)]
    zero = dev(np.zeros(2, i32))
    kw = dict(num_accepted=zero) if rows != "prompt" else {}
    if rows == "tree":
        kw |= dict(parent=dev(np.full(40, -1, i32)), last_node=zero)
    c.write(sv, x, [None, None], [0, 1], offsets, "new", rows=rows, **kw)
    if rows == "prompt":
        out = torch.full((1, 40, 1, 32), 5.0, device="cuda"), torch.full((1, 40, 1, 32), 5.0, device="cuda")
        sv.spec_cache_read(*c.tensors, c.d_lengths, dev(np.array(offsets, i32)), 40, out=out)
        assert (out[0] == 5).all() and (out[1] == 5).all()


def test_strided_inputs(sv):
    """Keys and values as parts of a joint projection's output, and of a longer buffer."""
    rng = np.random.default_rng(8)
    c = Case(3, 2, 40, 2, 64, rng)
    qkv = dev(rng.standard_normal((3, 24, 8, 64)).astype(f32)).to(torch.bfloat16)
    k, v = qkv[:, 2:22, 4:6], qkv[:, 2:22, 6:8]
    c.write(sv, [(k, k.float().cpu().numpy()), (v, v.float().cpu().numpy())], [list(range(12)), list(range(12, 20))], [1, 0], [0, 12, 20], "new", rows="prompt")
    # one layer at a time, the lengths with the last
    c = Case(3, 2, 40, 2, 64, rng)
    for layer in range(3):
        sv.spec_cache_write(*(t[layer:layer + 1] for t in c.tensors), c.d_lengths, k[layer], v[layer], dev(np.array([0, 12, 20], i32)), rows="prompt",
                            out_lengths=c.d_lengths if layer == 2 else None)
    for r, x in zip(c.refs, (k, v)):
        r.write(x.float().cpu().numpy(), [list(range(12)), list(range(12, 20))], [0, 1])
    c.check(c.d_lengths)


def test_positions_past_32_bits(sv):
    """A pool of more than 2^32 elements: rows written and read near its end."""
    L, P, T, H, D = 1, 3, 1 << 20, 8, 192
    k = torch.zeros((L, P, T, H, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.zeros((L, P, T, H, 6), dtype=torch.uint8, device="cuda")
    lengths = dev(np.array([T - 3, 5, T - 2], i32))
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((1, 5, H, D), generator=g, device="cuda")
    sv.spec_cache_write(k, scale, None, None, lengths, x, None, dev(np.array([0, 3, 5], i32)), rows="prompt", slots=dev(np.array([0, 2], i32)), out_lengths=lengths)
    assert lengths.tolist() == [T, 5, T]
    got, none = sv.spec_cache_read(k, scale, None, None, lengths, dev(np.array([0, 3, 5], i32)), 5, first=dev(np.array([T - 3, T - 2], i32)),
                                   slots=dev(np.array([0, 2], i32)), dtype=torch.float32)
    want = ref.dequantise(*ref.quantise(x.cpu().numpy()))
    assert none is None and (got.double().cpu().numpy() == want).all()
    assert int(scale.count_nonzero()) == 5 * H * 6


def test_state_object_streams_and_capture(sv):
    """CacheState: written on another stream, reordered, read; a captured step replayed."""
    rng = np.random.default_rng(9)
    st = sv.CacheState(2, 4, 32, 2, 64)
    k, v = (dev(rng.standard_normal((2, 12, 2, 64)).astype(f32)).to(torch.bfloat16) for _ in range(2))
    off = dev(np.array([0, 3, 6, 9, 12], i32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.write(k, v, off, rows="prompt", stream=side)
    got = st.read(off, 12, stream=side, dtype=torch.float32)
    side.synchronize()
    want = [ref.dequantise(*ref.quantise(t.float().cpu().numpy())) for t in (k, v)]
    assert all((g.double().cpu().numpy() == w).all() for g, w in zip(got, want)) and st.lengths.tolist() == [3] * 4
    st.reorder(dev(np.array([1, 0, 0, 3], i32)), dev(np.array([0, 4], i32)))
    got = st.read(off, 12, dtype=torch.float32)
    order = np.concatenate([np.arange(3) + 3 * s for s in (1, 0, 0, 3)])
    assert all((g.double().cpu().numpy() == w[:, order]).all() for g, w in zip(got, want))
    torch.cuda.synchronize()
    slots = dev(np.arange(4).astype(i32))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.write(k[:, :4], v[:, :4], rows="next", slots=slots)
    for i in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert st.lengths.tolist() == [6] * 4
    got = st.read(dev(np.array([0, 3, 6, 9, 12], i32)), 12, first=dev(np.full(4, 3, i32)), dtype=torch.float32)
    rows = np.repeat(np.arange(4), 3)
    assert all((x.double().cpu().numpy() == w[:, rows]).all() for x, w in zip(got, want))


def test_binding_refusals(sv):
    st = sv.CacheState(2, 4, 32, 2, 64)
    k = torch.zeros((2, 4, 2, 64), device="cuda")
    off = dev(np.array([0, 4], i32))
    for bad, match in ((dict(rows="draft"), "rows must be"), (dict(rows="target"), "num_accepted"), (dict(rows="next"), "slots"),
                       (dict(rows="prompt", num_accepted=dev(np.zeros(1, i32))), "num_accepted")):
        with pytest.raises(ValueError, match=match):
            st.write(k, k, off, **bad)
    with pytest.raises(ValueError, match="values and v"):
        st.write(k, None, off, rows="prompt")
    with pytest.raises(ValueError, match="keys must be"):
        st.write(k[:1], k[:1], off, rows="prompt")
    with pytest.raises(ValueError, match="one type"):
        st.write(k, k.bfloat16(), off, rows="prompt")
    with pytest.raises(ValueError, match="contiguous in heads"):
        x = torch.zeros((2, 4, 64, 2), device="cuda").transpose(2, 3)
        st.write(x, x, off, rows="prompt")
    with pytest.raises(TypeError):
        st.write(k.half(), k.half(), off, rows="prompt")
    with pytest.raises(ValueError, match="fewer rows"):
        st.write(k, k, rows="next", slots=dev(np.zeros(5, i32)))
    with pytest.raises(sv.SpecError, match="ALIGN"):
        x = torch.zeros(2 * 4 * 128 + 4, device="cuda")[4:].view(2, 4, 2, 64)
        st.write(x, x, off, rows="prompt")
    with pytest.raises(ValueError, match="out must be"):
        st.read(off, 4, out=(k, None))
