"""Calls of the logit operators that their documentation allows and that lie at
its edges: padded buffers, streams, empty arguments, long lists."""
from __future__ import annotations

import numpy as np
import pytest

import logits_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to({"fp32": torch.float32, "bf16": torch.bfloat16}[dtype])


def host(t):
    return t.float().cpu().numpy()


def tree(n):
    """One tree of n nodes, each a child of the one before."""
    return ref.Rows("tree", i32([0, n]), np.arange(n) % 8, np.arange(n) - 1)


# ------------------------------------------------------------------ padded buffers
@pytest.mark.parametrize("in_place", [False, True])
def test_buffer_of_many_more_rows_than_sequences(sv, in_place):
    """2^28 + 40 rows of 8 columns for one tree of 64 nodes: how a sequence's rows are split goes by what a
    sequence can own (by the buffer's rows, a part's first row would pass 32 bits)."""
    R, V, n = (1 << 28) + 40, 8, 64
    rng = np.random.default_rng(0)
    rows = tree(n)
    z = ref.to_bf16(rng.standard_normal((n, V)).astype(f32))
    counts = rng.integers(0, 3, (1, V)).astype(i32)
    p = dict(counts=counts, seen=ref.pack(np.stack([rng.random((1, V)) < 0.3, counts > 0], 1)), repetition=f32([1.3]),
             frequency=f32([0.2]), presence=f32([0.1]))
    want, _, _ = ref.process(z, rows, p, ref.BF16)
    x = torch.full((R, V), 2.0, dtype=torch.bfloat16, device="cuda")
    x[:n] = dev(z, "bf16")
    out = x if in_place else torch.full_like(x, 2.0)
    sv.spec_logits_process(x, dev(rows.offsets), dev(rows.tokens.astype(i32)), rows="tree", parent=dev(rows.parent.astype(i32)), out=out,
                           **{k: dev(v) for k, v in p.items()})
    assert np.array_equal(host(out[:n]), want)
    assert bool((out[n:] == 2.0).all())


@pytest.mark.parametrize("mode", ["target", "draft", "next", "tree"])
@pytest.mark.parametrize("in_place", [False, True])
def test_padded_buffers(sv, mode, in_place):
    """Buffers of ten times the rows, as a captured graph keeps them."""
    rng = np.random.default_rng(len(mode))
    V, ks = 4104, np.array([3, 0, 5, 32])
    per = ks + (mode == "tree")
    off = np.concatenate([[0], np.cumsum(per)]).astype(i32)
    tokens = rng.integers(0, V, off[-1]).astype(i32)
    parent = np.concatenate([[-1] + [off[b] + rng.integers(0, g) for g in range(1, m)] for b, m in enumerate(per)]).astype(i32) if mode == "tree" else None
    rows = ref.Rows(mode, off, tokens, parent)
    n = rows.count()
    z = ref.to_bf16(rng.standard_normal((10 * n, V)).astype(f32))
    counts = np.where(rng.random((4, V)) < 0.2, rng.integers(1, 4, (4, V)), 0).astype(i32)
    p = dict(counts=counts, seen=ref.pack(np.stack([rng.random((4, V)) < 0.1, counts > 0], 1)), repetition=f32([1.3, 1, 2, 0.8]))
    want, _, _ = ref.process(z, rows, p, ref.BF16)
    x = dev(z, "bf16")
    out = x if in_place else x.clone()
    sv.spec_logits_process(x, dev(off), dev(tokens), rows=mode, parent=None if parent is None else dev(parent), out=out,
                           **{k: dev(v) for k, v in p.items()})
    assert np.array_equal(host(out), np.concatenate([want[:n], z[n:]]))


# ----------------------------------------------------------------- empty arguments
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pool_without_masks(sv, dtype, in_place):
    """No grammar is in use: M = 0 and every row names none.  A row that names one is NaN."""
    rng = np.random.default_rng(2)
    V, off = 264, i32([0, 2, 3])
    z = rng.standard_normal((5, V)).astype(f32)
    z = ref.to_bf16(z) if dtype == "bf16" else z
    pool = torch.zeros((0, (V + 31) // 32), dtype=torch.int32, device="cuda")
    bias = dict(bias_offsets=dev(i32([0, 0, 1])), bias_tokens=dev(i32([7])), bias_values=dev(f32([2.0])))
    want = z.copy()
    want[3:, 7] += 2
    want = ref.to_bf16(want) if dtype == "bf16" else want
    for names in ([-1] * 5, [-1, 0, -1, -1, -1]):
        x = dev(z, dtype)
        y = host(sv.spec_logits_process(x, dev(off), dev(i32([1, 2, 3])), mask=pool, mask_rows=dev(i32(names)), out=x if in_place else None, **bias))
        none = np.array(names) == -1
        assert np.array_equal(y[none], want[none]) and np.isnan(y[~none]).all()


def test_empty_lists(sv):
    """Lists without entries are as no lists: biases, drafted tokens, prompts."""
    V = 1032
    x = torch.randn(2, V, device="cuda")
    off, none, zero = dev(i32([0, 0, 0])), torch.zeros(0, dtype=torch.int32, device="cuda"), dev(i32([0, 0, 0]))
    st = sv.PenaltyState(2, V)
    st.reset(dev(i32([0, 1])), zero, none, zero, none)
    assert not st.counts.any() and not st.seen.any()
    y = sv.spec_logits_process(x, off, none, counts=st.counts, seen=st.seen, bias_offsets=zero, bias_tokens=none,
                               bias_values=torch.zeros(0, device="cuda"))
    assert torch.equal(x, y)


# ---------------------------------------------------------------- the longest lists
def test_lists_that_end_at_31_bits(sv):
    """Lists of 2^31 - 1 entries, of which the last few hundred are a sequence's: no index passes 31 bits."""
    n, V = (1 << 31) - 1, 4104
    rng = np.random.default_rng(5)
    tail = rng.integers(0, V, 700).astype(i32)
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    tokens[-700:] = dev(tail)
    st = sv.PenaltyState(2, V)
    off = dev(np.array([n - 700, n], i32))
    st.reset(dev(i32([1])), off, tokens, off, tokens)
    counts = np.bincount(tail, minlength=V).astype(i32)
    assert np.array_equal(st.counts.cpu().numpy(), np.stack([np.zeros(V, i32), counts]))
    words = ref.pack(np.stack([counts > 0, counts > 0]))
    assert np.array_equal(st.seen.cpu().numpy()[1], words) and not st.seen[0].any()
    values = torch.zeros(n, device="cuda")
    v = rng.choice(f32([1, -2, 0.25]), 700)
    values[-700:] = dev(v)
    z = rng.standard_normal((1, V)).astype(f32)
    want, _, _ = ref.process(z, ref.Rows("next", i32([0, 0]), np.zeros(0, i32)),
                             dict(bias_offsets=i32([0, 700]), bias_tokens=tail, bias_values=v), ref.F32)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = dev(z)
    for out in (None, x):
        y = sv.spec_logits_process(x, dev(i32([0, 0])), none, rows="next", bias_offsets=off, bias_tokens=tokens, bias_values=values, out=out)
        assert np.array_equal(host(y), want)


# ---------------------------------------------------------------------- long lists
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,V", [("bf16", 4104), ("fp32", 32000), ("bf16", 128256)])
@pytest.mark.parametrize("what", ["every", "one", "twice", "blocks"])
def test_long_bias_lists(sv, what, dtype, V, in_place):
    """A bias on every token, thousands for one token, tokens named twice anywhere in the list: the entries of a
    token are added up in list order, bit for bit."""
    rng = np.random.default_rng(V + len(what))
    if what == "every":
        lists = [rng.permutation(V), np.arange(V)[::-1]]
    elif what == "one":
        lists = [np.full(5000, V - 1), np.repeat([3, 70, 3], [40, 33, 2000])]
    elif what == "twice":
        lists = [np.concatenate([rng.permutation(V)[:3000]] * 2), np.tile(np.arange(0, V, 100), 3)]
    else:  # columns of one word and of neighbouring ones, more than are listed at a time
        lists = [np.arange(min(V, 4096)), np.concatenate([np.arange(600, 1500), np.arange(700, 720), np.arange(640, 672)])]
    n = np.array([len(t) for t in lists])
    tokens = np.concatenate(lists).astype(i32)
    values = (rng.standard_normal(len(tokens)) * rng.choice([1e-3, 1, 30], len(tokens))).astype(f32)
    values[rng.random(len(tokens)) < 0.02] = -0.0
    counts = np.where(rng.random((2, V)) < 0.01, 2, 0).astype(i32)
    p = dict(counts=counts, seen=ref.pack(np.stack([rng.random((2, V)) < 0.01, counts > 0], 1)), frequency=f32([0.5, 0.1]),
             bias_offsets=np.concatenate([[0], np.cumsum(n)]).astype(i32), bias_tokens=tokens, bias_values=values)
    off = i32([0, 1, 1])
    rows = ref.Rows("target", off, i32([5]))
    z = rng.standard_normal((3, V)).astype(f32)
    z[:, ::97] = -0.0
    z = ref.to_bf16(z) if dtype == "bf16" else z
    want, _, _ = ref.process(z, rows, p, dtype)
    x = dev(z, dtype)
    got = host(sv.spec_logits_process(x, dev(off), dev(i32([5])), out=x if in_place else None, **{k: dev(v) for k, v in p.items()}))
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


# ----------------------------------------------------------------- many sequences
@pytest.mark.parametrize("B", [2047, 2048, 4096])
@pytest.mark.parametrize("dtype,V", [("bf16", 9000), ("fp32", 4100)])
def test_rows_of_few_and_of_many_sequences(sv, dtype, V, B):
    """The layouts for up to 2047 sequences and for more of them give the definition's rows."""
    rng = np.random.default_rng(B)
    ks = rng.integers(0, 3, B)
    off = np.concatenate([[0], np.cumsum(ks)]).astype(i32)
    tokens = rng.integers(0, V, off[-1]).astype(i32)
    R = int(off[-1]) + B
    z = rng.standard_normal((40, V)).astype(f32)
    z = (ref.to_bf16(z) if dtype == "bf16" else z)[rng.integers(0, 40, R)]
    counts = np.where(rng.random((5, V)) < 0.1, 3, 0).astype(i32)
    counts[:, :100] = 1
    n = rng.integers(0, 5, B)
    e = np.concatenate([[0], np.cumsum(n)]).astype(i32)
    p = dict(counts=counts, seen=ref.pack(np.stack([rng.random((5, V)) < 0.1, counts > 0], 1)), slots=rng.integers(0, 5, B).astype(i32),
             repetition=rng.choice(f32([1, 1.3]), B), frequency=rng.choice(f32([0, 0.4]), B), presence=rng.choice(f32([0, 0.2]), B),
             bias_offsets=e, bias_tokens=rng.integers(0, V, e[-1]).astype(i32), bias_values=rng.standard_normal(e[-1]).astype(f32),
             mask=ref.pack(rng.random((6, V)) < 0.6), mask_rows=rng.integers(-1, 6, R).astype(i32))
    got = host(sv.spec_logits_process(dev(z, dtype), dev(off), dev(tokens), **{k: dev(v) for k, v in p.items()}))
    for b in np.concatenate([[0, 1, B - 2, B - 1], rng.choice(B, 12, replace=False)]):
        rows = slice(off[b] + b, off[b + 1] + b + 1)
        q = {k: v for k, v in p.items() if k in ("counts", "seen", "mask")}
        q.update({k: p[k][b:b + 1] for k in ("slots", "repetition", "frequency", "presence")}, mask_rows=p["mask_rows"][rows],
                 bias_offsets=i32([0, n[b]]), bias_tokens=p["bias_tokens"][e[b]:e[b + 1]], bias_values=p["bias_values"][e[b]:e[b + 1]])
        want, _, _ = ref.process(z[rows], ref.Rows("target", i32([0, ks[b]]), tokens[off[b]:off[b + 1]]), q, dtype)
        assert np.array_equal(got[rows], want), b


# ------------------------------------------------------------------- the smallest rows
@pytest.mark.parametrize("dtype,V", [("fp32", 4), ("bf16", 8)])
def test_smallest_rows(sv, dtype, V):
    """One vector a row: state, processing, truncation."""
    rng = np.random.default_rng(V)
    st = sv.PenaltyState(2, V)
    st.reset(dev(i32([1, 0])), dev(i32([0, 2, 3])), dev(i32([0, V - 1, 1])), dev(i32([0, 0, 2])), dev(i32([2, 2])))
    st.update(dev(i32([3, 3, 1])), dev(i32([1, 0])), dev(i32([0, 1, 1])), slots=dev(i32([1, 0])))
    counts = np.zeros((2, V), i32)
    counts[0, 2], counts[1, 3], counts[0, 1] = 2, 2, 1
    assert np.array_equal(st.counts.cpu().numpy(), counts)
    off, tokens = i32([0, 2, 2]), i32([0, V - 1])
    rows = ref.Rows("target", off, tokens)
    z = rng.standard_normal((4, V)).astype(f32)
    z = ref.to_bf16(z) if dtype == "bf16" else z
    p = dict(counts=counts, seen=st.seen.cpu().numpy(), repetition=f32([1.5, 0.5]), frequency=f32([0.25, 0]), presence=f32([0, 1]),
             mask=ref.pack(rng.random((4, V)) < 0.8))
    want, _, _ = ref.process(z, rows, p, dtype)
    T, s = f32([1, 0.5]), dict(top_k=i32([3, V - 1]), top_p=f32([0.8, 0.6]), min_p=f32([0, 0.01]))
    cut, margin = ref.truncate(want, ref.row_sequences(rows), T, **s)
    assert margin.min() > 1e-6
    got = sv.spec_logits_process_truncate(dev(z, dtype), dev(T), dev(off), dev(tokens), **{k: dev(v) for k, v in {**p, **s}.items()})
    assert np.array_equal(host(got), cut)


# --------------------------------------------------------------------- captured calls
CAPTURED = {"cluster": ("bf16", 128256, 2, False), "cluster in place": ("bf16", 128256, 2, True), "rows": ("bf16", 32000, 200, False),
            "held": ("fp32", 32000, 3, False), "fp32": ("fp32", 128256, 3, True), "small": ("fp32", 4100, 40, True)}


@pytest.mark.parametrize("name", sorted(CAPTURED))
def test_captured_calls(sv, name):
    """Processing and truncation of every kind of row, captured beside another graph of the same buffers, replayed
    in turn with it on inputs that change."""
    dtype, V, B, in_place = CAPTURED[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    tokens = torch.randint(V, (B,), generator=g, device="cuda").int()
    T = torch.full((B,), 0.8, device="cuda")
    st = sv.PenaltyState(B, V)
    n = 50
    a = dict(counts=st.counts, seen=st.seen, frequency=torch.full((B,), 0.3, device="cuda"), bias_offsets=off * n,
             bias_tokens=torch.randint(V, (B * n,), generator=g, device="cuda").int(),
             bias_values=torch.randn(B * n, generator=g, device="cuda"))
    t = dict(top_k=torch.randint(1, 200, (B,), generator=g, device="cuda").int(), top_p=torch.full((B,), 0.95, device="cuda"))
    kind = torch.float32 if dtype == "fp32" else torch.bfloat16
    x = torch.zeros(2 * B, V, dtype=kind, device="cuda")
    out = x if in_place else torch.empty_like(x)
    emitted, accepted = torch.randint(V, (2 * B,), generator=g, device="cuda").int(), torch.ones(B, dtype=torch.int32, device="cuda")

    def both():
        return sv.spec_logits_process_truncate(x, T, off, tokens, out=out, **a, **t)

    def update():
        st.update(emitted, accepted, off)

    both(), update()
    st.reset(torch.arange(B, dtype=torch.int32, device="cuda"))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, call in zip(graphs, (both, update)):
        with torch.cuda.graph(graph):
            call()
    for i in range(3):
        z = (torch.randn(2 * B, V, generator=g, device="cuda") * 3).to(kind)
        tokens.copy_(torch.randint(V, (B,), generator=g, device="cuda"))
        emitted.copy_(torch.randint(V, (2 * B,), generator=g, device="cuda"))
        want = sv.spec_logits_truncate(sv.spec_logits_process(z, off, tokens, **a), T, off, **t)
        x.copy_(z)
        graphs[0].replay()
        assert torch.equal(out, want)
        graphs[1].replay()
        assert int(st.counts.sum()) == 2 * B * (i + 1)
