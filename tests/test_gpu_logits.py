"""Logit operators on the GPU against their plain restatements (logits_ref):
processing bit for bit with the definition's fp32 steps and within those
steps' bound of 64 bits, truncation against a full sort in 64 bits (rows whose
top-p border lies within 1e-10 of Z of another answer may differ there), the
counts exactly."""
from __future__ import annotations

import numpy as np
import pytest

import logits_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
LOWEST = {"fp32": np.finfo(f32).min, "bf16": f32(-3.3895313892515355e38)}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()  # raises if the library is missing: no fallback
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to({"fp32": torch.float32, "bf16": torch.bfloat16}[dtype])


def host(t):
    return t.float().cpu().numpy()


def same_bits(a, b):
    """Equal values, NaN where NaN, and -0 apart from +0."""
    return ((a == b) | (np.isnan(a) & np.isnan(b))) & ((np.signbit(a) == np.signbit(b)) | np.isnan(a))


# ------------------------------------------------------------------ processing
def make_rows(rng, mode, ks, V):
    per = np.asarray(ks) + (1 if mode == "tree" else 0)
    off = np.concatenate([[0], np.cumsum(per)]).astype(i32)
    tokens = (rng.random(off[-1]) ** 3 * V).astype(i32)
    parent = None
    if mode == "tree":
        parent = np.concatenate([[-1] + [off[b] + rng.integers(0, g) for g in range(1, n)] for b, n in enumerate(per)]).astype(i32)
        tokens[off[:-1]] = -77  # a root's token is not read
    return ref.Rows(mode, off, tokens, parent)


def make_logits(rng, R, V, dtype, special=True):
    z = (rng.standard_normal((R, V)) * 4 - 3).astype(f32)
    if special:
        odd = f32([np.inf, -np.inf, np.nan, 0.0, -0.0, LOWEST[dtype], 1e-40])
        at = rng.random((R, V)) < 0.05
        z[at] = odd[rng.integers(0, len(odd), int(at.sum()))]
    return ref.to_bf16(z) if dtype == "bf16" else z


def make_params(rng, rows, R, V, pen=True, bias=True, mask=True, S=None):
    B, p = rows.B, {}
    if pen:
        S = S or B + 3
        counts = np.where(rng.random((S, V)) < 0.1, rng.integers(1, 9, (S, V)), 0).astype(i32)
        counts[0, 0] = 1 << 30  # a count past fp32's whole numbers
        p.update(counts=counts, slots=rng.permutation(S)[np.arange(B) % S].astype(i32),
                 seen=ref.pack(np.stack([rng.random((S, V)) < 0.1, counts > 0], 1)),
                 repetition=rng.choice(f32([1, 1.1, 0.7, 2.5]), B), frequency=rng.choice(f32([0, 0.3, -1.5]), B),
                 presence=rng.choice(f32([0, 0.4, -0.8]), B))
    if bias:
        n = rng.integers(0, 9, B)
        n[rng.integers(0, B)] = 300  # more than one block reads at once
        p["bias_offsets"] = np.concatenate([[0], np.cumsum(n)]).astype(i32)
        p["bias_tokens"] = rng.integers(0, V, n.sum()).astype(i32)
        p["bias_values"] = rng.choice(f32([-100, -0.3, 1.7, 5, -np.inf]), n.sum())
    if mask:
        M = max(1, R // 2)
        p["mask"] = ref.pack(rng.random((M, V)) < rng.choice([0.0, 0.01, 0.5, 1.0], (M, 1)))
        p["mask_rows"] = rng.integers(-1, M, R).astype(i32)
    return p


def process(sv, z, rows, p, dtype, **kw):
    return sv.spec_logits_process(dev(z, dtype), dev(rows.offsets), dev(rows.tokens), rows=rows.mode,
                                  parent=None if rows.parent is None else dev(rows.parent),
                                  **{k: dev(v) for k, v in p.items()}, **kw)


KS = {"ragged": [3, 0, 7, 1, 0, 0, 32, 5], "one": [0], "none": [0, 0, 0], "five": [5, 5, 5], "only": [0, 0, 0, 2, 0]}


@pytest.mark.parametrize("V", [8, 24, 264, 1000, 1032, 4104, 32000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode,ks", [("target", "ragged"), ("target", "one"), ("target", "none"), ("draft", "ragged"),
                                     ("draft", "only"), ("next", "ragged"), ("tree", "ragged"), ("tree", "five")])
def test_process(sv, mode, ks, dtype, V):
    rng = np.random.default_rng(V + len(mode) + len(ks))
    rows = make_rows(rng, mode, KS[ks], V)
    z = make_logits(rng, rows.count(), V, dtype)
    p = make_params(rng, rows, len(z), V)
    want, want64, tol = ref.process(z, rows, p, dtype)
    got = host(process(sv, z, rows, p, dtype))
    assert same_bits(got, want).all()
    finite = np.isfinite(want64) & np.isfinite(want)  # past the type's largest value it rounds to inf
    assert (abs(got[finite] - want64[finite]) <= tol[finite]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want64))


@pytest.mark.parametrize("which", ["pen", "bias", "mask", "nothing"])
@pytest.mark.parametrize("dtype,V", [("bf16", 1032), ("fp32", 516)])
def test_process_parts(sv, which, dtype, V):
    """Each part by itself, the optional arrays left out (slots, the three factors, mask_rows)."""
    rng = np.random.default_rng(11)
    rows = make_rows(rng, "target", KS["ragged"], V)
    z = make_logits(rng, rows.count(), V, dtype)
    p = make_params(rng, rows, len(z), V, which == "pen", which == "bias", which == "mask", S=rows.B)
    if which == "pen":
        del p["slots"], p["repetition"], p["presence"]
    if which == "mask":
        p = {"mask": ref.pack(rng.random((len(z) + 2, V)) < 0.3)}
    want, _, _ = ref.process(z, rows, p, dtype)
    assert same_bits(host(process(sv, z, rows, p, dtype)), want).all()


@pytest.mark.parametrize("dtype,V", [("bf16", 4104), ("fp32", 1004)])
def test_process_in_place_and_padded(sv, dtype, V):
    """In place, and rows behind the last sequence's left as they were."""
    rng = np.random.default_rng(12)
    rows = make_rows(rng, "target", KS["ragged"], V)
    R = rows.count()
    z = make_logits(rng, R + 3, V, dtype)
    p = make_params(rng, rows, R + 3, V)
    want, _, _ = ref.process(z, rows, p, dtype)
    x = dev(z, dtype)
    args = dict(rows="target", **{k: dev(v) for k, v in p.items()})
    y = sv.spec_logits_process(x, dev(rows.offsets), dev(rows.tokens), out=x, **args)
    assert y is x and same_bits(host(x), want).all()
    out = torch.full_like(x, 7.0)
    sv.spec_logits_process(dev(z, dtype), dev(rows.offsets), dev(rows.tokens), out=out, **args)
    assert same_bits(host(out)[:R], want[:R]).all() and (host(out)[R:] == 7).all()


@pytest.mark.parametrize("mode", ["target", "next", "tree"])
@pytest.mark.parametrize("dtype,V", [("bf16", 264), ("bf16", 32000), ("fp32", 9004)])
def test_process_in_place_without_masks(sv, mode, dtype, V):
    """In place and without masks only the touched columns are visited (another kernel); frequent ids are the lowest."""
    rng = np.random.default_rng(15)
    rows = make_rows(rng, mode, KS["ragged"], V)
    z = make_logits(rng, rows.count(), V, dtype)
    p = make_params(rng, rows, len(z), V, mask=False)
    p["counts"][:, :200] = 3  # dense words
    p["seen"][:, 1] = ref.pack(p["counts"] > 0)
    want, _, _ = ref.process(z, rows, p, dtype)
    x = dev(z, dtype)
    sv.spec_logits_process(x, dev(rows.offsets), dev(rows.tokens), rows=mode, parent=None if rows.parent is None else dev(rows.parent),
                           out=x, **{k: dev(v) for k, v in p.items()})
    assert same_bits(host(x), want).all()
    bad = host(process(sv, z, rows, {**p, "repetition": np.where(np.arange(rows.B) == 2, f32(-1), p["repetition"])}, dtype, out=dev(z, dtype)))
    seq = ref.row_sequences(rows)
    assert np.isnan(bad[seq == 2]).all() and same_bits(bad[seq != 2], want[seq != 2]).all()


def test_process_spread_and_whole_units(sv):
    """The layouts for small calls and for large ones (over 300 MB) give the same rows."""
    rng = np.random.default_rng(16)
    V, B = 64008, 700
    rows = make_rows(rng, "target", [3] * B, V)
    z = make_logits(rng, 64, V, "bf16")
    z = z[rng.integers(0, 64, rows.count())]
    p = make_params(rng, rows, len(z), V, S=5, mask=False)
    p["mask"] = ref.pack(rng.random((7, V)) < 0.5)
    p["mask_rows"] = rng.integers(-1, 7, len(z)).astype(i32)
    got = host(process(sv, z, rows, p, "bf16"))
    at = rng.choice(B, 6, replace=False)
    for b in at:
        one = ref.Rows("target", i32([0, 3]), rows.tokens[3 * b:3 * b + 3])
        sl = slice(4 * b, 4 * b + 4)
        e = p["bias_offsets"]
        q = {k: v for k, v in p.items() if k in ("counts", "seen", "mask")}
        q.update({k: p[k][b:b + 1] for k in ("slots", "repetition", "frequency", "presence")}, mask_rows=p["mask_rows"][sl],
                 bias_offsets=i32([0, e[b + 1] - e[b]]), bias_tokens=p["bias_tokens"][e[b]:e[b + 1]], bias_values=p["bias_values"][e[b]:e[b + 1]])
        assert same_bits(got[sl], ref.process(z[sl], one, q, "bf16")[0]).all()


def broken(name, rows, p, V):
    """Makes one sequence (its number is returned) or one row (as ~row) invalid."""
    o = rows.offsets
    if name in ("repetition", "frequency", "presence"):
        p[name][2] = {"repetition": 0, "frequency": np.nan, "presence": np.inf}[name]
        return 2
    if name == "slot":
        p["slots"][3] = len(p["counts"])
        return 3
    if name == "slot_negative":
        p["slots"][3] = -1
        return 3
    if name == "token":
        rows.tokens[o[2] + 1] = V
        return 2
    if name == "token_negative":
        rows.tokens[o[2] + 2] = -1
        return 2
    if name == "parent":
        rows.parent[o[2] + 1] = o[2] + 1
        return 2
    if name == "parent_other":
        rows.parent[o[2] + 1] = o[2] - 1
        return 2
    if name == "root":
        rows.parent[o[2]] = 0
        return 2
    e = p["bias_offsets"]
    b = int(np.argmax(np.diff(e)))
    if name == "bias_token":
        p["bias_tokens"][e[b] + 200] = V
        return b
    if name == "bias_nan":
        p["bias_values"][e[b]] = np.nan
        return b
    if name == "bias_inf":
        p["bias_values"][e[b + 1] - 1] = np.inf
        return b
    if name == "mask_row":
        p["mask_rows"][5] = len(p["mask"])
        return ~5
    p["mask_rows"][4] = -2
    return ~4


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence", "slot", "slot_negative", "token", "token_negative",
                                  "parent", "parent_other", "root", "bias_token", "bias_nan", "bias_inf", "mask_row", "mask_row_low"])
def test_process_data_errors(sv, name):
    """An invalid sequence has NaN rows, an invalid mask row a NaN row; the others are as ever."""
    rng = np.random.default_rng(13)
    mode = "tree" if name in ("parent", "parent_other", "root") else "target"
    rows = make_rows(rng, mode, [3, 2, 7, 1, 4], 2056)
    z = make_logits(rng, rows.count(), 2056, "bf16", special=False)
    p = make_params(rng, rows, len(z), 2056)
    want, _, _ = ref.process(z, rows, p, "bf16")
    seq = ref.row_sequences(rows)
    bad = broken(name, rows, p, 2056)
    got = host(process(sv, z, rows, p, "bf16"))
    hit = np.arange(len(z)) == ~bad if bad < 0 else seq == bad
    assert hit.any() and np.isnan(got[hit]).all()
    assert same_bits(got[~hit], want[~hit]).all()


OFFSETS = {"start": [1, 2, 4], "falls": [0, 3, 2], "long": [0, 33, 34], "rows": [0, 2, 9], "negative": [0, -1, 4]}


@pytest.mark.parametrize("name", sorted(OFFSETS))
@pytest.mark.parametrize("op", ["process", "truncate", "process_truncate"])
def test_invalid_offsets_fail_the_call(sv, name, op):
    x = torch.randn(40 if name == "long" else 6, 1032, device="cuda")
    off, tok, T = dev(i32(OFFSETS[name])), torch.zeros(64, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
    if op == "process":
        y = sv.spec_logits_process(x, off, tok)
    elif op == "truncate":
        y = sv.spec_logits_truncate(x, T, off, top_k=torch.full((2,), 3, dtype=torch.int32, device="cuda"))
    else:
        y = sv.spec_logits_process_truncate(x, T, off, tok, top_k=torch.full((2,), 3, dtype=torch.int32, device="cuda"))
    assert torch.isnan(y).all()


def test_too_few_tokens_fail_the_call(sv):
    """Penalties whose offsets ask for more drafted tokens than were given."""
    x = torch.randn(8, 1032, device="cuda")
    st = sv.PenaltyState(2, 1032)
    y = sv.spec_logits_process(x, dev(i32([0, 3, 6])), torch.zeros(5, dtype=torch.int32, device="cuda"), counts=st.counts, seen=st.seen)
    assert torch.isnan(y).all()


@pytest.mark.parametrize("V", [264, 2056])
def test_process_many_sequences(sv, V):
    """MAX_B sequences, long runs of them without rows."""
    rng = np.random.default_rng(14)
    ks = np.where(rng.random(sv.MAX_B) < 0.02, rng.integers(1, 33, sv.MAX_B), 0)
    rows = make_rows(rng, "draft", ks, V)
    z = make_logits(rng, rows.count(), V, "bf16")
    p = make_params(rng, rows, len(z), V, S=64)
    want, _, _ = ref.process(z, rows, p, "bf16")
    assert same_bits(host(process(sv, z, rows, p, "bf16")), want).all()


def test_binding_refuses_on_the_gpu(sv):
    x = torch.randn(3, 264, device="cuda")
    off, tok = dev(i32([0, 2])), dev(i32([1, 2]))
    st = sv.PenaltyState(1, 264)
    pen = dict(counts=st.counts, seen=st.seen)
    with pytest.raises(ValueError, match="counts, seen and draft_tokens"):
        sv.spec_logits_process(x, off, **pen)
    with pytest.raises(ValueError, match="counts, seen and draft_tokens"):
        sv.spec_logits_process(x, off, tok, repetition=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="parent"):
        sv.spec_logits_process(x, off, tok, rows="tree", **pen)
    with pytest.raises(ValueError, match="seen must have"):
        sv.spec_logits_process(x, off, tok, counts=st.counts, seen=st.seen[:, :1].contiguous())
    with pytest.raises(ValueError, match="biases"):
        sv.spec_logits_process(x, off, tok, bias_offsets=off)
    with pytest.raises(ValueError, match="mask_rows"):
        sv.spec_logits_process(x, off, tok, mask_rows=tok)
    with pytest.raises(ValueError, match="mask needs"):
        sv.spec_logits_process(x, off, tok, mask=torch.zeros(2, 9, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="mask must have"):
        sv.spec_logits_process(x, off, tok, mask=torch.zeros(3, 8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        sv.spec_logits_process(x[:, ::2], off, tok)
    with pytest.raises(TypeError):
        sv.spec_logits_process(x.half(), off, tok)
    with pytest.raises(TypeError):
        sv.spec_logits_truncate(x, torch.ones(1, device="cuda"), off, top_k=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="temperature must have"):
        sv.spec_logits_truncate(x, torch.ones(2, device="cuda"), off)
    with pytest.raises(ValueError, match="out must have"):
        sv.spec_logits_truncate(x, torch.ones(1, device="cuda"), off, out=x[:2].contiguous())
    with pytest.raises(sv.SpecError) as e:  # an output that overlaps the logits
        buf = torch.randn(5 * 264, device="cuda")
        sv.spec_logits_process(buf[:3 * 264].view(3, 264), off, tok, out=buf[264:4 * 264].view(3, 264))
    assert e.value.code == -1
    with pytest.raises(sv.SpecError) as e:
        sv.spec_logits_process(torch.randn(3, 262, device="cuda"), off, tok)
    assert e.value.code == -2
    with pytest.raises(ValueError, match="offsets and tokens"):
        st.reset(tok, prompt_offsets=dev(i32([0, 1, 2])))
    with pytest.raises(ValueError, match="'target' or 'tree'"):
        st.update(tok, tok[:1], off, rows="draft")


# ------------------------------------------------------------------- the counts
@pytest.mark.parametrize("V", [8, 1000, 4100, 9000])
def test_reset_and_update(sv, V):
    rng = np.random.default_rng(V)
    S, n = 9, 6
    st = sv.PenaltyState(S, V)
    counts, prompt = np.zeros((S, V), i32), np.zeros((S, V), bool)
    # stale contents, that a reset has to replace
    st.counts.fill_(5)
    st.seen.fill_(-1)
    counts[:] = 5
    slots = i32([4, 0, 8, 4, S, -1])  # slot 4 twice: the later entry has it; two slots that do not exist
    lens, outs = i32([3, 0, 700, 40, 2, 2]), i32([0, 5, 900, 7, 1, 1])
    po, oo = np.concatenate([[0], np.cumsum(lens)]).astype(i32), np.concatenate([[0], np.cumsum(outs)]).astype(i32)
    pt, ot = rng.integers(0, V, po[-1]).astype(i32), (rng.random(oo[-1]) ** 4 * V).astype(i32)
    pt[po[2]], ot[oo[2]] = V, -1  # not counted
    for i in (1, 2, 3):
        s = slots[i]
        a, b = pt[po[i]:po[i + 1]], ot[oo[i]:oo[i + 1]]
        counts[s], prompt[s] = np.bincount(b[(b >= 0) & (b < V)], minlength=V), False
        prompt[s, a[(a >= 0) & (a < V)]] = True
    st.reset(dev(slots), dev(po), dev(pt), dev(oo), dev(ot))
    assert (st.counts.cpu().numpy() == counts).all()
    touched = [0, 4, 8]
    words = ref.pack(np.stack([prompt, counts > 0], 1))
    assert (st.seen.cpu().numpy()[touched] == words[touched]).all()
    untouched = [s for s in range(S) if s not in touched]
    assert (st.seen.cpu().numpy()[untouched] == -1).all()
    st.reset(dev(np.arange(S, dtype=i32)))  # every slot empty
    assert not st.counts.any() and not st.seen.any()

    for mode in ("target", "tree"):
        ks = np.array([3, 0, 32, 1, 5, 2])
        rows = make_rows(rng, mode, ks, V)
        R = rows.count()
        toks = (rng.random(R) ** 4 * V).astype(i32)
        toks[1] = -1
        acc = i32([3, 0, 20, -1, 6, 1])  # a data error; more accepted than drafted
        slots = i32([2, 2, 5, 1, 1, S])  # a shared slot; one that does not exist
        counts, first = st.counts.cpu().numpy(), rows.offsets[:-1] + (np.arange(6) if mode == "target" else 0)
        for b in (0, 1, 2):
            t = toks[first[b]:first[b] + acc[b] + 1]
            counts[slots[b]] += np.bincount(t[t >= 0], minlength=V).astype(i32)
        before = st.counts.clone()
        st.update(dev(toks), dev(acc), dev(i32([0, 3, 2, 4, 5, 6, 7])), rows=mode, slots=dev(slots))
        assert torch.equal(st.counts, before)  # invalid offsets: nothing is counted
        st.update(dev(toks), dev(acc), dev(rows.offsets), rows=mode, slots=dev(slots))
        assert (st.counts.cpu().numpy() == counts).all()
        assert (st.seen.cpu().numpy() == ref.pack(np.stack([np.zeros((S, V), bool), counts > 0], 1))).all()


def test_update_most_sequences(sv):
    B, V = sv.MAX_B, 264
    rng = np.random.default_rng(3)
    ks = rng.integers(0, 33, B)
    off = np.concatenate([[0], np.cumsum(ks)]).astype(i32)
    toks = rng.integers(0, V, off[-1] + B).astype(i32)
    acc = (rng.random(B) * (ks + 1)).astype(i32)
    st = sv.PenaltyState(B, V)
    st.update(dev(toks), dev(acc), dev(off))
    want = np.zeros((B, V), i32)
    for b in range(B):
        np.add.at(want[b], toks[off[b] + b:off[b] + b + acc[b] + 1], 1)
    assert (st.counts.cpu().numpy() == want).all()
    assert (st.seen.cpu().numpy()[:, 1] == ref.pack(want > 0)).all()


# ------------------------------------------------------------------- truncation
def zipf(rng, R, V, dtype, quantum=0.0):
    z = -1.1 * np.log1p(rng.random((R, V)) * V) + rng.standard_normal((R, V))
    if quantum:
        z = np.round(z / quantum) * quantum
    z = z.astype(f32)
    return ref.to_bf16(z) if dtype == "bf16" else z


def settings(rng, kind, B, V):
    s = {}
    if "k" in kind:
        s["top_k"] = rng.choice(i32([1, 2, 7, 50, V // 2, V - 1, V, 2 * V, 0]), B)
    if "p" in kind:
        s["top_p"] = rng.choice(f32([1e-30, 0.1, 0.5, 0.9, 0.95, 0.999, 1 - 2.0 ** -24, 1.0]), B)
    if "m" in kind:
        s["min_p"] = rng.choice(f32([0, 1e-30, 1e-4, 0.02, 0.1, 0.9, 1.0]), B)
    return s


def check_truncate(got, z, seq, T, s):
    want, margin = ref.truncate(z, seq, T, **s)
    ok = same_bits(got, want).all(axis=1)
    assert (ok | (margin < 1e-10)).all(), (np.flatnonzero(~ok), margin[~ok], [np.flatnonzero(~same_bits(got[r], want[r]))[:5] for r in np.flatnonzero(~ok)[:3]])
    return int((~ok).sum())


def truncate(sv, z, off, T, s, dtype, **kw):
    return sv.spec_logits_truncate(dev(z, dtype), dev(T), dev(off), **{k: dev(v) for k, v in s.items()}, **kw)


@pytest.mark.parametrize("V", [8, 264, 1000, 4104, 32000, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["k", "p", "m", "kp", "kpm"])
def test_truncate(sv, kind, dtype, V):
    rng = np.random.default_rng(V + 7 * len(kind))
    B = 24 if V < 32000 else 10
    rows = make_rows(rng, "target", rng.integers(0, 3, B), V)
    seq = ref.row_sequences(rows)
    z = zipf(rng, len(seq), V, dtype)
    T = rng.choice(f32([0.0, 0.1, 0.7, 1.0, 1.0, 3.0]), B)
    s = settings(rng, kind, B, V)
    got = host(truncate(sv, z, rows.offsets, T, s, dtype))
    assert check_truncate(got, z, seq, T, s) == 0


@pytest.mark.parametrize("dtype,V", [("bf16", 4104), ("fp32", 4104), ("fp32", 32000), ("bf16", 152064)])
@pytest.mark.parametrize("what", ["ties", "coarse", "equal", "lowest", "masked", "few", "huge", "tiny", "both_signs", "constant_tail"])
def test_truncate_hard_rows(sv, what, dtype, V):
    """Ties by the thousand, rows of one value, masks of the type's lowest value or -inf, values of any size."""
    rng = np.random.default_rng(len(what))
    B = 14
    z = zipf(rng, B, V, dtype)
    T = rng.choice(f32([0.3, 1.0, 2.0]), B)
    if what == "ties":
        z = zipf(rng, B, V, dtype, 0.25)
    elif what == "coarse":
        z = zipf(rng, B, V, dtype, 4.0)
    elif what == "equal":
        z[:] = f32(1.5)
    elif what == "lowest":
        z[rng.random(z.shape) < 0.9] = LOWEST[dtype]
    elif what == "masked":
        z[rng.random(z.shape) < 0.99] = -np.inf
    elif what == "few":
        z[:] = -np.inf
        z[np.arange(B), rng.integers(0, V, B)] = 3.0
        z[:B // 2, V - 1] = 3.0
    elif what == "huge":
        z *= f32(2.0) ** rng.integers(10, 120, (B, 1)).astype(f32)
        T = (f32(2.0) ** rng.integers(0, 100, B)).astype(f32)
    elif what == "tiny":
        z *= f32(2.0) ** -rng.integers(20, 120, (B, 1)).astype(f32)
        T = (f32(2.0) ** -rng.integers(0, 100, B)).astype(f32)
    elif what == "both_signs":
        z = z * 0.01
        z[:, ::3] *= -1
        z[:, ::7] = 0.0
        z[:, 1::7] = -0.0
    else:
        z[:, V // 8:] = f32(-2.0)
    z = ref.to_bf16(z) if dtype == "bf16" else z.astype(f32)
    off = np.zeros(B + 1, i32)
    for kind in ("k", "p", "kpm"):
        s = settings(rng, kind, B, V)
        got = host(truncate(sv, z, off, T, s, dtype))
        check_truncate(got, z, np.arange(B), T, s)


@pytest.mark.parametrize("V", [10000, 20000, 70000])
@pytest.mark.parametrize("B", [3, 60, 120, 330])
def test_truncate_rows_shared_or_not(sv, V, B):
    """Few rows are shared by clusters of 2, 4 and 8 CTAs, many are not; ties across the CTAs' parts of a row."""
    rng = np.random.default_rng(B + V)
    z = zipf(rng, min(B, 24), V, "bf16", 0.25)
    z[1, 5] = 2.0 ** -40  # a value without a bin
    z[2, ::2] = -np.inf
    rows = np.arange(B) % len(z)
    off, T = np.zeros(B + 1, i32), rng.choice(f32([0.5, 1.0]), B)
    s = settings(rng, "kp", B, V)
    got = host(truncate(sv, z[rows], off, T, s, "bf16"))
    check = np.arange(B) if B < 30 else np.concatenate([np.arange(12), rng.choice(np.arange(12, B), 12, replace=False)])
    check_truncate(got[check], z[rows[check]], check, T, s)


@pytest.mark.parametrize("dtype,V", [("bf16", 1032), ("fp32", 4100)])
def test_truncate_left_alone(sv, dtype, V):
    """Greedy rows, rows with NaN or +inf, rows of -inf: their own bits.  And nothing set: every row."""
    rng = np.random.default_rng(5)
    z = zipf(rng, 6, V, dtype)
    z[1, 7], z[2, V - 1], z[3] = np.nan, np.inf, -np.inf
    T = f32([0, 1, 1, 1, 1, 1])
    off = np.zeros(7, i32)
    s = dict(top_k=i32([3, 3, 3, 3, 0, 0]), top_p=f32([.5, .5, .5, .5, 1, 1]), min_p=f32([.5, .5, .5, .5, 0, 0]))
    for given in (s, {}):
        for in_place in (False, True):
            x = dev(z, dtype)
            got = host(sv.spec_logits_truncate(x, dev(T), dev(off), out=x if in_place else None, **{k: dev(v) for k, v in given.items()}))
            assert same_bits(got, z).all()


@pytest.mark.parametrize("dtype,V", [("bf16", 1032), ("fp32", 4100)])
def test_truncate_data_errors(sv, dtype, V):
    rng = np.random.default_rng(6)
    B = 12
    z = zipf(rng, B, V, dtype)
    T, s = np.ones(B, f32), dict(top_k=np.full(B, 20, i32), top_p=np.full(B, 0.9, f32), min_p=np.full(B, 0.01, f32))
    T[1], T[2], T[3] = -1, np.nan, np.inf
    s["top_k"][4] = -1
    s["top_p"][5], s["top_p"][6], s["top_p"][7] = 0, 1.5, np.nan
    s["min_p"][8], s["min_p"][9], s["min_p"][10] = -0.1, 1.1, np.nan
    bad = np.arange(1, 11)
    off = np.zeros(B + 1, i32)
    good = [0, 11]
    for in_place in (False, True):
        x = dev(z, dtype)
        got = host(sv.spec_logits_truncate(x, dev(T), dev(off), out=x if in_place else None, **{k: dev(v) for k, v in s.items()}))
        assert np.isnan(got[bad]).all()
        check_truncate(got[good], z[good], [0, 11], T, s)


@pytest.mark.parametrize("mode", ["draft", "next", "tree"])
def test_truncate_layouts(sv, mode):
    rng = np.random.default_rng(8)
    rows = make_rows(rng, mode, KS["ragged"], 2056)
    seq = ref.row_sequences(rows)
    z = zipf(rng, len(seq) + 2, 2056, "bf16")
    T, s = rng.choice(f32([0.5, 1.0]), rows.B), settings(rng, "kp", rows.B, 2056)
    out = torch.full((len(z), 2056), 7.0, dtype=torch.bfloat16, device="cuda")
    got = host(truncate(sv, z, rows.offsets, T, s, "bf16", rows=mode, out=out))
    assert check_truncate(got[:-2], z[:-2], seq, T, s) == 0 and (got[-2:] == 7).all()
    x = dev(z, "bf16")
    sv.spec_logits_truncate(x, dev(T), dev(rows.offsets), rows=mode, out=x, **{k: dev(v) for k, v in s.items()})
    assert same_bits(host(x)[:-2], got[:-2]).all() and same_bits(host(x)[-2:], z[-2:]).all()


# ------------------------------------------------------------------- the limits
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_vocabulary(sv, dtype):
    """MAX_V columns, processed and truncated."""
    rng = np.random.default_rng(31)
    V = sv.MAX_V
    rows = ref.Rows("target", i32([0, 1]), i32([V - 1]))
    z = zipf(rng, 2, V, dtype)
    st = sv.PenaltyState(1, V)
    prompt = rng.integers(0, V, 5000).astype(i32)
    st.reset(dev(i32([0])), dev(i32([0, 5000])), dev(prompt), dev(i32([0, 3])), dev(i32([7, V - 1, 7])))
    p = dict(counts=st.counts.cpu().numpy(), seen=st.seen.cpu().numpy(), repetition=f32([1.5]), frequency=f32([0.5]))
    assert p["counts"].sum() == 3 and p["counts"][0, V - 1] == 1
    want, _, _ = ref.process(z, rows, p, dtype)
    x = process(sv, z, rows, {k: v for k, v in p.items()}, dtype)
    assert same_bits(host(x), want).all()
    s = dict(top_p=f32([0.9]), min_p=f32([1e-5]))
    got = host(sv.spec_logits_truncate(x, dev(f32([0.8])), dev(rows.offsets), **{k: dev(v) for k, v in s.items()}))
    check_truncate(got, want, [0, 0], f32([0.8]), s)


def test_offsets_past_32_bits(sv):
    """Rows that start behind 4 GB: the last ones as the same rows alone."""
    V, B = sv.MAX_V, 140  # 4.7 GB of bf16
    x = torch.empty(B, V, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.randn(1, V, device="cuda"))
    x[-2:] = torch.randn(2, V, device="cuda").to(torch.bfloat16)
    last = x[-2:].clone()
    off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    tok = torch.zeros(0, dtype=torch.int32, device="cuda")
    bias = dict(bias_tokens=torch.full((B,), V - 1, dtype=torch.int32, device="cuda"), bias_values=torch.full((B,), 9.0, device="cuda"))
    count = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    y = sv.spec_logits_process(x, off, tok, bias_offsets=count, **bias)
    one = sv.spec_logits_process(last, off[:3], tok, bias_offsets=count[:3], **{k: v[:2] for k, v in bias.items()})
    assert torch.equal(y[-2:], one) and float(one[0, -1]) == float((last[0, -1].float() + 9).to(torch.bfloat16))
    assert torch.equal(y[:-2, :-1], x[:-2, :-1])
    sv.spec_logits_process(x, off, tok, bias_offsets=count, out=x, **bias)
    assert torch.equal(x, y)
    k = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    sv.spec_logits_truncate(x, torch.ones(B, device="cuda"), off, top_k=k, out=x)
    alone = sv.spec_logits_truncate(one, torch.ones(2, device="cuda"), off[:3], top_k=k[:2])
    assert torch.equal(x[-2:], alone) and bool((torch.isfinite(x).sum(1) == 40).all())


# ------------------------------------------------------------------------- both
@pytest.mark.parametrize("mode", ["target", "draft", "next", "tree"])
@pytest.mark.parametrize("dtype,V", [("bf16", 264), ("bf16", 32000), ("fp32", 4100)])
def test_both_equal_the_two_calls(sv, mode, dtype, V):
    rng = np.random.default_rng(V)
    rows = make_rows(rng, mode, KS["ragged"], V)
    z = zipf(rng, rows.count(), V, dtype)
    p = make_params(rng, rows, len(z), V)
    if "slots" in p:
        p["slots"][1] = -5  # an invalid sequence among them
    T, s = rng.choice(f32([0.0, 0.7, 1.0]), rows.B), settings(rng, "kpm", rows.B, V)
    T[2] = np.nan
    x, off, tok = dev(z, dtype), dev(rows.offsets), dev(rows.tokens)
    a = {k: dev(v) for k, v in p.items()}
    t = {k: dev(v) for k, v in s.items()}
    parent = None if rows.parent is None else dev(rows.parent)
    one = sv.spec_logits_process(x, off, tok, rows=mode, parent=parent, **a)
    two = sv.spec_logits_truncate(one, dev(T), off, rows=mode, **t)
    both = sv.spec_logits_process_truncate(x, dev(T), off, tok, rows=mode, parent=parent, **a, **t)
    assert same_bits(host(both), host(two)).all()
    sv.spec_logits_process_truncate(x, dev(T), off, tok, rows=mode, parent=parent, out=x, **a, **t)
    assert same_bits(host(x), host(two)).all()


# ------------------------------------------------------------- streams and graphs
def test_streams_and_graph_replay(sv):
    """Two calls at once on two streams, and both operators captured and replayed on changed inputs."""
    rng = np.random.default_rng(21)
    V = 4104
    rows = make_rows(rng, "target", KS["ragged"], V)
    zs = [zipf(rng, rows.count(), V, "bf16") for _ in range(3)]
    p = make_params(rng, rows, len(zs[0]), V, mask=False)
    T, s = np.ones(rows.B, f32), settings(rng, "kpm", rows.B, V)
    off, tok, Td = dev(rows.offsets), dev(rows.tokens), dev(T)
    a, t = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in s.items()}
    x = [dev(z, "bf16") for z in zs]

    def go(x, out=None):
        return sv.spec_logits_process_truncate(x, Td, off, tok, out=out, **a, **t)

    want = [go(v) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st, v in zip(streams, x):
        with torch.cuda.stream(st):
            got.append(go(v))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert same_bits(host(g), host(w)).all()
    src, out = x[0].clone(), torch.empty_like(x[0])
    counts = sv.PenaltyState(rows.B, V)
    emitted, acc = dev(rng.integers(0, V, len(zs[0])).astype(i32)), dev(np.diff(rows.offsets).astype(i32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(src, out)
        counts.update(emitted, acc, off)
    for v, w in zip(x, want):
        src.copy_(v)
        graph.replay()
        assert same_bits(host(out), host(w)).all()
    assert int(counts.counts.sum()) == 3 * len(zs[0])
