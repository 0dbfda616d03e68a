"""The logit operators as a server runs them, round after round: draft rows
processed and truncated, drafted from, target rows processed and truncated with
the drafted tokens, verified, the emitted tokens counted.  Each step is held
to its plain restatement and to the fp64 oracle on the same logits."""
from __future__ import annotations

import numpy as np
import pytest

import logits_ref as ref
import oracle
from parity import FLAG_MARGIN

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(z, dtype):
    return (z.view(np.uint32) >> 16).astype(np.uint16) if dtype == "bf16" else z


@pytest.mark.parametrize("dtype,V", [("bf16", 1000), ("fp32", 1000), ("bf16", 32000)])
def test_rounds(sv, dtype, V):
    rng = np.random.default_rng(V)
    ks = np.array([4, 0, 2, 5, 3, 4])
    B, off = len(ks), np.concatenate([[0], np.cumsum(ks)]).astype(i32)
    R_d, R_t = int(off[-1]), int(off[-1]) + B
    torch_type = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = f32([1, 1, 0.7, 0, 1.3, 1])
    s = dict(top_k=i32([0, 40, 0, 10, 100, 0]), top_p=f32([0.9, 1, 0.95, 0.9, 0.8, 1]), min_p=f32([0, 0, 0, 0, 0, 0.05]))
    pen = dict(repetition=f32([1.2, 1, 1.1, 1.3, 1, 2]), frequency=f32([0.5, 0.2, 0, 0.4, 0, 1]), presence=f32([0, 0.5, 0.3, 0, 0, 1]))
    prompts = [rng.integers(0, V, n).astype(i32) for n in (5, 0, 100, 30, 1, 64)]
    po = np.concatenate([[0], np.cumsum([len(t) for t in prompts])]).astype(i32)
    slots = rng.permutation(B + 2)[:B].astype(i32)
    st = sv.PenaltyState(B + 2, V)
    st.reset(dev(slots), dev(po), dev(np.concatenate(prompts)))
    counts, prompt = np.zeros((B + 2, V), i32), np.zeros((B + 2, V), bool)
    for b, t in enumerate(prompts):
        prompt[slots[b], t] = True
    d_off, d_T, d_slots = dev(off), dev(T), dev(slots)
    settings = {k: dev(v) for k, v in {**pen, **s}.items()}
    base = (-1.1 * np.log1p(np.arange(V))).astype(f32)  # the same favourites every round, so that penalties bite
    for step in range(4):
        zt = base + rng.standard_normal((R_t, V)).astype(f32)
        zd = zt[np.concatenate([np.arange(off[b] + b, off[b + 1] + b) for b in range(B)])] + 0.5 * rng.standard_normal((R_d, V)).astype(f32)
        zt, zd = (ref.to_bf16(z) if dtype == "bf16" else z.astype(f32) for z in (zt, zd))
        mask = rng.random((R_t, V)) < 0.7
        mask[0] = False  # this grammar allows nothing at the first row of sequence 0
        words, mask_rows = ref.pack(mask), np.where(np.repeat(np.arange(B), ks + 1) % 2 == 0, np.arange(R_t), -1).astype(i32)
        if step < 3:
            mask_rows[0] = -1
        u = {n: (rng.integers(0, 1 << 24, m) * 2.0 ** -24).astype(f32) for n, m in (("d", R_d), ("a", R_d), ("r", R_t))}
        seen = ref.pack(np.stack([prompt, counts > 0], 1))
        plain = dict(counts=counts, seen=seen, slots=slots, **pen)

        # drafting: this test's drafter draws its rows in order, so that row i follows the tokens before it
        toks = np.zeros(R_d, i32)
        for i in range(int(ks.max())):
            rows = ref.Rows("draft", off, toks)
            want, _, _ = ref.process(zd, rows, plain, dtype)
            want, margin = ref.truncate(want, ref.row_sequences(rows), T, **s)
            got = sv.spec_logits_process_truncate(dev(zd).to(torch_type), d_T, d_off, dev(toks), rows="draft", counts=st.counts,
                                                  seen=st.seen, slots=d_slots, **settings)
            assert margin.min() > 1e-10 and np.array_equal(got.float().cpu().numpy(), want)
            drawn = sv.spec_draft_sample(got, d_T, dev(u["d"]), d_off).cpu().numpy()
            od = oracle.draft_sample(bits(want, dtype), T, u["d"], off)
            ok = od.margin > FLAG_MARGIN
            assert (drawn[ok] == od.tokens[ok]).all() and (drawn >= 0).all()
            at = off[:-1][ks > i] + i
            toks[at] = drawn[at]
            assert np.isfinite(want[at, toks[at]]).all()
        q = got

        rows = ref.Rows("target", off, toks)
        want, _, _ = ref.process(zt, rows, {**plain, "mask": words, "mask_rows": mask_rows}, dtype)
        want, margin = ref.truncate(want, ref.row_sequences(rows), T, **s)
        p = sv.spec_logits_process(dev(zt).to(torch_type), d_off, dev(toks), counts=st.counts, seen=st.seen, slots=d_slots,
                                   mask=dev(words), mask_rows=dev(mask_rows), **{k: settings[k] for k in pen})
        p = sv.spec_logits_truncate(p, d_T, d_off, out=p, **{k: settings[k] for k in s})
        assert margin.min() > 1e-10 and np.array_equal(p.float().cpu().numpy(), want)

        out, n = sv.spec_verify(p, q, dev(toks), dev(u["a"]), dev(u["r"]), d_T, d_off)
        ov = oracle.verify(bits(want, dtype), bits(q.float().cpu().numpy(), dtype), toks, u["a"], u["r"], T, off)
        out_h, n_h = out.cpu().numpy(), n.cpu().numpy()
        if step == 3:
            assert n_h[0] == -1  # nothing was allowed: a data error of that sequence alone
        for b in range(B):
            o = off[b] + b
            if ov.num_accepted[b] >= 0 and ov.margin[b] <= FLAG_MARGIN:
                continue
            assert n_h[b] == ov.num_accepted[b] and (out_h[o:o + ks[b] + 1] == ov.tokens[o:o + ks[b] + 1]).all()
        st.update(out, n, d_off, slots=d_slots)
        for b in range(B):
            for t in out_h[off[b] + b:off[b] + b + n_h[b] + 1]:
                counts[slots[b], t] += 1
        assert np.array_equal(st.counts.cpu().numpy(), counts)
        assert np.array_equal(st.seen.cpu().numpy(), ref.pack(np.stack([prompt, counts > 0], 1)))
