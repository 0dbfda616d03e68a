"""GPU: beam selection against the restatement in 64 bits.

Tolerance of scores and log-sum-exps, in units of u = 2^-24 (half a step of fp32, relative): a term
2^((z - m) log2 e) is off by its argument's three roundings (the difference, the constant, the product: 3 u |arg| ln 2, at most
3 ln V u on average over the distribution, under 51 u for V = 2^24) and 4 u of the
exponential; a sum of at most 16 additions per term 16 u; the factor that brings a piece's sum to the row's
largest logit the same 51 u + 4 u again and one rounding.  Under 128 u in all, and u of the
result for its own rounding."""
from __future__ import annotations

import numpy as np
import pytest

import states_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TOL = 128 * U
f32, i32 = np.float32, np.int32
LOWEST = {"bf16": -3.3895313892515355e38, "fp32": float(np.finfo(np.float32).min)}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def logits(z, dtype):
    """The device tensor of the type, and its values."""
    t = dev(z.astype(f32), torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.float().cpu().numpy()


def compare(got, want, rows=None):
    s, t, r = (x.cpu().numpy() for x in got[:3])
    ws, wt, wr, wlse, every, z = want
    assert (np.isnan(s) == np.isnan(ws)).all()
    for b in range(len(ws)):
        if np.isnan(ws[b, 0]):
            assert (t[b] == -1).all() and (r[b] == -1).all()
            continue
        empty = ws[b] == -np.inf
        assert ((s[b] == -np.inf) == empty).all(), (b, s[b], ws[b])
        close = TOL + U * np.abs(ws[b][~empty])
        assert (np.abs(s[b][~empty] - ws[b][~empty]) <= close).all(), (b, s[b], ws[b])
        assert (t[b][empty] == -1).all() and (r[b][empty] == -1).all()
        differ = (t[b] != wt[b]) | (r[b] != wr[b])
        if not differ.any():
            continue
        # another candidate only where two rows' scores lie within the tolerance; within a row the order is exact
        pairs = list(zip(r[b][~empty], t[b][~empty]))
        assert len(set(pairs)) == len(pairs)
        for i in np.flatnonzero(differ):
            if every[r[b, i], t[b, i]] == -np.inf:  # an ended row's
                continue
            assert abs(every[r[b, i], t[b, i]] - ws[b, i]) <= 2 * TOL, (b, i)
            assert r[b, i] != wr[b, i], (b, i)
        for row in set(r[b][~empty]):
            order = [(-z[row, v], v) for rr, v in pairs if rr == row]
            assert order == sorted(order)
    if len(got) > 3:
        lse, wlse = got[3].cpu().numpy()[:rows], wlse[:rows]  # (rows behind the last group's are not written)
        assert (np.isnan(lse) == np.isnan(wlse)).all()
        fine = np.isfinite(wlse)
        assert (np.abs(lse[fine] - wlse[fine]) <= TOL + U * np.abs(wlse[fine])).all()
        assert (lse[~fine & ~np.isnan(wlse)] == wlse[~fine & ~np.isnan(wlse)]).all()


def run(sv, z, scores, offsets, n, dtype, ended=None, end_token=0, **kw):
    t, values = logits(z, dtype)
    got = sv.spec_beam_select(t, dev(scores.astype(f32)), dev(np.asarray(offsets, i32)), n,
                              ended=None if ended is None else dev(ended), end_token=end_token, lse=True, **kw)
    compare(got, ref.beam_select(values, scores.astype(f32), offsets, n, ended, end_token), offsets[-1])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [8, 16, 504, 1000, 1024, 1032, 32000, 128256])
@pytest.mark.parametrize("n", [1, 7, 32, 128])
def test_sizes(sv, dtype, V, n):
    rng = np.random.default_rng(V + n)
    per = [4, 0, 1, 8, 3] if V > 2000 else [4, 0, 1, 64, 33, 7]
    off = np.concatenate([[0], np.cumsum(per)])
    R = off[-1]
    z = -1.1 * np.log1p(rng.integers(0, V, (R, V))) + rng.standard_normal((R, V))
    run(sv, z, rng.standard_normal(R) * 2 - 20, off, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["equal", "few", "sorted", "rising", "front", "steps", "lowest", "all lowest", "masked", "empty rows", "large", "peak"])
@pytest.mark.parametrize("V,n", [(2000, 5), (9000, 64), (9000, 128)])
def test_rows_of_every_kind(sv, dtype, kind, V, n):
    """Ties, rows in order, masks of -inf and of the lowest value, large and peaked logits."""
    rng = np.random.default_rng(len(kind) + V)
    R, off = 12, [0, 4, 12]
    z = rng.standard_normal((R, V))
    if kind == "equal":
        z[:] = 1.5
    elif kind == "few":
        z = np.round(z)
    elif kind == "sorted":
        z = -np.sort(-z, axis=1)
    elif kind == "rising":
        z = np.sort(z, axis=1)
    elif kind == "front":
        z -= 2 * np.log1p(np.arange(V))
    elif kind == "steps":
        z = -(np.arange(V) // 700).astype(float)[None].repeat(R, 0)
    elif kind == "lowest":
        z[rng.random((R, V)) < 0.999] = LOWEST[dtype]
    elif kind == "all lowest":
        z[:6] = LOWEST[dtype]
        z[6:, 3:] = LOWEST[dtype]
    elif kind == "masked":
        z[rng.random((R, V)) < 0.999] = -np.inf
    elif kind == "empty rows":
        z[::2] = -np.inf
        z[5:, 2:] = -np.inf
    elif kind == "large":
        z = z * 1e6
    elif kind == "peak":
        z[:, 17] = 60
    run(sv, z, rng.standard_normal(R) - 3, off, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_rows_go_by_row_then_token(sv, dtype):
    z = np.tile(np.round(np.random.default_rng(3).standard_normal((1, 3000))), (8, 1))
    got = run(sv, z, np.zeros(8), [0, 8], 128, dtype)
    want = ref.beam_select(logits(z, dtype)[1], np.zeros(8, f32), [0, 8], 128)
    assert (got[1].cpu().numpy() == want[1]).all() and (got[2].cpu().numpy() == want[2]).all()


@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e3, 1e5, 1e30])
def test_scores_of_any_size(sv, scale):
    rng = np.random.default_rng(5)
    z = rng.standard_normal((10, 5000))
    run(sv, z, rng.standard_normal(10) * scale, [0, 3, 10], 20, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_dead_and_ended_rows_are_not_read(sv, dtype):
    rng = np.random.default_rng(7)
    R, V = 20, 4000
    z = rng.standard_normal((R, V))
    scores = rng.standard_normal(R) - 5
    ended = rng.random(R) < 0.3
    dead = rng.random(R) < 0.3
    scores[dead] = -np.inf
    z[ended | dead] = np.nan
    ended[16:] = True  # a group that has ended altogether
    scores[12:16] = -np.inf  # and one without a hypothesis
    run(sv, z, scores, [0, 5, 12, 16, 20], 12, dtype, ended, 11)
    # the first step: one row lives
    scores[:] = -np.inf
    scores[[0, 5]] = 0
    z[[0, 5]] = rng.standard_normal((2, V))
    run(sv, z, scores, [0, 5, 12], 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_data_errors_stay_in_their_group(sv, dtype):
    rng = np.random.default_rng(9)
    z = rng.standard_normal((14, 3000))
    scores = rng.standard_normal(14)
    z[1, 2999], z[4, 0], scores[7], scores[9] = np.nan, np.inf, np.nan, np.inf
    z[11] = -np.inf
    run(sv, z, scores, [0, 3, 6, 8, 10, 12, 14], 6, dtype)


@pytest.mark.parametrize("offsets", [[1, 4, 8], [0, 5, 4], [0, 4, 9], [0, -1, 4], [0, 4, 2 ** 31 - 1]])
def test_invalid_offsets(sv, offsets):
    t = torch.zeros(8, 1000, device="cuda")
    s, tok, r, lse = sv.spec_beam_select(t, torch.zeros(8, device="cuda"), dev(np.array(offsets, i32)), 4, lse=True)
    assert s.isnan().all() and (tok == -1).all() and (r == -1).all() and lse.isnan().all()
    t = torch.zeros(70, 1000, device="cuda")  # a group of more rows than a group may have
    s, tok, r = sv.spec_beam_select(t, torch.zeros(70, device="cuda"), dev(np.array([0, 65, 70], i32)), 4)
    assert s.isnan().all() and (tok == -1).all()


def test_padded_buffers_and_no_rows(sv):
    rng = np.random.default_rng(11)
    z = rng.standard_normal((10, 2000))
    t, values = logits(z, "fp32")
    t[6:] = np.nan
    got = sv.spec_beam_select(t, dev(np.zeros(10, f32)), dev(np.array([0, 2, 6], i32)), 5)
    compare(got, ref.beam_select(values[:6], np.zeros(6, f32), [0, 2, 6], 5))
    s, tok, r = sv.spec_beam_select(t, dev(np.zeros(10, f32)), dev(np.array([0], i32)), 5)
    assert s.shape == (0, 5)
    s, tok, r = sv.spec_beam_select(t[:0], dev(np.zeros(0, f32)), dev(np.array([0, 0, 0], i32)), 5)
    assert (s == -np.inf).all() and (tok == -1).all() and (r == -1).all()


def test_largest_vocabulary(sv):
    V = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn(3, V, generator=g, device="cuda")
    s, tok, r, lse = sv.spec_beam_select(z, torch.tensor([0.0, -1.0, -0.5], device="cuda"), dev(np.array([0, 3], i32)), 128, lse=True)
    every = torch.log_softmax(z.double(), 1) + torch.tensor([[0.0], [-1.0], [-0.5]], device="cuda").double()
    top = every.flatten().topk(128)
    assert (s[0].double() - top.values).abs().max() <= TOL + U * 30
    where = r[0].long() * V + tok[0].long()
    assert (every.flatten()[where] - top.values).abs().max() <= 2 * TOL
    assert (lse.double() - torch.logsumexp(z.double(), 1)).abs().max() <= TOL + U * 20


def test_many_groups(sv):
    rng = np.random.default_rng(13)
    per = rng.integers(0, 4, 4096)
    off = np.concatenate([[0], np.cumsum(per)])
    run(sv, rng.standard_normal((off[-1], 256)), rng.standard_normal(off[-1]), off, 3, "bf16")


@pytest.mark.parametrize("B", [3, 24])
def test_streams_workspace_and_capture(sv, B):
    """The same bits on another stream, with a workspace of the caller's that holds anything, and replayed; few groups
    in one launch, more in two."""
    rng = np.random.default_rng(15)
    t, _ = logits(rng.standard_normal((24, 20000)), "bf16")
    s, off = dev(rng.standard_normal(24).astype(f32)), dev((np.arange(B + 1) * (24 // B)).astype(i32))
    want = sv.spec_beam_select(t, s, off, 16, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_beam_select(t, s, off, 16, lse=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.full((sv.beam_workspace_bytes(24, 20000, sv.BF16),), 255, dtype=torch.uint8, device="cuda")
    got = sv.spec_beam_select(t, s, off, 16, lse=True, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(sv.SpecError, match="WORKSPACE"):
        sv.spec_beam_select(t, s, off, 16, workspace=ws[:-256])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.spec_beam_select(t, s, off, 16, lse=True)
    t2, _ = logits(rng.standard_normal((24, 20000)), "bf16")
    t.copy_(t2)
    g.replay()
    torch.cuda.synchronize()
    again = sv.spec_beam_select(t2, s, off, 16, lse=True)
    assert all(torch.equal(a, b) for a, b in zip(again, got)) and not torch.equal(want[1], got[1])


@pytest.mark.parametrize("B", [2, 30])
def test_many_more_rows_than_groups_hold(sv, B):
    """A buffer of far more rows than B groups can have."""
    rng = np.random.default_rng(17)
    z = rng.standard_normal((64 * B + 700, 264))
    off = np.concatenate([[0], np.cumsum(rng.integers(0, 65, B))])
    off[-1] = min(off[-2] + 64, off[-1])
    run(sv, z, rng.standard_normal(len(z)), off, 9, "bf16")


def test_two_calls_at_once(sv):
    """Calls on two streams, which may overlap, give what they give alone."""
    rng = np.random.default_rng(19)
    calls = []
    for B in (40, 4):
        t, _ = logits(rng.standard_normal((8 * B, 30000)), "bf16")
        calls.append((t, dev(rng.standard_normal(8 * B).astype(f32)), dev((np.arange(B + 1) * 8).astype(i32)), 16))
    want = [sv.spec_beam_select(*c, lse=True) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k in range(2):
            got[k].append(sv.spec_beam_select(*calls[k], lse=True, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for g in got[k] for a, b in zip(want[k], g))


def test_binding_refusals(sv):
    z, s, off = torch.zeros(4, 1000, device="cuda"), torch.zeros(4, device="cuda"), dev(np.array([0, 4], i32))
    with pytest.raises(ValueError, match="n must be"):
        sv.spec_beam_select(z, s, off, 129)
    with pytest.raises(ValueError, match="scores"):
        sv.spec_beam_select(z, s[:3], off, 4)
    with pytest.raises(ValueError, match="contiguous"):
        sv.spec_beam_select(z.t(), s, off, 4)
    with pytest.raises(TypeError):
        sv.spec_beam_select(z.half(), s, off, 4)
    with pytest.raises(TypeError):
        sv.spec_beam_select(z, s, off.long(), 4)
    with pytest.raises(sv.SpecError, match="INVALID"):
        sv.spec_beam_select(z, s, off, 4, ended=torch.zeros(4, dtype=torch.bool, device="cuda"), end_token=1000)
    with pytest.raises(sv.SpecError, match="ALIGN"):
        sv.spec_beam_select(torch.zeros(4, 1001, device="cuda"), s, off, 4)
