"""GPU: beam selection where scores and logits are far from ordinary: hypotheses that went on with a token masked by
a large finite value have that value for a score."""
from __future__ import annotations

import numpy as np
import pytest

import states_ref as ref
from beam_check import LOWEST, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
LOWEST_BF16 = -3.3895313892515355e38
MASKS = [-1e9, -1e29, -1e30, -1e31, -1e32, -3e38, LOWEST_BF16, LOWEST]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(sv, z, scores, offsets, n, dtype, ended=None, end_token=0):
    t = dev(np.clip(z, LOWEST_BF16, None).astype(f32)).bfloat16() if dtype == "bf16" else dev(z.astype(f32))
    got = sv.spec_beam_select(t, dev(scores.astype(f32)), dev(np.asarray(offsets, i32)), n,
                              ended=None if ended is None else dev(ended), end_token=end_token, lse=True)
    check(got, t.float().cpu().numpy(), scores.astype(f32), offsets, n, ended, end_token)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", MASKS)
@pytest.mark.parametrize("mask", MASKS)
def test_a_masked_score_over_masked_logits(sv, dtype, score, mask):
    """Tokens masked by a finite value before and behind the ordinary ones, in rows of ordinary and of masked scores."""
    z = np.array([[mask, 4, 2, mask, -1, 0, mask, 3], [1, mask, mask, mask, 5, mask, mask, 4], [mask] * 8], f32)
    scores = np.array([score, score, score, -2, -3, score], f32)
    got = run(sv, z[[0, 1, 2, 0, 1, 2]], scores, [0, 1, 3, 6], 8, dtype)
    assert got[1][0].tolist() == [1, 7, 2, 5, 4, 0, 3, 6]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G,V", [(1, 2000), (30, 2000), (170, 504)])
def test_rows_of_many_magnitudes(sv, dtype, G, V):
    """Logits and scores over all of the type's range, few groups and many."""
    rng = np.random.default_rng(G + V)
    R = 4 * G
    big = 10.0 ** rng.uniform(0, 38.5, (R, V))
    z = np.where(rng.random((R, V)) < 0.3, -big, rng.standard_normal((R, V)))
    z[::5] = np.where(rng.random((len(z[::5]), V)) < 0.5, big[::5], -big[::5])
    scores = -(10.0 ** rng.uniform(-3, 38.5, R))
    scores[::7] = 3e38
    ended = rng.random(R) < 0.1
    run(sv, z, scores, np.arange(0, R + 1, 4), 12, dtype, ended, 3)


def test_distances_past_float32(sv):
    """Logits from the lowest to the largest value, scores that bring their distance back, and scores below the lowest
    value, whose order is still the row's."""
    near = np.nextafter(f32(LOWEST), f32(0))
    z = np.array([[3e38, LOWEST, near, -1e38, 1e38, LOWEST, 2.9e38, -3e38],
                  [0, LOWEST, near, LOWEST, -1e38, near, -3e38, 1],
                  [1e36, near, LOWEST, near, LOWEST, LOWEST, near, near]], f32)
    for scores in ([3e38, 3e38, 3e38], [0, -1e30, -5], [LOWEST, LOWEST, LOWEST], [3.4e38, LOWEST, 1e31], [-1e38, -2e38, -3e38]):
        run(sv, z, np.array(scores, f32), [0, 3], 24, "fp32")
        run(sv, z, np.array(scores, f32), [0, 1, 2, 3], 5, "fp32")


def test_ordered_by_its_logits_at_a_very_low_score(sv):
    """A row's order at a score whose float32 step is far larger than its logits."""
    rng = np.random.default_rng(1)
    z = rng.standard_normal((3, 3000)).astype(f32)
    z[:, ::3] = -1e31
    run(sv, z, np.array([-1e31, -1e31, LOWEST], f32), [0, 2, 3], 100, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-1e18, -1e20, -1e29, -1e30, -1e31, -1e35, LOWEST_BF16, LOWEST])
@pytest.mark.parametrize("G,V", [(1, 64), (24, 2048), (160, 64)])
def test_masked_tokens_of_several_rows_tie(sv, dtype, mask, G, V):
    """More candidates than tokens that are not masked: those masked by one value have equal scores in 64 bits, whatever
    their rows' scores, and go by row, then token."""
    rng = np.random.default_rng(G)
    W, n = 3, 48
    R = G * W
    z = np.full((R, V), max(mask, LOWEST_BF16) if dtype == "bf16" else mask, f32)
    for r in range(R):  # ten tokens, an eighth and more apart from each other within the group
        at = rng.permutation(V)[:10]
        z[r, at] = np.arange(10) * 0.5
    scores = (rng.permutation(R) % 7 - 20 + 0.125 * (np.arange(R) % W)).astype(f32)
    t = dev(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    off = np.arange(0, R + 1, W)
    want = ref.beam_select(t.float().cpu().numpy(), scores, off, n)
    got = sv.spec_beam_select(t, dev(scores), dev(off.astype(i32)), n)
    assert (np.abs(np.diff(want[0][:, :30])) > 1e-3).all()  # no two of the others so close that their order is open
    assert (got[1].cpu().numpy() == want[1]).all() and (got[2].cpu().numpy() == want[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G", [1, 24])
def test_equal_logits_below_the_largest(sv, dtype, G):
    """Terms whose roundings are all alike and do not average out: a row's sum is off by more than float32's
    step, as far as the header says and no further."""
    rng = np.random.default_rng(G)
    V = 128256
    z = np.empty((2 * G, V), f32)
    for i in range(2 * G):
        z[i] = rng.uniform(-20, 20)
        z[i, rng.integers(V)] = z[i, 0] + rng.uniform(5, 15)
    z[0], z[0, 5] = 8.823372, 20.057129
    run(sv, z, np.zeros(2 * G, f32), np.arange(0, 2 * G + 1, 2), 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-1e9, -1e30, -1e31, LOWEST_BF16])
@pytest.mark.parametrize("B", [2, 24])
def test_a_search_with_too_few_tokens(sv, dtype, mask, B):
    """Three steps; in the first, fewer tokens than beams are not masked, so that some hypotheses go on with a masked one."""
    rng = np.random.default_rng(B)
    W, V = 4, 40
    R = B * W
    offsets = np.arange(0, R + 1, W)
    scores = np.where(np.arange(R) % W == 0, 0, -np.inf).astype(f32)
    for step in range(3):
        z = rng.standard_normal((R, V)) * 3
        z[rng.random((R, V)) < (0.9 if step else 0)] = mask
        if step == 0:
            z[:, 2:] = mask
        got = run(sv, z, scores, offsets, W, dtype)
        scores = got[0].flatten().cpu().numpy()
        assert step or (scores.reshape(B, W) < -1e8).sum() == 2 * B
