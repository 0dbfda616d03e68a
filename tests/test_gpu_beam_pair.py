"""GPU: beam selection in two launches, rows and then groups, as an ordinary batch runs: more groups than one launch of
clusters takes, with no more groups than SMs and with more of them, rows of 20 pieces and more."""
from __future__ import annotations

import numpy as np
import pytest

from beam_check import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
LOWEST = {"bf16": -3.3895313892515355e38, "fp32": float(np.finfo(f32).min)}
ROW = {"bf16": 20 * 1024 + 24, "fp32": 21 * 512 + 4}  # 2 KB pieces, the last one short


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
    t = dev(z.astype(f32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    got = sv.spec_beam_select(t, dev(scores.astype(f32)), dev(np.asarray(offsets, i32)), n,
                              ended=None if ended is None else dev(ended), end_token=end_token, lse=True)
    check(got, t.float().cpu().numpy(), scores.astype(f32), offsets, n, ended, end_token)
    return got


def groups(G, rng):
    """Offsets of G groups: of 0 to 3 rows where there are many, of up to 20 among few."""
    per = rng.integers(0, 4, G)
    per[:3] = (1, 20, 17) if G < 100 else (1, 5, 0)
    return np.concatenate([[0], np.cumsum(per)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["usual", "equal", "few", "sorted", "rising", "front", "lowest", "all lowest", "masked", "empty rows", "large", "peak"])
@pytest.mark.parametrize("G,n", [(24, 16), (24, 128), (160, 5)])
def test_rows_of_every_kind(sv, dtype, kind, G, n):
    rng = np.random.default_rng(G + n + len(kind))
    off, V = groups(G, rng), ROW[dtype]
    R = off[-1]
    z = rng.standard_normal((R, V), f32)
    if kind == "equal":
        z[:] = 1.5
    elif kind == "few":
        z = np.round(z)
    elif kind == "sorted":
        z = -np.sort(-z, axis=1)
    elif kind == "rising":
        z = np.sort(z, axis=1)
    elif kind == "front":
        z -= 2 * np.log1p(np.arange(V, dtype=f32))
    elif kind == "lowest":
        z[rng.random((R, V), f32) < 0.9997] = LOWEST[dtype]
    elif kind == "all lowest":
        z[::2] = LOWEST[dtype]
        z[1::2, 3:] = LOWEST[dtype]
    elif kind == "masked":
        z[rng.random((R, V), f32) < 0.9997] = -np.inf
    elif kind == "empty rows":
        z[::2] = -np.inf
        z[R // 2:, 2:] = -np.inf
    elif kind == "large":
        z *= f32(1e6)
    elif kind == "peak":
        z[:, 17] = 60
    run(sv, z, rng.standard_normal(R) - 3, off, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G", [24, 160])
@pytest.mark.parametrize("scale", [1.0, 1e5, 1e30])
def test_scores_ended_and_dead_rows(sv, dtype, G, scale):
    """Rows that are not read hold NaN; a tenth of the groups has ended, another has no hypothesis."""
    rng = np.random.default_rng(G)
    off, V = groups(G, rng), ROW[dtype]
    R = off[-1]
    z = rng.standard_normal((R, V), f32)
    scores = rng.standard_normal(R) * scale - 5
    ended, dead = rng.random(R) < 0.3, rng.random(R) < 0.2
    for b in range(0, G, 10):
        ended[off[b]: off[b + 1]] = True
        dead[off[b + 3]: off[b + 4]] = True
    scores[dead] = -np.inf
    z[ended | dead] = np.nan
    run(sv, z, scores, off, 12, dtype, ended, V - 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G", [24, 160])
def test_data_errors_stay_in_their_group(sv, dtype, G):
    rng = np.random.default_rng(G)
    V = ROW[dtype]
    off = np.arange(0, 2 * G + 1, 2)
    z, scores = rng.standard_normal((2 * G, V), f32), rng.standard_normal(2 * G)
    z[1, V - 1], z[4, 0], scores[7], scores[9], z[2 * G - 1, V // 2] = np.nan, np.inf, np.nan, np.inf, np.nan
    z[11] = -np.inf
    got = run(sv, z, scores, off, 6, dtype)
    assert torch.isnan(got[0][:, 0]).nonzero().flatten().tolist() == [0, 2, 3, 4, G - 1]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G", [24, 160])
@pytest.mark.parametrize("wrong", ["start", "falling", "past", "wide"])
def test_invalid_offsets(sv, dtype, G, wrong):
    rows = 3 * G if wrong != "wide" else 3 * G + 65
    off = np.arange(0, 3 * G + 1, 3)
    if wrong == "start":
        off[0] = 1
    elif wrong == "falling":
        off[G // 2] = off[G // 2 + 1] + 1
    elif wrong == "past":
        off[G] = rows + 1
    else:
        off[G] = off[G - 1] + 65
    t = torch.zeros((rows, ROW[dtype]), device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    s, tok, r, lse = sv.spec_beam_select(t, torch.zeros(rows, device="cuda"), dev(off.astype(i32)), 4, lse=True)
    assert s.isnan().all() and (tok == -1).all() and (r == -1).all() and lse.isnan().all()
