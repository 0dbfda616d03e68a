"""Where top-p's border falls, against exact arithmetic: rows of few values, whose
kept number is computed in decimals of 60 digits, with top_p set next to the
border on purpose.

What the kernels may be off by.  The maximum's weight is exactly 1; another
weight exp(-x) has a relative error of at most 2^-46 + x 2^-47 (the two-term
exponential's own, and that of the product x in two fp32 terms), and the sums
of these rows add at most 2^-43: below EPS = 2^-42 in all for the x <= 3 used
here.  For a row of n0 tokens at the maximum and n1 beside it, of weight w, the
mass of n0 + c tokens less p Z is therefore off by at most (c + p n1) EPS w <=
2 n1 EPS w, which is 2 n1 EPS of one token beside it: a border further than
that from a whole number of tokens has one answer."""
from __future__ import annotations

from decimal import ROUND_CEILING, Decimal, getcontext

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

f32, i32 = np.float32, np.int32
EPS = 2.0 ** -42
getcontext().prec = 60


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


def to_bf16(x):
    u = np.asarray(x, f32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(f32)


def weight(z, zmax, T):
    return ((Decimal(float(z)) - Decimal(float(zmax))) / Decimal(float(T))).exp()


def kept(levels, p):
    """levels: (tokens, weight) in the order.  How many tokens top-p keeps, and how
    far the border is from a whole number of tokens of its level."""
    target = Decimal(float(p)) * sum(n * w for n, w in levels)
    before, tokens = Decimal(0), 0
    for n, w in levels:
        if before + n * w >= target:
            x = (target - before) / w
            up = x.to_integral_value(ROUND_CEILING)
            return tokens + int(up), float(min(up - x, x - up + 1))
        before, tokens = before + n * w, tokens + n
    raise AssertionError("p <= 1")


def near_borders(n0, n1, w, least, each=2):
    """fp32 top_p whose border lies next to a whole number of the n1 tokens of weight w behind
    n0 of weight 1: the nearest on either side that are at least `least` of a token away."""
    if n1 > 1 << 16:
        c = np.unique(np.linspace(1, n1 - 1, 1 << 16).astype(np.int64))
    else:
        c = np.arange(0 if n1 == 1 else 1, max(n1, 1))
    Z = n0 + n1 * w
    p = ((n0 + c * w) / Z).astype(f32)
    off = (p.astype(np.float64) * Z - n0) / w - c  # in tokens: below 0 keeps n0 + c, above one more
    out = []
    for side in (-off, off):
        at = np.flatnonzero((side >= 2 * least) & (p < 1))
        out += list(p[at[np.argsort(side[at], kind="stable")[:each]]])
    return out


def rows_of(rng, V, levels, dtype):
    """A row with n tokens of each value, shuffled; the rest is -inf."""
    z = np.full(V, -np.inf, f32)
    z[:sum(n for n, _ in levels)] = np.concatenate([np.full(n, v, f32) for n, v in levels])
    z = rng.permutation(z)
    return to_bf16(z) if dtype == "bf16" else z


def run(sv, z, T, p, dtype, k=None):
    x = torch.from_numpy(z).cuda()
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    off = torch.zeros(len(z) + 1, dtype=torch.int32, device="cuda")
    dev = lambda a, t: torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    y = sv.spec_logits_truncate(x, dev(T, f32), off, top_p=dev(p, f32), top_k=None if k is None else dev(k, i32))
    return y.float().cpu().numpy()


def check(got, z, want):
    """The first `want` tokens of the order keep their bits, the others are -inf."""
    for r, n in enumerate(want):
        order = np.lexsort((np.arange(z.shape[1]), -z[r].astype(np.float64)))
        here = np.isfinite(got[r])
        assert here.sum() == n, (r, int(here.sum()), n)
        assert here[order[:n]].all() and (got[r][order[:n]] == z[r][order[:n]]).all()


# Distances below the maximum: a little under 0, 1, 2 and 3 halvings of the weight (the
# table's first entry, from below), and others.
NEAR = {"fp32": [-1e-6, -0.0003, -0.0054, -0.694372177, -0.693822205, -0.6945, -1.3869, -2.0801, -0.3, -1.9],
        "bf16": [-0.00048828125, -0.005401611328125, -0.69921875, -0.6953125, -1.390625, -2.078125, -0.30078125, -1.8984375]}


@pytest.mark.parametrize("V", [4104, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_top_p_of_two_values(sv, dtype, V):
    rng = np.random.default_rng(V)
    rows, T, ps, want = [], [], [], []
    for i, d in enumerate(NEAR[dtype]):
        t = f32([1.0, 1.0, 0.75, 2.0][i % 4])
        zmax = f32([0.0, 0.0, 3.0][i % 3]) if dtype == "fp32" else f32(0.0)
        z1 = f32(zmax + f32(d * t))
        z1 = float(to_bf16([z1])[0]) if dtype == "bf16" else float(z1)
        w = weight(z1, zmax, t)
        n0 = V // 2 + (0 if i % 2 else V // 3)
        n1 = V - n0
        least = 2 * n1 * EPS
        for p in near_borders(n0, n1, float(w), least):
            n, far = kept([(n0, Decimal(1)), (n1, w)], p)
            assert far > least
            rows.append(rows_of(rng, V, [(n0, zmax), (n1, z1)], dtype))
            T.append(t), ps.append(p), want.append(n)
    z = np.stack(rows)
    assert len(z) >= 20
    check(run(sv, z, T, ps, dtype), z, want)


def test_top_p_of_two_values_stated_rows(sv):
    """Borders of one token in two, and of one in 128256, that a weight off by 2^-24 puts on the wrong side."""
    z = np.full((2, 8), -np.inf, f32)
    z[0, [5, 2]] = 0.0, -0.694372177
    z[1, [1, 6]] = 0.0, -0.693822205
    ps = f32([0.666938841, 0.666816652])
    want = [kept([(1, Decimal(1)), (1, weight(z[r].min(where=np.isfinite(z[r]), initial=0), 0, 1))], ps[r]) for r in (0, 1)]
    assert [n for n, _ in want] == [2, 1] and all(far > 1e-9 for _, far in want)
    check(run(sv, z, np.ones(2), ps, "fp32"), z, [2, 1])
    rng = np.random.default_rng(1)
    z1 = -0.005401611328125
    row = rows_of(rng, 128256, [(109664, 0.0), (18592, z1)], "bf16")[None]
    n, far = kept([(109664, Decimal(1)), (18592, weight(z1, 0, 1))], f32(0.9))
    assert n == 115372 and far > 2 * 18592 * EPS
    for dtype in ("bf16", "fp32"):
        check(run(sv, row, np.ones(1), f32([0.9]), dtype), row, [n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_top_p_next_to_one_over_two_tokens(sv, dtype):
    """Two tokens, top_p the floats around 1 / (1 + w): the second one stays or goes."""
    rng = np.random.default_rng(3)
    rows, ps, want = [], [], []
    for d in NEAR[dtype]:
        w = weight(f32(d), 0, 1)
        p0 = f32(float(1 / (1 + w)))
        for p in (np.nextafter(p0, f32(0)), p0, np.nextafter(p0, f32(1))):
            n, far = kept([(1, Decimal(1)), (1, w)], p)
            if far <= 2 * EPS:
                continue
            rows.append(rows_of(rng, 264, [(1, 0.0), (1, d)], dtype))
            ps.append(p), want.append(n)
    assert set(want) == {1, 2} and len(rows) >= 20
    z = np.stack(rows)
    check(run(sv, z, np.ones(len(z)), ps, dtype), z, want)


@pytest.mark.parametrize("dtype,V,k", [("bf16", 32000, 9000), ("fp32", 32000, 9000), ("fp32", 32000, 700), ("bf16", 32000, 700)])
def test_top_p_of_the_first_k(sv, dtype, V, k):
    """Z is the mass of the first k tokens, whose ties go by index."""
    rng = np.random.default_rng(k)
    rows, ps, want = [], [], []
    for d in NEAR[dtype]:
        w, n0 = weight(f32(d), 0, 1), k // 2
        least = 2 * k * EPS
        for p in near_borders(n0, k - n0, float(w), least, 1):
            n, far = kept([(n0, Decimal(1)), (k - n0, w)], p)
            assert far > least
            rows.append(rows_of(rng, V, [(n0, 0.0), (V - n0, d)], dtype))
            ps.append(p), want.append(n)
    z = np.stack(rows)
    check(run(sv, z, np.ones(len(z)), ps, dtype, np.full(len(z), k)), z, want)


# ------------------------------------------------------------------ flat tails
# Many tokens of the same small weight: what is lost of each is lost of all alike.
def tail_borders(Z1, w, n1, least):
    """top_p that cut a tail of n1 tokens of about weight w behind a mass of 1 (Z1 in all): the fp32
    values nearest to a whole number of them on either side, and some others."""
    lo = f32(1 / Z1)
    bits = np.arange(int(lo.view(np.uint32)), int(f32(1).view(np.uint32)), dtype=np.uint32)
    p = bits.view(f32)[:1 << 16]
    x = (p.astype(np.float64) * Z1 - 1) / w
    frac = x - np.floor(x)
    ok = np.flatnonzero((x > 1) & (x < n1 - 1) & (frac > least) & (frac < 1 - least))
    order = ok[np.argsort(frac[ok], kind="stable")]
    return p[np.concatenate([order[:3], order[-3:], order[len(order) // 2:][:2]])]


# V, distance; the sums' rounding in a row of 2^24 columns is 2^-37, so that the bound
# is 2 n1 (2^-37 + 2^-41) of a token there
TAILS = [("fp32", 128256, -22.7), ("fp32", 128256, -25.0), ("fp32", 128256, -18.25), ("fp32", 4104, -20.3),
         ("bf16", 128256, -22.75), ("bf16", 128256, -18.25), ("fp32", 1 << 24, -24.3), ("bf16 any", 128256, -22.75)]


@pytest.mark.parametrize("dtype,V,d", TAILS)
def test_top_p_within_a_flat_tail(sv, dtype, V, d):
    rng = np.random.default_rng(V)
    top = f32(0)
    if dtype == "bf16 any":  # a value without a bin sends the row down the path for any row
        dtype, top = "bf16", f32(2.0 ** -40)
    d, n1 = float(f32(d)), V - 1
    w = weight(d, top, 1)
    least = 2 * n1 * (EPS if V < 1 << 20 else 2.0 ** -36.9)
    ps = tail_borders(float(1 + n1 * w), float(w), n1, max(least, 2.0 ** -9))
    assert len(ps) == 8
    want = []
    for p in ps:
        n, far = kept([(1, Decimal(1)), (n1, w)], p)
        assert far > least
        want.append(n)
    if V < 1 << 20:
        z = np.stack([rows_of(rng, V, [(1, top), (n1, d)], dtype) for _ in ps])
        check(run(sv, z, np.ones(8), ps, dtype), z, want)
    else:  # the order is the index's, but for the first token
        z = np.full((8, V), d, f32)
        z[:, 1000] = top
        got = run(sv, z, np.ones(8), ps, dtype)
        for r, n in enumerate(want):
            assert np.isfinite(got[r]).sum() == n and got[r, 1000] == 0 and np.isfinite(got[r, :n - 1]).all()


def test_top_p_within_thousands_of_small_values(sv):
    """bf16: 3840 values of either sign next to zero, a token each, far below one large value: their weights are
    the same to 2^-16, so that a rounding of each goes the same way."""
    V = 262144
    m = (2.0 ** np.arange(-32, -17)[:, None] * (1 + np.arange(128) / 128)).ravel()
    small = np.sort(np.concatenate([m, -m]).astype(f32))[::-1]
    rng = np.random.default_rng(8)
    rows, ps, want = [], [], []
    for top in (16.0, 18.0, 19.0, 19.5, 20.0, 20.25, 20.5):
        levels = [(1, Decimal(1))] + [(1, weight(v, top, 1)) for v in small]
        tail = sum(w for _, w in levels[1:])
        least = 2 * len(small) * EPS
        for p in tail_borders(float(1 + tail), float(tail) / len(small), len(small), 0.0):
            n, far = kept(levels, p)
            if far <= least:
                continue
            rows.append(rows_of(rng, V, [(1, top)] + [(1, v) for v in small], "bf16"))
            ps.append(p), want.append(n)
    z = np.stack(rows)
    assert len(z) >= 40
    check(run(sv, z, np.ones(len(z)), ps, "bf16"), z, want)


# -------------------------------------------------- rows near several borders at once
def lengths(row, T, k, p, m, delta):
    """The order, and the fewest and the most tokens kept if the masses are off by up to delta Z."""
    V = len(row)
    order = np.lexsort((np.arange(V), -row.astype(np.float64)))
    s = row[order].astype(np.float64)
    x = (s - s[0]) / float(T)
    most = V if k == 0 else min(k, V)
    w = np.exp(x[:most]).astype(np.longdouble)
    before = np.concatenate([[0], np.cumsum(w)[:-1]])
    Z = w.sum()
    short = max(int((before < (float(p) - delta) * Z).sum()), 1) if p < 1 else most
    long = max(int((before < (float(p) + delta) * Z).sum()), 1) if p < 1 else most
    by_min = int((x >= np.log(float(m))).sum()) if m > 0 else V
    return order, min(short, by_min), min(long, by_min)


@pytest.mark.parametrize("dtype,V", [("bf16", 4104), ("fp32", 4104), ("fp32", 32000), ("bf16", 152064)])
@pytest.mark.parametrize("what", ["ties", "coarse", "equal", "masked", "flat", "steps", "both_signs"])
def test_kept_tokens_are_a_prefix(sv, what, dtype, V):
    """Whatever the row, a prefix of the order is kept, and its length is the one of exact masses unless tokens
    within 2^-40 of the border are concerned (the masses' relative error, with a factor of two to spare)."""
    rng = np.random.default_rng(len(what) + V)
    B = 16
    z = (-1.1 * np.log1p(rng.random((B, V)) * V) + rng.standard_normal((B, V))).astype(f32)
    if what == "ties":
        z = (np.round(z * 4) / 4).astype(f32)
    elif what == "coarse":
        z = (np.round(z / 4) * 4).astype(f32)
    elif what == "equal":
        z[:] = f32(-1.5)
    elif what == "masked":
        z[rng.random(z.shape) < 0.98] = -np.inf
    elif what == "flat":
        z[:, V // 16:] = f32(-16.0)
    elif what == "steps":
        z = (z.max(axis=1, keepdims=True) - f32(0.6953125) * rng.integers(0, 20, z.shape)).astype(f32)
    elif what == "both_signs":
        z = (z * rng.choice(f32([1, -1]), z.shape) * f32(0.02)).astype(f32)
    z = to_bf16(z) if dtype == "bf16" else z
    T = rng.choice(f32([0.3, 1.0, 2.0]), B)
    for with_k, with_m in ((False, False), (True, False), (True, True)):
        p = rng.choice(f32([0.1, 0.5, 0.9, 0.99, 0.9999, 1 - 2.0 ** -20, 1 - 2.0 ** -24]), B)
        k = rng.choice(i32([0, 1, 60, V // 3, V - 1]), B) if with_k else np.zeros(B, i32)
        m = rng.choice(f32([0, 1e-6, 0.01]), B) if with_m else np.zeros(B, f32)
        x = torch.from_numpy(z).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        got = sv.spec_logits_truncate(x, dev(T), torch.zeros(B + 1, dtype=torch.int32, device="cuda"), top_p=dev(p), top_k=dev(k),
                                      min_p=dev(m)).float().cpu().numpy()
        for r in range(B):
            order, fewest, most = lengths(z[r], T[r], k[r], p[r], m[r], 2.0 ** -40)
            there = int(np.isfinite(z[r]).sum())
            n = int(np.isfinite(got[r]).sum())
            assert min(fewest, there) <= n <= most, (r, fewest, n, most)
            assert (got[r][order[:n]] == z[r][order[:n]]).all()
