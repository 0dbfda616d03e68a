"""What a selection of beams has to be, from the definition: scores in exact
rational arithmetic on log-sums in 64 bits, and what its float32 results may be off by."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

U = 2.0 ** -24
# A row's log-sum-exp, of float32 terms, in units of U, half a step of float32: a term's argument is off by its three
# roundings (under 51 on average over the distribution, for 2^24 tokens), the exponential by 4; a sum of at most 16 additions per
# term by 16; the factor that brings a piece's sum to the row's largest logit by 51 + 4 + 1.
TOL = 128 * U
LOWEST = float(np.finfo(np.float32).min)


class Row:
    """A row's candidates: how many, the first n in the order of the row, and each one's score."""

    def __init__(self, z, score, ended, end_token, n):
        self.score, self.ended, self.z, self.end_token = Fraction(0), ended, z, end_token
        self.bad = bool(np.isnan(score) or score == np.inf)
        self.lse, self.order, self.count = np.nan, [], 0
        if score == -np.inf or self.bad:
            return
        self.score = Fraction(float(score))
        if ended:
            self.order, self.count = [end_token], 1
            return
        z64 = z.astype(np.float64)
        top = z64.max()
        if not top < np.inf:
            self.bad = True
            return
        self.lse = top
        if top == -np.inf:
            return
        log_sum = np.log(np.exp(z64 - top).sum())
        self.lse = top + log_sum
        self.base = self.score - Fraction(float(top)) - Fraction(float(log_sum))
        self.count = int((z > -np.inf).sum())
        some = np.arange(len(z)) if len(z) <= n else np.flatnonzero(z >= np.partition(z, len(z) - n)[len(z) - n])
        some = some[z[some] > -np.inf]
        self.order = [int(v) for v in some[np.lexsort((some, -z[some].astype(np.float64)))][:n]]

    def of(self, token):
        return self.score if self.ended else self.base + Fraction(float(self.z[token]))


def check(got, z, scores, offsets, n, ended=None, end_token=0):
    """z, scores: the values that the kernel saw, as float32 arrays; got: what it returned, the log-sum-exps last."""
    s, t, r, lse = (x.cpu().numpy() for x in got)
    for b in range(len(offsets) - 1):
        group = range(offsets[b], offsets[b + 1])
        rows = {i: Row(z[i], scores[i], bool(ended is not None and ended[i]), end_token, n) for i in group}
        for i in group:
            if np.isfinite(rows[i].lse):
                assert abs(lse[i] - rows[i].lse) <= TOL + U * abs(rows[i].lse), (b, i)
            elif not rows[i].bad:
                assert lse[i] == rows[i].lse or (np.isnan(lse[i]) and np.isnan(rows[i].lse)), (b, i)
        if any(row.bad for row in rows.values()):
            assert np.isnan(s[b]).all() and (t[b] == -1).all() and (r[b] == -1).all(), b
            continue
        found = min(n, sum(row.count for row in rows.values()))
        assert (s[b, found:] == -np.inf).all() and (t[b, found:] == -1).all() and (r[b, found:] == -1).all(), b
        taken, exact = {i: 0 for i in group}, []
        for k in range(found):
            i, token = int(r[b, k]), int(t[b, k])
            # within a row: its candidates in its own order, none left out
            assert i in rows and taken[i] < len(rows[i].order) and rows[i].order[taken[i]] == token, (b, k, i, token)
            taken[i] += 1
            exact.append(rows[i].of(token))
            want = max(float(exact[-1]), LOWEST)
            assert abs(float(s[b, k]) - want) <= TOL + U * abs(want), (b, k, s[b, k], want)
        # between rows: what comes later, or does not come, is not better by more than the two rows' sums may be off by
        # and the 48 bits that scores are compared in
        room = lambda x: Fraction(2 * TOL) + abs(x) * Fraction(2.0 ** -46)  # noqa: E731
        for x, y in zip(exact, exact[1:]):
            assert y - x <= room(x), (b, float(x), float(y))
        for i in group:
            if exact and taken[i] < len(rows[i].order):
                assert rows[i].of(rows[i].order[taken[i]]) - exact[-1] <= room(exact[-1]), (b, i)
