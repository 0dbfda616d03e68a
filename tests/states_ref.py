"""Plain restatements in numpy, in 64 bits, of beam selection, the reordering of
states and the 8-bit cache."""
from __future__ import annotations

import numpy as np


def beam_rows(z, scores, ended=None):
    """Each row's candidates' scores [R, V] (-inf: none; an ended row's all -inf) and its log-sum-exp (NaN: not read)."""
    z = z.astype(np.float64)
    R = len(z)
    out, lse = np.full(z.shape, -np.inf), np.full(R, np.nan)
    for r in range(R):
        if scores[r] == -np.inf or (ended is not None and ended[r]):
            continue
        m = z[r].max()
        if m == -np.inf:
            lse[r] = m
            continue
        if not np.isfinite(m):
            continue
        log_sum = np.log(np.exp(z[r] - m).sum())
        lse[r] = m + log_sum
        out[r] = (np.float64(scores[r]) - log_sum) + (z[r] - m)
    return out, lse


def beam_select(z, scores, offsets, n, ended=None, end_token=0):
    """(scores [B, n] float64, tokens, rows, lse [R], every candidate's score [R, V], z).  Within a row the order is the
    logits', also where scores are so large that 64 bits do not tell them apart."""
    B, V = len(offsets) - 1, z.shape[1]
    every, lse = beam_rows(z, scores, ended)
    os, ot, orow = np.full((B, n), -np.inf), np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32)
    for b in range(B):
        rows = np.arange(offsets[b], offsets[b + 1])
        live = [r for r in rows if scores[r] != -np.inf and not (ended is not None and ended[r])]
        if np.isnan(scores[rows]).any() or (scores[rows] == np.inf).any() or any(np.isnan(z[r]).any() or (z[r] == np.inf).any() for r in live):
            os[b] = np.nan
            continue
        found = []
        for r in rows:
            if scores[r] == -np.inf:
                continue
            if ended is not None and ended[r]:
                found.append((-np.float64(scores[r]), int(r), 0.0, end_token))
                continue
            top = np.lexsort((np.arange(V), -z[r].astype(np.float64)))[:n]
            found += [(-every[r, v], int(r), -float(z[r, v]), int(v)) for v in top if every[r, v] > -np.inf]
        for i, (s, r, _, v) in enumerate(sorted(found)[:n]):
            os[b, i], orow[b, i], ot[b, i] = -s, r, v
    return os, ot, orow, lse, every, z


def reorder(x, rows, offsets, slots=None, lengths=None, position=None):
    """x [S, ..] with the slots in the first dimension (positions in dimension `position`), a new array."""
    out = x.copy()
    slots = np.arange(len(rows)) if slots is None else slots
    for b in range(len(offsets) - 1):
        group = range(offsets[b], offsets[b + 1])
        named = [slots[i] for i in group]
        if len(set(named)) < len(named) or any(not 0 <= s < len(x) for s in named):
            continue
        if any(rows[i] != -1 and rows[i] not in group for i in group):
            continue
        for i in group:
            if rows[i] < 0:
                continue
            source = slots[rows[i]]
            if lengths is None:
                out[slots[i]] = x[source]
            elif position is None:
                if lengths[source] > 0:
                    out[slots[i]] = x[source]
            else:
                part = (slice(None),) * (position - 1) + (slice(0, max(0, lengths[source])),)
                out[slots[i]][part] = x[source][part]
    return out


def to_e4m3(y):
    """The nearest e4m3 values (ties to even) of finite numbers up to 448."""
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(y / step) * step


def quantise(x):
    """x [.., D] -> (values in e4m3 [.., D], NaN for NaN and infinities; exponents + 127 [.., blocks])."""
    x = x.astype(np.float64)
    D = x.shape[-1]
    q, scale = np.empty_like(x), np.empty((*x.shape[:-1], -(-D // 32)), np.uint8)
    for j in range(scale.shape[-1]):
        part = x[..., 32 * j: 32 * j + 32]
        big = np.where(np.isfinite(part), np.abs(part), 0).max(-1)
        f, p = np.frexp(big)  # big = (2 f) 2^(p - 1)
        e = np.where(big > 0, np.maximum(p - 1 - 8 + (2 * f > 1.75), -127), -127)
        with np.errstate(invalid="ignore"):
            y = np.where(np.isfinite(part), part, 0) * np.ldexp(1.0, -e)[..., None]
        q[..., 32 * j: 32 * j + 32] = np.where(np.isfinite(part), to_e4m3(y), np.nan)
        scale[..., j] = e + 127
    return q, scale


def dequantise(q, scale):
    D = q.shape[-1]
    return q.astype(np.float64) * np.repeat(np.ldexp(1.0, scale.astype(np.int64) - 127), 32, -1)[..., :D]


class Cache:
    """[L, P, T, H, D] values in e4m3 and their scales' bytes, as float64 and uint8."""

    def __init__(self, q, scale, lengths, pages=None):
        self.q, self.scale, self.lengths, self.pages = q.copy(), scale.copy(), lengths.copy(), pages

    def entry(self, slot, p):
        """(page, place), None where there is none."""
        T = self.q.shape[2]
        if self.pages is None:
            return (slot, p) if p < T else None
        if p >= self.pages.shape[1] * T:
            return None
        page = self.pages[slot, p // T]
        return (page, p % T) if 0 <= page < self.q.shape[1] else None

    def write(self, x, paths, slots):
        """x [L, R, H, D]; paths: the kept rows of each sequence, None for one that is skipped."""
        after = self.lengths.copy()
        for b, path in enumerate(paths):
            if path is None or not 0 <= slots[b] < len(self.lengths) or self.lengths[slots[b]] < 0:
                continue
            room = True
            for i, r in enumerate(path):
                at = self.entry(slots[b], self.lengths[slots[b]] + i)
                if at is None:
                    room = False
                    continue
                self.q[:, at[0], at[1]], self.scale[:, at[0], at[1]] = quantise(x[:, r])
            after[slots[b]] = self.lengths[slots[b]] + len(path) if room else -1
        self.after = after

    def read(self, offsets, R, slots, first=None):
        """[L, R, H, D], NaN where nothing is held; rows behind the last sequence's are 0."""
        L, _, _, H, D = self.q.shape
        out = np.zeros((L, R, H, D))
        for b in range(len(offsets) - 1):
            for r in range(offsets[b], offsets[b + 1]):
                p = r - offsets[b] + (0 if first is None else first[b])
                held = 0 <= slots[b] < len(self.lengths) and 0 <= p < self.lengths[slots[b]]
                at = self.entry(slots[b], p) if held else None
                out[:, r] = np.nan if at is None else dequantise(self.q[:, at[0], at[1]], self.scale[:, at[0], at[1]])
        return out


def tree_path(parent, o, nodes, last, n):
    """The n + 1 nodes from the root o to last, None if they are none."""
    path, node = [], last
    if not o <= last < o + nodes or not 0 <= n < nodes:
        return None
    while node != o:
        path.insert(0, node)
        if not o <= parent[node] < node:
            return None
        node = parent[node]
    path.insert(0, o)
    return path if len(path) == n + 1 else None
