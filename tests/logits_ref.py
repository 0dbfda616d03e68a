"""Plain restatements of the logit operators (spec_logits_*, spec_penalty_*),
row by row in numpy, for the tests: the processing both in the definition's
fp32 steps (the kernels have to give these bits) and in 64 bits with the
bound that those steps allow, the truncation by a full sort in 64 bits."""
from __future__ import annotations

import dataclasses

import numpy as np

F32, BF16 = "fp32", "bf16"


def to_bf16(x):
    """fp32 values rounded to the nearest bf16 (ties to even), as fp32 values."""
    u = np.asarray(x, np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    r = np.where(np.isnan(x), np.uint32(0x7FC00000), r)
    return r.view(np.float32)


def pack(bits):
    """[.., V] truth values -> int32 words, bit v % 32 of word v // 32."""
    V = bits.shape[-1]
    b = np.zeros((*bits.shape[:-1], -(-V // 32) * 32), np.uint8)
    b[..., :V] = bits
    return np.packbits(b, axis=-1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def unpack(words, V):
    return np.unpackbits(np.ascontiguousarray(words).view(np.uint8), axis=-1, bitorder="little")[..., :V].astype(bool)


@dataclasses.dataclass
class Rows:
    """Which rows a call has: for each, its sequence and the drafted tokens it follows."""
    mode: str
    offsets: np.ndarray
    tokens: np.ndarray
    parent: np.ndarray | None = None

    @property
    def B(self):
        return len(self.offsets) - 1

    def __iter__(self):
        o = self.offsets
        for b in range(self.B):
            t = self.tokens[o[b]:o[b + 1]]
            if self.mode == "target":
                yield from ((b, t[:i]) for i in range(len(t) + 1))
            elif self.mode == "draft":
                yield from ((b, t[:i]) for i in range(len(t)))
            elif self.mode == "next":
                yield b, t
            else:
                for g in range(o[b], o[b + 1]):
                    path, u = [], g
                    while self.parent[u] >= 0:
                        path.append(self.tokens[u])
                        u = self.parent[u]
                    yield b, np.array(path, np.int64)

    def count(self):
        return sum(1 for _ in self)


def process(z, rows: Rows, p, dtype):
    """p: a dict of the operator's arguments as numpy arrays (any may be
    missing).  Returns (the definition's fp32 steps rounded to dtype, the same
    in 64 bits, the bound of the difference)."""
    V = z.shape[1]
    f32 = np.float32
    out, ref, tol = z.copy(), z.astype(np.float64), np.zeros(z.shape)
    half = 2.0 ** -24
    for r, (b, path) in enumerate(rows):
        y, y64, e, touched = z[r].astype(f32), z[r].astype(np.float64), np.zeros(V), np.zeros(V, bool)
        if "counts" in p:
            s = p["slots"][b] if "slots" in p else b
            c = p["counts"][s].astype(np.int64) + np.bincount(np.asarray(path, np.int64), minlength=V)
            seen = (c > 0) | unpack(p["seen"][s, 0], V)
            rho, phi, pi = (p[n][b] if n in p else f32(d) for n, d in (("repetition", 1), ("frequency", 0), ("presence", 0)))
            with np.errstate(all="ignore"):
                t = np.where(y > 0, y / rho, y * rho).astype(f32)
                t = (t - phi * c.astype(f32)).astype(f32)
                t = np.where(c > 0, t - pi, t).astype(f32)
                y = np.where(seen, t, y)
                a = np.where(y64 > 0, y64 / float(rho), y64 * float(rho))
                a1 = a - float(phi) * c
                a2 = a1 - float(pi) * (c > 0)
                e = np.where(seen, half * (abs(a) + abs(float(phi) * c) + abs(a1) + abs(a2)), 0)
                y64 = np.where(seen, a2, y64)
                touched |= seen
        if "bias_offsets" in p:
            total, total64, has = np.zeros(V, f32), np.zeros(V), np.zeros(V, bool)
            for k in range(p["bias_offsets"][b], p["bias_offsets"][b + 1]):
                t, v = p["bias_tokens"][k], p["bias_values"][k]
                total[t] = f32(total[t] + v) if has[t] else v
                total64[t] += float(v)
                e[t] += half * abs(total64[t]) if has[t] else 0
                has[t] = True
            with np.errstate(all="ignore"):
                y = np.where(has, y + total, y)
                y64 = np.where(has, y64 + total64, y64)
                e = np.where(has, e + half * abs(y64), e)
                touched |= has
        if "mask" in p:
            m = p["mask_rows"][r] if "mask_rows" in p else r
            if m >= 0:
                ok = unpack(p["mask"][m], V)
                y, y64, touched = np.where(ok, y, f32(-np.inf)), np.where(ok, y64, -np.inf), touched & ok
        out[r] = to_bf16(y) if dtype == BF16 else y
        ref[r] = y64
        # Rounding to the output type: at most half a step, relative to the value.
        # Below the smallest normal number a rounding is off by up to half the
        # smallest subnormal instead, whatever the value: 2^-150 for each of the
        # at most 4 + entries fp32 steps, 2^-134 for the one to bf16.
        steps = 4 + (p["bias_offsets"][b + 1] - p["bias_offsets"][b] if "bias_offsets" in p else 0)
        with np.errstate(all="ignore"):
            e = e + steps * 2.0 ** -150
            tol[r] = np.where(touched, e + ((abs(y64) + e) * 2.0 ** -8 + 2.0 ** -134 if dtype == BF16 else 0), 0)
    return out, ref, tol


def truncate(z, seq, T, top_k=None, top_p=None, min_p=None):
    """Rows z [R, V] of sequences seq [R].  Returns (rows with -inf outside
    the kept set, margin [R]: how near a row's top-p border is to another
    answer, relative to Z; inf where there is none)."""
    out, margin = z.copy(), np.full(len(z), np.inf)
    V = z.shape[1]
    for r, b in enumerate(seq):
        row = z[r]
        if T[b] == 0 or np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
            continue
        order = np.lexsort((np.arange(V), -row.astype(np.float64)))
        s = row[order].astype(np.float64)
        x = (s - s[0]) / float(T[b])
        keep = np.ones(V, bool)
        if top_k is not None and top_k[b] > 0:
            keep &= np.arange(V) < top_k[b]
        if top_p is not None and top_p[b] < 1:
            w = np.where(keep, np.exp(x), 0).astype(np.longdouble)
            before = np.concatenate([[0], np.cumsum(w)[:-1]])
            Z = w.sum()
            border = np.longdouble(float(top_p[b])) * Z
            # the last token that has weight at all ends the order for this purpose
            margin[r] = float(np.min(abs(before[w > 0] - border)) / Z)
            keep &= before < border
        if min_p is not None and min_p[b] > 0:
            keep &= x >= np.log(float(min_p[b]))
        out[r, order[~keep]] = -np.inf
    return out, margin


def row_sequences(rows: Rows):
    return np.array([b for b, _ in rows], np.int64)
