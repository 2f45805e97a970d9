"""float64 oracle of the 8-bit paged attention cache: what is stored, attention over it, and the pages.

Written to be read, in plain numpy loops over sequences, heads and blocks; it shares no code with the GPU
library.  A cache is modelled by what a user sees of it: the stored values of each sequence (codes times
2^e, kept as float64) with the exponent of each block of 32 tokens and head, the table and the counts.
"""

from __future__ import annotations

import math

import numpy as np

KV_BLOCK = 32
KV_TOP = {"e4m3": 448.0, "int8": 127.0}
KV_MAX = {"f16": 65504.0, "bf16": float((2 - 2.0 ** -7) * 2.0 ** 127)}


def kv_exponent(amax: float, code: str) -> int:
    """The smallest integer e with amax <= TOP * 2^e, kept in [-126, 127]; -126 for 0."""
    if amax == 0:
        return -126
    e = math.floor(math.log2(amax / KV_TOP[code])) - 1
    while amax > math.ldexp(KV_TOP[code], e):
        e += 1
    return min(max(e, -126), 127)


def kv_round(x: np.ndarray, e: int, code: str) -> np.ndarray:
    """x rounded to nearest even on the grid of the code at exponent e (float64 values)."""
    y = np.ldexp(np.asarray(x, dtype=np.float64), -e)
    if code == "int8":
        return np.ldexp(np.rint(y), e)
    _, ex = np.frexp(y)                                   # |y| in [2^(ex-1), 2^ex)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)      # e4m3: 3 bits of mantissa, normal from 2^-6
    return np.ldexp(np.rint(y / step) * step, e)


def kv_clean(x: np.ndarray, act: str) -> np.ndarray:
    """Inputs as they are stored: infinities saturate, NaN becomes zero."""
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isnan(x), 0.0, np.clip(x, -KV_MAX[act], KV_MAX[act]))


class KvModel:
    """The stored tokens [len][kv_heads][dim] of one sequence of K (or of V)."""

    def __init__(self, kv_heads: int, dim: int, code: str, act: str):
        self.code, self.act = code, act
        self.values = np.zeros((0, kv_heads, dim))
        self.exps: list[list[int]] = []                   # [block][head]

    def append(self, x: np.ndarray) -> None:
        """Store tokens that come in one call."""
        x = kv_clean(x, self.act)
        before = self.values.shape[0]
        both = np.concatenate([self.values, x])
        for b in range(before // KV_BLOCK, -(-both.shape[0] // KV_BLOCK)):
            lo, hi = b * KV_BLOCK, min((b + 1) * KV_BLOCK, both.shape[0])
            if hi <= before:
                continue
            if b == len(self.exps):
                self.exps.append([-126] * x.shape[1])
            for h in range(x.shape[1]):
                fresh = both[max(lo, before):hi, h]
                e = kv_exponent(float(np.abs(fresh).max()), self.code)
                if lo < before:
                    e = max(e, self.exps[b][h])
                self.exps[b][h] = e
                both[lo:hi, h] = kv_round(both[lo:hi, h], e, self.code)
        self.values = both


def kv_visible(p: int, length: int, window: int, sinks: int) -> np.ndarray:
    """Which of `length` tokens the row at position p sees."""
    u = np.arange(length)
    seen = u <= p
    if window:
        seen &= (u > p - window) | (u < sinks)
    return seen


def kv_attend(q, k, v, window=0, sinks=0, scale=None):
    """Rows q [count][heads][dim], the last of the tokens k and v [len][kv_heads][dim]: out, lse, and for error
    bounds mass = sum p |v| per element and reach = max over seen tokens of scale * sum |q k| per row."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    count, heads, dim = q.shape
    length, kvh, _ = k.shape
    scale = dim ** -0.5 if scale is None else scale
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((count, heads), -np.inf), np.zeros((count, heads))
    for j in range(count):
        seen = kv_visible(length - count + j, length, window, sinks)
        if not seen.any():
            continue
        for h in range(heads):
            a = h // (heads // kvh)
            x = scale * (k[seen, a] @ q[j, h])
            top = x.max()
            w = np.exp(x - top)
            total = w.sum()
            lse[j, h] = top + np.log(total)
            out[j, h] = w @ v[seen, a] / total
            mass[j, h] = w @ np.abs(v[seen, a]) / total
            reach[j, h] = scale * (np.abs(k[seen, a]) @ np.abs(q[j, h])).max()
    return out, lse, mass, reach


# ---- pages: lists and integers, as pi_kv.h states them ---------------------------------------------------


def kv_free(table, lens, refs, seqs):
    for s in seqs:
        for j, p in enumerate(table[s]):
            if p >= 0:
                refs[p] -= 1
            table[s][j] = -1
        lens[s] = 0


def kv_fork(table, lens, refs, src, dst):
    for a, b in zip(src, dst):
        table[b] = list(table[a])
        lens[b] = lens[a]
        for p in table[b]:
            if p >= 0:
                refs[p] += 1


def kv_reserve(table, lens, refs, seqs, counts, page):
    """Returns the copies [(from, to)] and how many sequences could not grow."""
    free = [p for p, r in enumerate(refs) if r <= 0]
    width = len(table[0])
    copies, failed, full, taken, dropped = [], 0, False, 0, []
    for s, c in zip(seqs, counts):
        end = lens[s] + c
        if c < 0 or end > width * page:
            failed += 1
            continue
        have, want = -(-lens[s] // page), -(-end // page)
        last = table[s][have - 1] if lens[s] % page else -1
        shared = c > 0 and last >= 0 and refs[last] > 1
        # columns past the length that still name a page: its own stays, a shared one is let go
        fill = [j for j in range(have, want) if table[s][j] < 0 or refs[table[s][j]] != 1]
        need = len(fill) + (1 if shared else 0)
        if full or taken + need > len(free):
            full = True
            failed += 1
            continue
        mine = free[taken:taken + need]
        taken += need
        if shared:
            copies.append((last, mine[0]))
            dropped.append(last)
            table[s][have - 1] = mine.pop(0)
        for j, p in zip(fill, mine):
            if table[s][j] >= 0 and refs[table[s][j]] > 1:
                dropped.append(table[s][j])
            table[s][j] = p
        lens[s] = end
    for p in free[:taken]:
        refs[p] = 1
    for p in dropped:
        refs[p] -= 1
    return copies, failed


def kv_compact(table, refs):
    """Returns the copies [(from, to)]."""
    live = sum(r > 0 for r in refs)
    holes = [p for p in range(live) if refs[p] <= 0]
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    where = dict(zip(movers, holes))
    for a, b in where.items():
        refs[b], refs[a] = refs[a], 0
    for row in table:
        for j, p in enumerate(row):
            row[j] = where.get(p, p)
    return list(where.items())
