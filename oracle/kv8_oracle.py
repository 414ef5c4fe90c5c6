"""Float64 CPU oracle of the 8-bit paged KV cache and of the steps around it (test infrastructure only).

Plain NumPy and Python, from the definitions:
  * e4m3 codes: 1 sign, 4 exponent (bias 7) and 3 mantissa bits, no infinities, 0x7f and 0xff NaN;
  * append: the rotated keys and the values of a block of 16 slots and head under one power of two;
  * attend: the dense oracle's, over codes times scales;
  * plan: rows admitted one after the other, pages from the front of a queue and back to its end;
  * verify: one draft after the other, and a running sum.
Each function is pinned by a CPU test against something other than itself.
"""
from __future__ import annotations

from collections import deque
from fractions import Fraction

import numpy as np

from oracle import kv_oracle as KO

BLOCK = 16
TOP = 448.0


def decode(codes) -> np.ndarray:
    """Values of uint8 codes."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag)


VALUES = decode(np.arange(127))                          # of the codes without sign, ascending


def encode(x) -> np.ndarray:
    """Codes of the nearest values, ties to the even code, past 448 the largest; NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), TOP)
    hi = np.minimum(np.searchsorted(VALUES, np.nan_to_num(mag)), 126)
    lo = np.maximum(hi - 1, 0)
    up = VALUES[hi] - mag
    down = mag - VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return np.where(np.signbit(x) & ~np.isnan(x), code | 128, code).astype(np.uint8)


def scale_for(top: float) -> float:
    """The least 2^k, k from -64 to 64, that brings top to 448 or below."""
    k = -64
    while k < 64 and top > TOP * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(codes, scales, x, row_start, kv_len, page_table):
    """Writes x [tokens][heads][d] (float64, already normed and rotated) into codes [pages][page][heads][d] and scales
    [pages][page / 16][heads], in place."""
    ps = codes.shape[1]
    for b in range(len(kv_len)):
        new = [(tok, t) for tok, t in KO.row_slots(row_start, kv_len, b) if t >= 0]
        for block in sorted({t // BLOCK for _, t in new}):
            mine = [(tok, t) for tok, t in new if t // BLOCK == block]
            older = mine[0][1] - block * BLOCK
            pg, off = KO.slot(page_table, ps, b, block * BLOCK)
            for h in range(codes.shape[2]):
                s = scale_for(max(float(np.abs(x[tok, h]).max()) for tok, _ in mine))
                if older:
                    was = float(scales[pg, off // BLOCK, h])
                    if s > was:
                        codes[pg, off:off + older, h] = encode(decode(codes[pg, off:off + older, h]) * (was / s))
                    s = max(s, was)
                scales[pg, off // BLOCK, h] = s
                for tok, t in mine:
                    codes[pg, off + t - block * BLOCK, h] = encode(x[tok, h] / s)


def values(codes, scales) -> np.ndarray:
    """[pages][page][heads][d] float64."""
    return decode(codes) * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)[..., None]


def plan(new, kv_len, held, table, ring, state, page_size, n_tokens):
    """(row_start, kv_len, held, state, positions, slots, table, ring) behind the step."""
    table, ring, state = np.array(table), np.array(ring), [int(x) for x in state]
    n_pages, per = len(ring), table.shape[1]
    back = sum(int(h) for n, h in zip(new, held) if n < 0 and 0 <= h <= per)
    whole = 0 <= state[0] < n_pages and state[1] >= 0 and state[1] + back <= n_pages   # else the ring is left as it is
    free = deque(int(ring[(state[0] + i) % n_pages]) for i in range(state[1] if whole else 0))
    given, start, lens, hold, pos, slots, shut = [], [0], [], [], [], [], False
    for b, n in enumerate(new):
        L, have = int(kv_len[b]), int(held[b])
        if n < 0 and not (whole and 0 <= have <= per):
            n = 0
        if n < 0:
            given += [int(p) for p in table[b, :have]]
            L = have = n = 0
        need = max(0, -(-(L + n) // page_size) - have) if n > 0 else 0
        # the free pages that the rows ahead left, and the packed places
        if shut or need > len(free) or start[-1] + n > n_tokens:
            shut, n, need = True, 0, 0
        for i in range(need):
            table[b, have + i] = free.popleft()
        for t in range(L, L + n):
            pos.append(t)
            slots.append(int(table[b, t // page_size]) * page_size + t % page_size)
        start.append(start[-1] + n)
        lens.append(L + n)
        hold.append(have + need)
    end = state[0] + state[1]
    for i, p in enumerate(given):
        ring[(end + i) % n_pages] = p
    rest = n_tokens - len(pos)
    head = (state[0] + state[1] - len(free)) % n_pages
    state = [head, len(free) + len(given)] if whole else state
    return start, lens, hold, state, pos + [0] * rest, slots + [-1] * rest, table, ring


def verify(target, draft, draft_tokens, uniforms):
    """One request: target [n][vocab], draft [n - 1][vocab] or None, draft_tokens [n - 1], uniforms [n]: the drafts' and, last,
    the drawn token's. (accepted drafts, the drawn token or -1). Exact: rational numbers."""
    def prob(x):
        x = float(x)
        return Fraction(x) if x > 0 else Fraction(0)

    def uniform(x):                                      # the ends of [0, 1) in fp32
        x = float(x)
        return Fraction(max(x, 0.0)) if x < 1 else 1 - Fraction(1, 2 ** 24)

    n = len(target)
    a = 0
    while a < n - 1:
        x = int(draft_tokens[a])
        if not 0 <= x < len(target[a]):
            break
        q = Fraction(1) if draft is None else prob(draft[a][x])
        if not uniform(uniforms[a]) * q < prob(target[a][x]):
            break
        a += 1
    w = [prob(p) for p in target[a]]
    if a < n - 1:
        if draft is None:
            less = [Fraction(0) if v == int(draft_tokens[a]) else p for v, p in enumerate(w)]
        else:
            less = [max(p - prob(q), Fraction(0)) for p, q in zip(w, draft[a])]
        if sum(less) > 0:
            w = less
    total, run = sum(w), Fraction(0)
    for v, p in enumerate(w):
        run += p
        if run > uniform(uniforms[-1]) * total:
            return a, v
    return a, -1
