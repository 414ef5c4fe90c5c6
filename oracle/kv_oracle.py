"""Float64 CPU oracle of the paged dense KV cache's operators (test infrastructure only).

Plain NumPy, one token, head and row at a time, from the definitions:
  * norm_rope: y = R(pos) (x / sqrt(mean(x^2) + eps) * w), rotate-half pairs (k, k + d/2);
  * append: rotated keys and values at the slots of the row's pages;
  * attend: softmax over the slots the token sees, its weighted values and its natural log-sum-exp.
Each function is pinned by a CPU test against something other than itself.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.palu_oracle import rope_rotate


def norm_rope(x, w, positions, theta: float, eps: float) -> np.ndarray:
    """x [tokens][heads][d]; w [d] or None; positions [tokens]; theta 0: no rotation."""
    out = np.empty(x.shape, dtype=np.float64)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            y = np.asarray(x[t, h], dtype=np.float64)
            if w is not None:
                y = y / math.sqrt(float(np.sum(y * y)) / y.size + eps) * np.asarray(w, dtype=np.float64)
            out[t, h] = rope_rotate(y, float(positions[t]), theta) if theta > 0 else y
    return out


def slot(page_table, page_size: int, b: int, t: int):
    """(page, offset) of token t of row b; no table: row b is page b."""
    if page_table is None:
        return b, t
    return int(page_table[b][t // page_size]), t % page_size


def row_slots(row_start, kv_len, b: int):
    """(packed token, slot) of row b's new tokens."""
    n = int(row_start[b + 1] - row_start[b])
    return [(int(row_start[b]) + i, int(kv_len[b]) - n + i) for i in range(n)]


def append(pages_k, pages_v, k, v, row_start, kv_len, page_table, *, w=None, positions=None, theta=10000.0,
           eps=1e-6):
    """Writes into pages_k / pages_v [pages][page_size][heads][d] (float64, in place)."""
    ps = pages_k.shape[1]
    for b in range(len(kv_len)):
        for tok, t in row_slots(row_start, kv_len, b):
            if t < 0:
                continue
            pos = t if positions is None else int(positions[tok])
            pg, off = slot(page_table, ps, b, t)
            pages_k[pg, off] = norm_rope(k[tok:tok + 1], w, [pos], theta, eps)[0]
            pages_v[pg, off] = v[tok]


def attend(q, pages_k, pages_v, row_start, kv_len, page_table):
    """Returns (o [tokens][heads][d], lse [tokens][heads], size [tokens][heads][d]) with size = sum p |v|, and the
    largest sum |q_j k_j| / sqrt(d) of any visible pair: what the rounding of a computed o is measured by. Tokens
    of no row stay NaN."""
    n, d = q.shape[1], q.shape[2]
    ps, m = pages_k.shape[1], pages_k.shape[2]
    o = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    size = np.full(q.shape, np.nan)
    reach = 0.0
    for b in range(len(kv_len)):
        L = int(kv_len[b])
        at = [slot(page_table, ps, b, t) for t in range(L)]
        pg, off = np.array([x[0] for x in at], dtype=int), np.array([x[1] for x in at], dtype=int)
        for h in range(m):
            K = np.asarray(pages_k[pg, off, h], dtype=np.float64).reshape(L, d)
            V = np.asarray(pages_v[pg, off, h], dtype=np.float64).reshape(L, d)
            for tok, last in row_slots(row_start, kv_len, b):
                for i in range(h * (n // m), (h + 1) * (n // m)):
                    if last < 0:
                        o[tok, i], size[tok, i], lse[tok, i] = 0.0, 0.0, -math.inf
                        continue
                    x = np.asarray(q[tok, i], dtype=np.float64)
                    s = K[:last + 1] @ x / math.sqrt(d)
                    top = float(s.max())
                    p = np.exp(s - top)
                    tot = float(p.sum())
                    o[tok, i] = p @ V[:last + 1] / tot
                    size[tok, i] = p @ np.abs(V[:last + 1]) / tot
                    lse[tok, i] = top + math.log(tot)
                    reach = max(reach, float((np.abs(K[:last + 1]) @ np.abs(x)).max()) / math.sqrt(d))
    return o, lse, size, reach
