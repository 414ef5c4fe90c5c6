"""Shared helpers of the paged KV cache's GPU tests: seeded batches on the GPU and for the oracle, and the bounds
their outputs are held to.

Bounds, from the arithmetic. u = finfo(dtype).eps / 2 is the relative error of one rounding (0 for the fp32 path's
own term below), tiny = half the smallest subnormal step.
  * norm_rope / append: y is computed in fp32 and rounded once: |err| <= u |y| + tiny + 2^-20 (|a| + |b|), a and b
    being the normed pair. The last term covers the norm's sum of at most 128 squares and its root (relative 2^-21),
    the sine and cosine of a phase rounded to 24 bits (absolute 2^-22) and the rotation's two products.
  * attend: out is a sum p v / l of weights rounded to dtype, rounded once: |err| <= u |o| + (u + 2 e + 2^-20) A +
    T t max|v| + tiny, with A = sum p |v| / l, e the error of a score (a sum of d products accumulated in fp32,
    d <= 128, truncating at worst: 2^-16 of sum |q_j k_j| / sqrt(d), and 2^-20 for the exponential), and t = 2^-25
    for fp16, whose weights below 2^-14 keep only that absolute precision (bf16: none).
  * lse: e + 2^-20 (1 + |lse|).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv_oracle as KO

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ulp(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def tiny(dtype):
    f = torch.finfo(TYPES[dtype])
    return f.smallest_normal * f.eps / 2


def rounded(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dtype])


def check_rotated(got, ref, amplitude, dtype):
    """amplitude: |a| + |b| of each element's normed pair."""
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref)
    tol = ulp(dtype) * np.abs(ref) + tiny(dtype) + 2.0 ** -20 * amplitude
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3f} of the bound"


def pair_amplitude(x):
    h = x.shape[-1] // 2
    a = np.abs(x[..., :h]) + np.abs(x[..., h:])
    return np.concatenate([a, a], -1)


class Batch:
    """Rows of new tokens over paged caches, with every slot that no row may read set to NaN."""

    def __init__(self, *, n, m, d, dtype, news, lens, page, table=True, seed=0, q_scale=1.0, slack=2, extra_tokens=0,
                 max_new=None, max_kv=None):
        from rank_kv_cache_gb300 import palu as P
        rng = np.random.default_rng(seed)
        self.n, self.m, self.d, self.dtype, self.news, self.lens, self.page = n, m, d, dtype, news, lens, page
        B, top = len(news), max(max(lens), 1)
        per = -(-top // page) if table else 1
        assert table or page >= top
        pages = B * per + (slack if table else 0)
        self.row_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.N = int(self.row_start[-1]) + extra_tokens
        self.table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32) if table else None
        self.q = rounded(rng, (self.N, n, d), dtype, q_scale)
        gen = torch.Generator().manual_seed(seed)
        shape = (pages, page, m, d)
        self.pk, self.pv = (torch.randn(shape, generator=gen).to(TYPES[dtype]) for _ in range(2))
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, L in enumerate(lens):
            t = np.arange(L)
            pg = self.table[b][t // page] if table else np.full(L, b)
            used[torch.from_numpy(pg).long(), torch.from_numpy(t % page).long()] = True
        self.pk[~used] = float("nan")
        self.pv[~used] = float("inf")
        dev = torch.device("cuda:0")
        self.dev = dev
        self.layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, max_batch=B,
                                      max_tokens=max(self.N, 1))
        self.pages = P.KVPages(self.pk.to(dev), self.pv.to(dev))
        self.rows = P.KVRows(torch.from_numpy(self.row_start).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                             page_table=None if self.table is None else torch.from_numpy(self.table).to(dev),
                             n_tokens=self.N, max_new=max(news) if max_new is None else max_new,
                             max_kv_len=top if max_kv is None else max_kv)
        self.qd = self.q.to(dev)

    def attend(self, **kw):
        out = torch.full((self.N, self.n, self.d), 7.0, dtype=TYPES[self.dtype], device=self.dev)
        lse = torch.full((self.N, self.n), 7.0, dtype=torch.float32, device=self.dev)
        self.layer.attend(self.pages, self.rows, self.qd, out=out, lse=lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def bounds(self, o, size, lse, reach, vmax, T):
        u = ulp(self.dtype)
        e = 2.0 ** -16 * reach + 2.0 ** -20
        t = 2.0 ** -25 if self.dtype == "f16" else 0.0
        return (u * np.abs(o) + (u + 2 * e + 2.0 ** -20) * size + T * t * vmax + tiny(self.dtype),
                e + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0))))

    def check(self, out, lse, ref):
        o, s, size, reach = ref
        mine = ~np.isnan(s[:, 0])
        got, got_s = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(got[~mine] == 7.0) and np.all(got_s[~mine] == 7.0), "tokens of no row were written"
        v = self.pv.double().numpy()
        vmax = float(np.abs(v[np.isfinite(v)]).max()) if np.isfinite(v).any() else 0.0
        tol, tol_s = self.bounds(o, size, s, reach, vmax, max(self.lens))
        assert np.all(np.isfinite(got[mine]))
        err = np.abs(got - o)[mine]
        assert np.all(err <= tol[mine]), f"out: worst {np.max(err / tol[mine]):.3f} of the bound"
        inf = mine[:, None] & np.isneginf(s)
        assert np.all(np.isneginf(got_s[inf]))
        fin = mine[:, None] & np.isfinite(s)
        err = np.abs(got_s[fin] - s[fin])
        if err.size:
            assert np.all(err <= tol_s[fin]), f"lse: worst {np.max(err / tol_s[fin]):.3f} of the bound"

    def run_and_check(self):
        out, lse = self.attend()
        self.layer.check_device()
        self.check(out, lse, self.oracle())
        return out, lse

    def oracle(self):
        return KO.attend(self.q.double().numpy(), self.pk.double().numpy(), self.pv.double().numpy(), self.row_start,
                         self.lens, self.table)

    def sampled(self, tokens, heads):
        """The oracle at some tokens and heads of the batch, in float64 torch; the other tokens are NaN."""
        d, g = self.d, self.n // self.m
        o = np.full((self.N, self.n, d), np.nan)
        size, lse = o.copy(), np.full((self.N, self.n), np.nan)
        reach = 0.0
        for b, L in enumerate(self.lens):
            t = np.arange(L)
            pg = self.table[b][t // self.page] if self.table is not None else np.full(L, b)
            idx = torch.from_numpy(pg.astype(np.int64)) * self.page + torch.from_numpy(t % self.page)
            for i in heads:
                K = self.pk.flatten(0, 1)[idx, i // g].double()
                V = self.pv.flatten(0, 1)[idx, i // g].double()
                for tok in tokens:
                    if not self.row_start[b] <= tok < self.row_start[b + 1]:
                        continue
                    seen = L - self.news[b] + tok - int(self.row_start[b]) + 1
                    x = K[:seen] @ self.q[tok, i].double() / d ** 0.5
                    p = torch.softmax(x, 0)
                    o[tok, i], size[tok, i] = p @ V[:seen], p @ V[:seen].abs()
                    lse[tok, i] = torch.logsumexp(x, 0)
                    reach = max(reach, float((K[:seen].abs() @ self.q[tok, i].double().abs()).max()) / d ** 0.5)
        return o, lse, size, reach

    def check_sampled(self, out, lse, tokens, heads):
        o, s, size, reach = self.sampled(tokens, heads)
        vmax = 8.0
        tol, tol_s = self.bounds(o, size, s, reach, vmax, max(self.lens))
        got, got_s = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(np.isfinite(got[:int(self.row_start[-1])]))
        at = ~np.isnan(s)
        assert at.any()
        assert np.all(np.abs(got - o)[at] <= tol[at]), np.max(np.abs(got - o)[at] / tol[at])
        assert np.all(np.abs(got_s - s)[at] <= tol_s[at]), np.max(np.abs(got_s - s)[at] / tol_s[at])
