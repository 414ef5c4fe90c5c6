"""Shared helpers of the 8-bit paged KV cache's GPU tests: seeded batches, and the bounds their outputs are held to.

Bounds of the attention, from the arithmetic. u = finfo(out).eps / 2 and tiny = half the least subnormal step of the output.
  * A score x is a sum of d products accumulated in fp32 (truncating at worst: 2^-16 of sum |q_j k_j| / sqrt(d), as in
    the dense tests), times a scale; y = x + log2 s_v adds 2^-22 (1 + |log2 s_v|) for the logarithm and its sum (of
    bf16 queries 2^-39 of the row's largest is lost to fp16, far below the first term); an exponential 2^-20. Together e.
  * The weights 2^y are rounded to fp16, 2^-11 of themselves, and 2^-25 absolutely where they fall below 2^-14: the
    largest is at least 2^7, so T tokens lose at most T 2^-32 max(s_v) 448 of the output.
  * out: u |o| + (2^-11 + 2 e + 2^-19) A + T 2^-32 max(s_v) 448 + tiny, with A = sum p |v| / l. lse: e + 2^-20 (1 + |lse|).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv8_oracle as K8
from oracle import kv_oracle as KO
from tests.kv_cases import TYPES, Batch, check_rotated, pair_amplitude, rounded, tiny, ulp


def codes_tensor(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn)


class Batch8(Batch):
    """Rows of new tokens over 8-bit caches, with every code that no row may use NaN, and every scale infinite."""

    def __init__(self, *, n, m, d, dtype, news, lens, page, table=True, seed=0, q_scale=1.0, slack=2, extra_tokens=0,
                 max_new=None, max_kv=None, spread=1.0, pow2=True, flags=0, k_scale=1.0):
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
        blocks = (pages, page // 16, m)
        self.codes, self.scales = [], []
        for size in (k_scale, 1.0):
            x = rng.standard_normal((pages, page, m, d)).astype(np.float32) * size
            s = 2.0 ** np.round(rng.normal(-7, spread, blocks)) * size
            if not pow2:
                s = s * rng.uniform(0.6, 1.9, blocks)
            s = s.astype(np.float32)
            c = torch.from_numpy(x / np.repeat(s.astype(np.float64), 16, 1)[..., None])
            self.codes.append(c.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy())
            self.scales.append(s)
        used = np.zeros((pages, page), dtype=bool)
        for b, L in enumerate(lens):
            t = np.arange(L)
            used[self.table[b][t // page] if table else np.full(L, b), t % page] = True
        some = used.reshape(pages, page // 16, 16).any(-1)
        for c, s in zip(self.codes, self.scales):
            c[~used] = 0x7f
            s[~some] = np.inf
        self.pk, self.pv = (torch.from_numpy(K8.values(c, s)) for c, s in zip(self.codes, self.scales))
        dev = torch.device("cuda:0")
        self.dev = dev
        self.layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, max_batch=B,
                                      max_tokens=max(self.N, 1), flags=flags)
        self.pages = P.KVPages8(*(codes_tensor(c).to(dev) for c in self.codes),
                                *(torch.from_numpy(s).to(dev) for s in self.scales))
        self.rows = P.KVRows(torch.from_numpy(self.row_start).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                             page_table=None if self.table is None else torch.from_numpy(self.table).to(dev),
                             n_tokens=self.N, max_new=max(news) if max_new is None else max_new,
                             max_kv_len=top if max_kv is None else max_kv)
        self.qd = self.q.to(dev)

    def renew(self):
        """The pages and their float64 values from codes and scales that a test has changed."""
        for t, c in ((self.pages.k, self.codes[0]), (self.pages.v, self.codes[1])):
            t.view(torch.uint8).copy_(torch.from_numpy(c))
        self.pages.k_scale.copy_(torch.from_numpy(self.scales[0]))
        self.pages.v_scale.copy_(torch.from_numpy(self.scales[1]))
        self.pk, self.pv = (torch.from_numpy(K8.values(c, s)) for c, s in zip(self.codes, self.scales))

    def bounds(self, o, size, lse, reach, vmax, T):
        s = self.scales[1][np.isfinite(self.scales[1])]
        big, far = (float(s.max()), float(np.abs(np.log2(s)).max())) if s.size else (1.0, 0.0)
        e = 2.0 ** -16 * reach + 2.0 ** -20 + 2.0 ** -22 * (1 + far)
        return (ulp(self.dtype) * np.abs(o) + (2.0 ** -11 + 2 * e + 2.0 ** -19) * size + T * 2.0 ** -32 * big * 448
                + tiny(self.dtype), e + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0))))


class Appended:
    """A batch whose new tokens are appended: float64 rotated keys and values beside what the kernel left."""

    def __init__(self, *, n, m, d, dtype, x_dtype, news, lens, page, table=True, seed=0, norm=False, theta=10000.0, slack=2,
                 extra=0, positions=None, with_q=True, spread=2.0):
        from rank_kv_cache_gb300 import palu as P
        rng = np.random.default_rng(seed)
        self.dtype, self.theta = dtype, theta
        B, top = len(news), max(max(lens), 1)
        per = -(-top // page) if table else 1
        pages = B * per + (slack if table else 0)
        self.row_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.lens, self.N = lens, int(self.row_start[-1]) + extra
        self.table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32) if table else None
        self.codes = [K8.encode(rng.standard_normal((pages, page, m, d)) * 60) for _ in range(2)]
        self.scales = [(2.0 ** np.round(rng.normal(-7, spread, (pages, page // 16, m)))).astype(np.float32) for _ in range(2)]
        width = n + 2 * m
        x = rounded(rng, (self.N, width * d + 16), "f32") * torch.from_numpy(
            rng.choice([0.25, 1.0, 4.0], (self.N, 1)).astype(np.float32))
        x = x.to(TYPES[x_dtype])                                            # a column block of something wider
        sides = ((0, n), (n, n + m), (n + m, width))
        self.q, self.k, self.v = (x[:, lo * d:hi * d].unflatten(1, (hi - lo, d)) for lo, hi in sides)
        self.wq, self.wk = ((1 + rounded(rng, (d,), x_dtype, 0.2)).to(TYPES[x_dtype]) if norm else None for _ in range(2))
        self.positions = positions
        dev = torch.device("cuda:0")
        self.layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, x_dtype=x_dtype, rope_theta=theta,
                                      max_batch=B, max_tokens=max(1, self.N))
        self.pages = P.KVPages8(*(codes_tensor(c).to(dev) for c in self.codes),
                                *(torch.from_numpy(s).to(dev) for s in self.scales))
        self.rows = P.KVRows(torch.from_numpy(self.row_start).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                             page_table=None if self.table is None else torch.from_numpy(self.table).to(dev),
                             positions=None if positions is None else torch.tensor(positions, dtype=torch.int32, device=dev),
                             n_tokens=self.N, max_new=max(max(news), 1), max_kv_len=top)
        xd = x.to(dev)
        qd, kd, vd = (xd[:, lo * d:hi * d].unflatten(1, (hi - lo, d)) for lo, hi in sides)
        self.q_out = torch.full((self.N, n, d), 7.0, dtype=TYPES[dtype], device=dev) if with_q else None
        self.run = lambda: self.layer.append(
            self.pages, self.rows, kd, vd, q=qd if with_q else None, q_out=self.q_out,
            q_weight=None if self.wq is None or not with_q else self.wq.to(dev), k_weight=None if self.wk is None else self.wk.to(dev))

    def rotated(self, x, w):
        """Float64, at the tokens of the batch's rows; zeros elsewhere."""
        x = x.double().numpy()
        out = np.zeros(x.shape)
        for b in range(len(self.lens)):
            for tok, t in KO.row_slots(self.row_start, self.lens, b):
                pos = t if self.positions is None else self.positions[tok]
                out[tok] = KO.norm_rope(x[tok:tok + 1], None if w is None else w.double().numpy(), [pos], self.theta, 1e-6)[0]
        return out

    def check(self):
        """Scales are equal (no seed has a block whose largest lies within the arithmetic's error of a power's border),
        values' codes too; keys' codes are the nearest or, within the error of the rotated value, its neighbour's."""
        torch.cuda.synchronize()
        self.layer.check_device()
        mine = np.zeros(self.N, dtype=bool)
        for b in range(len(self.lens)):
            for tok, t in KO.row_slots(self.row_start, self.lens, b):
                mine[tok] = True
        if self.q_out is not None:
            ref = self.rotated(self.q, self.wq)
            got = self.q_out.cpu()
            amp = pair_amplitude(KO.norm_rope(self.q.double().numpy(), None if self.wq is None else self.wq.double().numpy(),
                                              [0] * self.N, 0.0, 1e-6))
            check_rotated(got[mine], ref[mine], amp[mine], self.dtype)
            assert torch.all(got[~mine] == 7.0), "tokens of no row were written"
        for which, (x, w) in enumerate(((self.k, self.wk), (self.v, None))):
            y = self.rotated(x, w) if which == 0 else x.double().numpy()
            codes, scales = self.codes[which].copy(), self.scales[which].copy()
            K8.append(codes, scales, y, self.row_start, self.lens, self.table)
            got = (self.pages.k if which == 0 else self.pages.v).view(torch.uint8).cpu().numpy()
            got_s = (self.pages.k_scale if which == 0 else self.pages.v_scale).cpu().numpy()
            assert np.array_equal(got_s, scales)
            # a value that is off by 2^-20 of its pair before its rounding may fall to the next code: by one step,
            # 2^-3 of it, and only if it lies so near the middle of two
            if which == 1:
                assert np.array_equal(got, codes)
                continue
            off = got != codes
            assert off.mean() < 1e-3
            a, b = K8.decode(got[off]), K8.decode(codes[off])
            assert np.all(np.abs(a - b) <= np.maximum(2.0 ** -3 * np.maximum(np.abs(a), np.abs(b)), 2.0 ** -9))
