"""GPU parity of the norm and rotation of queries and keys and of the append into the pages, against the float64
oracle; bounds in tests/kv_cases.py."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO
from tests.kv_cases import TYPES, check_rotated, pair_amplitude, rounded

pytestmark = pytest.mark.gpu
THETA, EPS = 10000.0, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    return cuda_device


def _layer(n, m, d, dtype, x_dtype=None, tokens=64, batch=4, theta=THETA):
    from rank_kv_cache_gb300 import palu as P
    return P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, x_dtype=x_dtype, rope_theta=theta,
                            norm_eps=EPS, max_batch=batch, max_tokens=tokens)


def _check(got, x, w, positions, dtype, theta=THETA):
    x = x.double().cpu().numpy()
    w = None if w is None else w.double().cpu().numpy()
    ref = KO.norm_rope(x, w, positions, theta, EPS)
    normed = KO.norm_rope(x, w, positions, 0.0, EPS)
    check_rotated(got, ref, pair_amplitude(normed), dtype)


@pytest.mark.parametrize("dtype,x_dtype", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"),
                                           ("bf16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("n,m,d,norm", [(8, 8, 64, True), (32, 8, 128, False), (7, 1, 128, True), (5, 5, 64, False)])
def test_norm_rope_types_and_heads(dtype, x_dtype, n, m, d, norm):
    rng = np.random.default_rng(0)
    N = 3
    q, k = rounded(rng, (N, n, d), x_dtype).cuda(), rounded(rng, (N, m, d), x_dtype).cuda()
    wq, wk = (rounded(rng, (d,), x_dtype).cuda() for _ in range(2)) if norm else (None, None)
    pos = np.array([0, 17, 40000], dtype=np.int32)
    layer = _layer(n, m, d, dtype, x_dtype)
    qo, ko = layer.norm_rope(q, k, torch.from_numpy(pos).cuda(), q_weight=wq, k_weight=wk)
    _check(qo, q, wq, pos, dtype)
    _check(ko, k, wk, pos, dtype)


@pytest.mark.parametrize("N", [1, 2, 63, 700])
def test_norm_rope_token_counts_without_keys(N):
    rng = np.random.default_rng(N)
    q = rounded(rng, (N, 6, 64), "f16").cuda()
    pos = rng.integers(-100, 131072, N).astype(np.int32)
    layer = _layer(6, 2, 64, "f16", tokens=N)
    qo, ko = layer.norm_rope(q, positions=torch.from_numpy(pos).cuda())
    assert ko is None
    _check(qo, q, None, pos, "f16")


def test_far_positions_keep_their_angles():
    rng = np.random.default_rng(5)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 8 + 7], dtype=np.int32)
    q, k = rounded(rng, (4, 2, 128), "f32").cuda(), rounded(rng, (4, 2, 128), "f32").cuda()
    layer = _layer(2, 2, 128, "f32")
    qo, ko = layer.norm_rope(q, k, torch.from_numpy(pos).cuda())
    # the oracle's own angle pos * w carries 2^-53 relative: at 2^31 that is 2^-22, the bound's share for the angle
    _check(qo, q, None, pos, "f32")
    _check(ko, k, None, pos, "f32")


def test_strided_views_in_place_and_untouched_values():
    rng = np.random.default_rng(6)
    N, n, m, d = 37, 8, 2, 128
    qkv = rounded(rng, (N, (n + 2 * m) * d), "bf16").cuda()
    before = qkv.clone()
    q, k = qkv[:, :n * d].unflatten(1, (n, d)), qkv[:, n * d:(n + m) * d].unflatten(1, (m, d))
    wq, wk = rounded(rng, (d,), "bf16").cuda(), rounded(rng, (d,), "bf16").cuda()
    pos = rng.integers(0, 5000, N).astype(np.int32)
    layer = _layer(n, m, d, "bf16")
    layer.norm_rope(q, k, torch.from_numpy(pos).cuda(), q_weight=wq, k_weight=wk, q_out=q, k_out=k)
    b = before.unflatten(1, (n + 2 * m, d))
    _check(q, b[:, :n], wq, pos, "bf16")
    _check(k, b[:, n:n + m], wk, pos, "bf16")
    assert torch.equal(qkv[:, (n + m) * d:], before[:, (n + m) * d:])


def test_no_rotation_and_zero_vectors():
    q = torch.zeros(2, 4, 64, dtype=torch.float16).cuda()
    k = rounded(np.random.default_rng(7), (2, 4, 64), "f16").cuda()
    w = torch.ones(64, dtype=torch.float16).cuda()
    layer = _layer(4, 4, 64, "f16", theta=0.0)
    qo, ko = layer.norm_rope(q, k, q_weight=w)          # positions are not needed
    assert torch.equal(qo, q) and torch.equal(ko, k)     # 0 * rsqrt(eps) = 0; no norm, no rotation: a copy


@pytest.mark.parametrize("d,m,page,table", [(128, 2, 16, True), (64, 8, 7, True), (128, 3, 1, True), (64, 1, 64, True),
                                            (64, 8, 68, False)])
@pytest.mark.parametrize("dtype,x_dtype,norm", [("f16", "f32", False), ("bf16", "bf16", True), ("f32", "f32", True)])
def test_append_ragged_rows(d, m, page, table, dtype, x_dtype, norm):
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(page)
    n, g = 2 * m, 2
    news, lens = [5, 0, 1, 33], [40, 12, 1, 33]
    row_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    N = int(row_start[-1]) + 3                           # three tokens behind the last row
    per = -(-max(lens) // page) if table else 1
    n_pages = 4 * per + 1
    tab = rng.permutation(n_pages)[:4 * per].reshape(4, per).astype(np.int32) if table else None
    pk, pv = rounded(rng, (n_pages, page, m, d), dtype), rounded(rng, (n_pages, page, m, d), dtype)
    qkv = rounded(rng, (N, (n + 2 * m) * d), x_dtype)
    dev = qkv.cuda()
    q, k, v = (dev[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, n), (n, n + m), (n + m, n + 2 * m)))
    wq, wk = (rounded(rng, (d,), x_dtype).cuda() for _ in range(2)) if norm else (None, None)
    layer = _layer(n, m, d, dtype, x_dtype)
    pages = P.KVPages(pk.cuda(), pv.cuda())
    rows = P.KVRows(torch.from_numpy(row_start).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), n_tokens=N,
                    max_new=max(news), max_kv_len=max(lens), page_table=None if tab is None else torch.from_numpy(tab).cuda())
    q_out = torch.full((N, n, d), 7.0, dtype=TYPES[dtype]).cuda()
    layer.append(pages, rows, k, v, q=q, q_weight=wq, k_weight=wk, q_out=q_out)
    layer.check_device()
    pos = np.zeros(N, dtype=np.int64)
    written = torch.zeros(n_pages, page, dtype=torch.bool)
    hk, hv = k.cpu(), v.cpu()
    for b in range(4):
        for tok, t in KO.row_slots(row_start, lens, b):
            pos[tok] = t
            pg, off = KO.slot(tab, page, b, t)
            written[pg, off] = True
            _check(pages.k[pg, off][None], hk[tok:tok + 1], wk, [t], dtype)
            assert torch.equal(pages.v[pg, off].cpu(), hv[tok].to(TYPES[dtype]))
    last = int(row_start[-1])
    _check(q_out[:last], q[:last], wq, pos[:last], dtype)
    assert torch.all(q_out[last:] == 7.0)
    assert torch.equal(pages.k.cpu()[~written], pk[~written]) and torch.equal(pages.v.cpu()[~written], pv[~written])


def test_append_at_given_positions_without_queries():
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(8)
    k, v = rounded(rng, (3, 2, 64), "f16").cuda(), rounded(rng, (3, 2, 64), "f16").cuda()
    pages = P.KVPages(torch.zeros(1, 8, 2, 64, dtype=torch.float16).cuda(), torch.zeros(1, 8, 2, 64, dtype=torch.float16).cuda())
    pos = np.array([100, 5, 70000], dtype=np.int32)
    rows = P.KVRows(torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([6], dtype=torch.int32).cuda(),
                    n_tokens=3, max_new=3, max_kv_len=8, positions=torch.from_numpy(pos).cuda())
    layer = _layer(2, 2, 64, "f16")
    assert layer.append(pages, rows, k, v) is None
    layer.check_device()
    _check(pages.k[0, 3:6], k, None, pos, "f16")
    assert torch.equal(pages.v[0, 3:6], v)
    assert torch.all(pages.k[0, :3] == 0) and torch.all(pages.k[0, 6:] == 0)


def test_bad_slots_are_reported_and_not_stored():
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(9)
    k, v = rounded(rng, (4, 1, 64), "f16").cuda(), rounded(rng, (4, 1, 64), "f16").cuda()
    layer = _layer(1, 1, 64, "f16")

    def run(lens, table, page=2, row_start=(0, 4)):
        pages = P.KVPages(torch.zeros(3, page, 1, 64, dtype=torch.float16).cuda(),
                          torch.zeros(3, page, 1, 64, dtype=torch.float16).cuda())
        rows = P.KVRows(torch.tensor(row_start, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        n_tokens=4, max_new=4, max_kv_len=4, page_table=torch.tensor(table, dtype=torch.int32).cuda())
        layer.append(pages, rows, k, v)
        with pytest.raises(P.PaluError):
            layer.check_device()
        layer.check_device()                              # reported once
        return pages

    p = run([4], [[1, 3]])                                # a page past the pool: its two tokens are dropped
    assert torch.equal(p.v[1], v[:2]) and torch.all(p.v[0] == 0) and torch.all(p.v[2] == 0)
    p = run([4], [[-1, 2]])
    assert torch.equal(p.v[2], v[2:]) and torch.all(p.v[:2] == 0)
    p = run([2], [[0, 1]])                                # four new tokens, two cached: the first two have no slot
    assert torch.equal(p.v[0], v[2:]) and torch.all(p.v[1:] == 0)
    p = run([6], [[0, 1]])                                # slots 2 .. 5 of a table for four
    assert torch.equal(p.v[1], v[:2]) and torch.all(p.v[0] == 0) and torch.all(p.v[2] == 0)


def test_refusals():
    from rank_kv_cache_gb300 import palu as P
    layer = _layer(4, 2, 64, "f16", tokens=8, batch=2)
    q, k = torch.zeros(3, 4, 64, dtype=torch.float16).cuda(), torch.zeros(3, 2, 64, dtype=torch.float16).cuda()
    pos = torch.zeros(3, dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        layer.norm_rope(q, k, pos.long())
    with pytest.raises(ValueError):
        layer.norm_rope(q.float(), k, pos)
    with pytest.raises(ValueError):
        layer.norm_rope(q.transpose(0, 1), k, pos)
    with pytest.raises(P.PaluError):
        layer.norm_rope(q, k)                             # a rotating handle needs positions
    big = torch.zeros(9, 4, 64, dtype=torch.float16).cuda()
    with pytest.raises(P.PaluError):
        layer.norm_rope(big, positions=torch.zeros(9, dtype=torch.int32).cuda())
    h, s = layer.handle, torch.cuda.current_stream().cuda_stream
    buf = torch.zeros(4096, dtype=torch.float16).cuda()
    x, o = q.data_ptr(), buf.data_ptr()
    bad = P.PALU_ERR_INVALID_ARG
    assert P.palu_norm_rope(h, x + 2, 256, None, 0, None, None, pos.data_ptr(), 3, o, 256, None, 0, s) == bad
    assert P.palu_norm_rope(h, x, 252, None, 0, None, None, pos.data_ptr(), 3, o, 256, None, 0, s) == bad
    assert P.palu_norm_rope(h, x, 260, None, 0, None, None, pos.data_ptr(), 3, o, 256, None, 0, s) == bad
    assert P.palu_norm_rope(h, x, 256, None, 0, None, None, pos.data_ptr(), 3, None, 256, None, 0, s) == bad
    assert P.palu_norm_rope(h, x, 256, k.data_ptr(), 128, None, None, pos.data_ptr(), 3, o, 256, None, 0, s) == bad
    assert P.palu_norm_rope(h, x, 256, None, 0, None, None, pos.data_ptr(), 3, x, 264, None, 0, s) == bad  # in place
    assert P.palu_norm_rope(h, x, 256, None, 0, x + 8, None, pos.data_ptr(), 3, o, 256, None, 0, s) == bad
    pages = P.KVPages(torch.zeros(2, 4, 2, 64, dtype=torch.float16).cuda(), torch.zeros(2, 4, 2, 64, dtype=torch.float16).cuda())
    start, length = torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    good = dict(n_tokens=3, max_new=3, max_kv_len=4)
    v = torch.zeros_like(k)
    layer.append(pages, P.KVRows(start, length, **good), k, v)
    for kw in (dict(good, max_kv_len=5), dict(good, max_new=-1), dict(good, max_kv_len=-1)):
        with pytest.raises(P.PaluError):                  # longer than a page without a table, or negative bounds
            layer.append(pages, P.KVRows(start, length, **kw), k, v)
    three = torch.zeros(3, dtype=torch.int32).cuda()
    with pytest.raises(P.PaluError):                      # more rows than max_batch
        layer.append(pages, P.KVRows(torch.zeros(4, dtype=torch.int32).cuda(), three, **good), k, v)
    with pytest.raises(ValueError):                       # q_out without q
        layer.append(pages, P.KVRows(start, length, **good), k, v, q_out=q)
    with pytest.raises(ValueError):                       # pages of other heads
        layer.append(P.KVPages(pages.k[:, :, :1].contiguous(), pages.v[:, :, :1].contiguous()),
                     P.KVRows(start, length, **good), k, v)
    layer.check_device()
