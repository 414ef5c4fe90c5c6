"""GPU tests of the 8-bit cache, the plan and the verification where calls are unusual: arguments that are refused, offsets past
32 bits, the largest and the smallest sizes, shared pages, other streams, and calls side by side."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8
from tests import test_gpu_kv_plan as plans
from tests import test_gpu_kv_verify as verifications
from tests.kv8_cases import Appended, Batch8
from tests.kv_cases import rounded

pytestmark = pytest.mark.gpu


def _copy(struct, **kw):
    x = type(struct)()
    for f, _ in struct._fields_:
        setattr(x, f, getattr(struct, f))
    for f, v in kw.items():
        setattr(x, f, v)
    return x


def _refused_pages_and_rows(call, p, r):
    """What append and attend alike refuse; call(pages, rows) -> status."""
    from rank_kv_cache_gb300 import palu as P
    bad = P.PALU_ERR_INVALID_ARG
    for field, value, status in (("n_pages", 0, bad), ("page_size", 0, bad), ("page_size", 8, bad), ("page_size", 24, bad), ("k", 0, bad),
                                 ("v", p.v + 8, bad), ("k_scale", 0, bad), ("v_scale", 0, bad), ("v_scale", p.v_scale + 2, bad),
                                 ("n_pages", 1 << 28, P.PALU_ERR_UNSUPPORTED)):
        assert call(_copy(p, **{field: value}), r) == status, field
    for field, value in (("row_start", 0), ("kv_len", 0), ("kv_len", r.kv_len + 2), ("page_table", r.page_table + 2),
                         ("batch", 2), ("batch", -1), ("n_tokens", 3), ("n_tokens", -1), ("max_new", -1), ("max_kv_len", 33),
                         ("max_kv_len", -1), ("table_pages", 0)):
        assert call(p, _copy(r, **{field: value})) == bad, field
    assert call(p, _copy(r, page_table=0, max_kv_len=17)) == bad                # longer than a page, without a table
    assert call(p, _copy(r, batch=0, row_start=0, kv_len=0)) == P.PALU_OK       # nothing to do
    assert call(p, _copy(r, n_tokens=0, row_start=0, kv_len=0)) == P.PALU_OK


def test_attend_refuses(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    b = Batch8(n=4, m=2, d=64, dtype="f16", news=[2], lens=[20], page=16, seed=15)
    h, s = b.layer.handle, torch.cuda.current_stream().cuda_stream
    p, r = b.pages.c_struct(), b.rows.c_struct()
    out = torch.zeros((2, 4, 64), dtype=torch.float16, device=b.dev)
    q, o, bad = b.qd.data_ptr(), out.data_ptr(), P.PALU_ERR_INVALID_ARG
    assert P.palu_attend_kv8(h, p, r, q, 256, o, None, s) == P.PALU_OK
    for args in ((q + 2, 256, o, None), (q, 255, o, None), (q, 260, o, None), (q, 256, o + 8, None), (q, 256, 0, None),
                 (0, 256, o, None), (q, 256, o, o + 2)):
        assert P.palu_attend_kv8(h, p, r, *args, s) == bad, args
    _refused_pages_and_rows(lambda x, y: P.palu_attend_kv8(h, x, y, q, 256, o, None, s), p, r)
    wide = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=64, dtype="f32", max_batch=1, max_tokens=2)
    assert P.palu_attend_kv8(wide.handle, p, r, q, 256, o, None, s) == P.PALU_ERR_UNSUPPORTED
    for kw in (dict(out=out.float()), dict(out=torch.zeros((2, 8, 64), dtype=torch.float16, device=b.dev)[:, ::2]),
               dict(lse=torch.zeros((2, 4), dtype=torch.float64, device=b.dev)), dict(lse=torch.zeros((4, 2), device=b.dev).T)):
        with pytest.raises(ValueError):
            b.layer.attend(b.pages, b.rows, b.qd, **kw)
    with pytest.raises(ValueError):                                            # pages of other heads
        b.layer.attend(P.KVPages8.empty(2, 16, 1, 64), b.rows, b.qd)
    with pytest.raises(ValueError):                                            # and on another device
        b.layer.attend(P.KVPages8.empty(2, 16, 2, 64, device="cpu"), b.rows, b.qd)
    b.layer.check_device()


def test_append_refuses(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    a = Appended(n=4, m=2, d=64, dtype="bf16", x_dtype="f32", news=[2], lens=[20], page=16)
    h, s = a.layer.handle, torch.cuda.current_stream().cuda_stream
    p, r = a.pages.c_struct(), a.rows.c_struct()
    x = torch.zeros(2, 8, 64, device="cuda")
    o = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda").data_ptr()
    q, k, v, bad = x.data_ptr(), x[:, 4:].data_ptr(), x[:, 6:].data_ptr(), P.PALU_ERR_INVALID_ARG
    good = (q, 512, k, 512, v, 512, None, None, o)
    assert P.palu_append_kv8(h, p, r, *good, s) == P.PALU_OK
    for at, value in ((0, q + 4), (1, 510), (1, 128), (2, 0), (2, k + 8), (3, 64), (3, 511), (4, 0), (5, 64), (6, q + 4), (7, q + 8),
                      (8, None), (8, o + 8), (0, None)):
        args = list(good)
        args[at] = value
        assert P.palu_append_kv8(h, p, r, *args, s) == bad, (at, value)
    assert P.palu_append_kv8(h, p, r, q, 512, k, 512, v, 512, None, None, q, s) == bad     # in place, of another type
    _refused_pages_and_rows(lambda y, z: P.palu_append_kv8(h, y, z, *good, s), p, r)
    wide = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=64, dtype="f32", max_batch=1, max_tokens=2)
    assert P.palu_append_kv8(wide.handle, p, r, *good, s) == P.PALU_ERR_UNSUPPORTED
    with pytest.raises(ValueError):                                            # q_out without q
        a.layer.append(a.pages, a.rows, x[:, 4:6], x[:, 6:], q_out=x[:, :4].bfloat16())
    a.layer.check_device()


def test_plan_refuses(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=2, max_tokens=8)
    h, s, bad = layer.handle, torch.cuda.current_stream().cuda_stream, P.PALU_ERR_INVALID_ARG
    pool = P.KVPool.empty(2, 3, 6, 16)
    z = torch.zeros(64, dtype=torch.int32, device="cuda")
    at = [z[8 * i:].data_ptr() for i in range(8)]
    good = [at[0], at[1], 2, 8, 8, 48, at[2], at[3], at[4], at[5], at[6], at[7]]
    call = lambda c, args: P.palu_plan_kv_rows(h, c, *args, s)
    assert call(pool.c_struct(), good) == P.PALU_OK
    for i, value, status in ((0, 0, bad), (0, at[0] + 2, bad), (1, 0, bad), (2, 3, bad), (2, -1, bad), (3, 9, bad), (3, -1, bad),
                             (4, -1, bad), (5, 49, bad), (5, -1, bad), (6, 0, bad), (7, 0, bad), (7, at[3] + 1, bad), (8, at[4] + 2, bad),
                             (9, at[5] + 2, bad), (10, at[6] + 2, bad), (11, at[7] + 2, bad), (2, 0, P.PALU_OK)):
        args = list(good)
        args[i] = value
        assert call(pool.c_struct(), args) == status, (i, value)
    c = pool.c_struct()
    for field, value, status in (("page_table", 0, bad), ("held", 0, bad), ("free_pages", 0, bad), ("free_state", 0, bad),
                                 ("held", c.held + 2, bad), ("n_pages", 0, bad), ("page_size", 0, bad), ("table_pages", 0, bad),
                                 ("n_pages", 1 << 28, P.PALU_ERR_UNSUPPORTED), ("table_pages", 1 << 31, P.PALU_ERR_UNSUPPORTED)):
        assert call(_copy(c, **{field: value}), good) == status, field
    i32 = dict(dtype=torch.int32, device="cuda")
    start, lens, new = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    rows = P.KVRows(start, lens, page_table=pool.page_table, n_tokens=8, max_new=8, max_kv_len=48)
    layer.plan(pool, new, lens, rows)
    for kw in (dict(new=new.long()), dict(new=new[:1]), dict(kv_len=torch.zeros(4, **i32)[::2]), dict(slots=torch.zeros(7, **i32)),
               dict(held_out=torch.zeros(3, **i32)), dict(state_out=torch.zeros(1, **i32)), dict(new=new.cpu()),
               dict(rows=P.KVRows(start, lens, page_table=pool.page_table.clone(), n_tokens=8, max_new=8, max_kv_len=48)),
               dict(rows=P.KVRows(start, lens, n_tokens=8, max_new=8, max_kv_len=48))):
        args = dict(dict(new=new, kv_len=lens, rows=rows), **kw)
        with pytest.raises(ValueError):
            layer.plan(pool, args.pop("new"), args.pop("kv_len"), args.pop("rows"), **args)
    layer.check_device()


def test_verify_refuses(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=2, max_tokens=6)
    h, s, bad, no = layer.handle, torch.cuda.current_stream().cuda_stream, P.PALU_ERR_INVALID_ARG, P.PALU_ERR_UNSUPPORTED
    B, K, V = 2, 2, 40
    p, q, u = torch.full((6, V), 1 / V, device="cuda"), torch.full((B, K, V), 1 / V, device="cuda"), torch.zeros(B, K + 1, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    start, drafts, lens = torch.tensor([0, 3, 6], **i32), torch.zeros(B, K, **i32), torch.full((B,), 9, **i32)
    tokens, accepted = torch.zeros(B, K + 1, **i32), torch.zeros(B, **i32)
    a = lambda t: t.data_ptr()
    good = [a(p), V, a(q), V, P.PALU_F32, V, a(start), B, 6, a(drafts), K, a(u), a(tokens), a(accepted), a(lens), a(lens)]
    assert P.palu_verify_drafts(h, *good, s) == P.PALU_OK
    for i, value, status in ((0, 0, bad), (0, a(p) + 2, bad), (1, V - 1, bad), (1, 1 << 40, bad), (2, a(q) + 1, bad), (3, V - 1, bad),
                             (3, 1 << 40, bad), (4, 9, bad), (4, P.PALU_INT4, no), (5, 0, bad), (5, (1 << 20) + 1, no), (6, 0, bad),
                             (6, a(start) + 2, bad), (7, 3, bad), (7, -1, bad), (8, 7, bad), (8, -1, bad), (9, 0, bad), (10, -1, bad),
                             (10, (1 << 20) + 1, no), (11, 0, bad), (12, 0, bad), (12, a(tokens) + 2, bad), (13, 0, bad), (14, None, bad),
                             (15, None, bad), (15, a(lens) + 2, bad), (7, 0, P.PALU_OK)):
        args = list(good)
        args[i] = value
        assert P.palu_verify_drafts(h, *args, s) == status, (i, value)
    args = dict(target=p, draft_tokens=drafts, uniforms=u, row_start=start, draft=q)
    layer.verify(**args)
    for kw in (dict(target=p.double()), dict(target=p.cpu()), dict(target=p.T), dict(target=p[0]), dict(draft=q.half()), dict(draft=q[:1]),
               dict(draft=q.transpose(0, 1)), dict(draft=torch.ones(B, 3, V, device="cuda")[:, :2]), dict(draft_tokens=drafts.long()),
               dict(draft_tokens=drafts[0]), dict(uniforms=u[:, :2]), dict(uniforms=u.double()), dict(row_start=start[:2]),
               dict(tokens=tokens[:1]), dict(accepted=accepted.float()), dict(kv_len=lens[:1]), dict(kv_len_out=lens)):
        with pytest.raises(ValueError):
            layer.verify(**dict(args, **kw))
    with pytest.raises(P.PaluError):                                           # rows that lie on one another
        layer.verify(**dict(args, target=p[:1].expand(6, V)))
    layer.check_device()


@pytest.mark.parametrize("new", [1, 6, 70])
@pytest.mark.parametrize("table", [True, False])
def test_pools_past_32_bit_offsets(cuda_device, new, table):
    """Pages at both ends of a pool of over 2^32 codes: the same bits, written and read, as from a small pool."""
    from rank_kv_cache_gb300 import palu as P
    rng, dev = np.random.default_rng(31), torch.device("cuda:0")
    n, m, d, B, L = 16, 8, 128, 2, 300
    page, small = (64, 12) if table else (320, B)
    far = 2 ** 32 // (m * d * 64) + 40 if table else B
    wide = 64 if table else 2 ** 32 // (m * d) + 64                     # without a table row 1 is page 1
    ids = (torch.tensor([far - 1 - i if i % 2 else i for i in range(small)]) if table else torch.arange(B)).to(dev)
    pools = []
    for pages, size in ((small, page), (far, wide)):
        codes = [torch.empty(pages, size, m, d, dtype=torch.uint8, device=dev) for _ in range(2)]
        pools.append(P.KVPages8(*codes, *(torch.empty(pages, size // 16, m, device=dev) for _ in range(2))))
    for name in ("k", "v"):
        x = torch.from_numpy(K8.encode(rng.standard_normal((small, page, m, d)) * 60)).to(dev)
        s = torch.from_numpy((2.0 ** rng.integers(-9, -5, (small, page // 16, m))).astype(np.float32)).to(dev)
        for pool, where in zip(pools, (torch.arange(small, device=dev), ids)):
            getattr(pool, name)[where, :page] = x
            getattr(pool, name + "_scale")[where, :page // 16] = s
    layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype="bf16", max_batch=B, max_tokens=B * new)
    start = torch.arange(0, B * new + 1, new, dtype=torch.int32, device=dev)
    lens = torch.tensor([L, L - 7], dtype=torch.int32, device=dev)
    order = torch.from_numpy(rng.permutation(small)[:B * 5].reshape(B, 5)).to(dev) if table else None
    q, k, v = (rounded(rng, (B * new, h, d), "bf16").to(dev) for h in (n, m, m))
    got = []
    for pool, where in zip(pools, (None, ids)):
        t = None if order is None else (order if where is None else where[order]).int()
        rows = P.KVRows(start, lens, n_tokens=B * new, max_new=new, max_kv_len=L, page_table=t)
        lse = torch.empty(B * new, n, device=dev)
        q_rot = layer.append(pool, rows, k, v, q=q)
        got.append((q_rot, layer.attend(pool, rows, q_rot, lse=lse), lse))
    layer.check_device()
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    for name in ("k", "v"):
        assert torch.equal(getattr(pools[0], name), getattr(pools[1], name)[ids, :page])
        assert torch.equal(getattr(pools[0], name + "_scale"), getattr(pools[1], name + "_scale")[ids, :page // 16])


def test_probabilities_past_32_bit_offsets(cuda_device):
    """The last rows of over 2^32 probabilities, and drafts whose rows lie 2^29 elements apart, judged as in small tensors."""
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(3)
    V, N, B, K = 1 << 16, (1 << 16) + 40, 3, 2
    c = verifications.make(rng, [3] * B, V, "f16")
    want = verifications.run(c)
    wide = torch.empty(N, V, dtype=torch.float16, device="cuda")
    wide[N - 9:] = c["target"].cuda()
    step = 1 << 29
    far = torch.empty(B * K * step, dtype=torch.float16, device="cuda").as_strided((B, K, V), (K * step, step, 1))
    far.copy_(c["draft"])
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B, max_tokens=N)
    tokens, accepted = layer.verify(wide, torch.from_numpy(c["drafts"]).cuda(), torch.from_numpy(c["u"]).cuda(),
                                    torch.tensor([N - 9, N - 6, N - 3, N], dtype=torch.int32, device="cuda"), draft=far)
    layer.check_device()
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])


@pytest.mark.parametrize("n,d,new", [(2, 64, 1), (4, 128, 1), (4, 128, 20)])
def test_the_most_rows_over_pages_that_they_share(cuda_device, n, d, new):
    """65535 rows (3276 of 20 tokens) that share their cached pages: all give one row's output, within the bounds."""
    from rank_kv_cache_gb300 import palu as P
    b = Batch8(n=n, m=1, d=d, dtype="bf16", news=[new], lens=[90], page=32, seed=7)
    B = 65535 // new
    layer = P.PagedAttention(n_heads=n, n_kv_heads=1, head_dim=d, dtype="bf16", max_batch=B, max_tokens=B * new)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.from_numpy(b.table).cuda().expand(B, b.table.shape[1]).contiguous()
    rows = P.KVRows(torch.arange(0, B * new + 1, new, **i32), torch.full((B,), 90, **i32), page_table=table, n_tokens=B * new, max_new=new,
                    max_kv_len=90)
    lse = torch.empty(B * new, n, device="cuda")
    out = layer.attend(b.pages, rows, b.qd.repeat(B, 1, 1), lse=lse).view(B, new, n, d)
    layer.check_device()
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse.view(B, -1), lse[:new].view(1, -1).expand(B, -1))
    b.check(out[0], lse[:new], b.oracle())


def test_the_most_rows_appended(cuda_device):
    a = Appended(n=2, m=1, d=64, dtype="bf16", x_dtype="bf16", news=[1] * 4096, lens=[1 + i % 32 for i in range(4096)], page=32, seed=4)
    a.run()
    a.check()
    from rank_kv_cache_gb300 import palu as P
    B = 65535
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(B, 2, 64, generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    layer = P.PagedAttention(n_heads=2, n_kv_heads=1, head_dim=64, dtype="bf16", rope_theta=0.0, max_batch=B, max_tokens=B)
    pages = P.KVPages8.empty(B, 16, 1, 64)
    rows = P.KVRows(torch.arange(B + 1, **i32), torch.ones(B, **i32), n_tokens=B, max_new=1, max_kv_len=16)
    layer.append(pages, rows, x[:, :1], x[:, 1:])
    layer.check_device()
    for t, codes, scale in ((x[:, 0], pages.k, pages.k_scale), (x[:, 1], pages.v, pages.v_scale)):
        s = scale[:, 0, 0]
        amax = t.float().abs().amax(1)
        assert torch.equal(torch.exp2(torch.ceil(torch.log2(amax / 448))), s)
        assert torch.equal(codes[:, 0, 0].float(), (t.float() / s[:, None]).to(torch.float8_e4m3fn).float())
        assert not codes[:, 1:].view(torch.uint8).any()


def test_the_most_rows_planned(cuda_device):
    c = plans.make(np.random.default_rng(12), 65535, 16, 60, 4, 300, 10)
    got, layer = plans.run(c, 65536 * 4)
    plans.check(c, got, 65536 * 4)
    layer.check_device()


def test_the_most_rows_verified(cuda_device):
    """Eighths, whose products, sums and differences are exact in any order."""
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(9)
    B, V = 65535, 5
    p, q = (rng.multinomial(8, [1 / V] * V, size) / 8 for size in ((B, 2), (B, 1)))
    x = np.array([rng.choice(V, p=w) for w in q[:, 0]])
    u = rng.integers(0, 64, (B, 2)) / 64
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B, max_tokens=2 * B)
    cuda = lambda t, dtype: torch.from_numpy(np.ascontiguousarray(t)).to(dtype).cuda()
    tokens, accepted = layer.verify(cuda(p.reshape(2 * B, V), torch.float16), cuda(x[:, None], torch.int32), cuda(u, torch.float32),
                                    torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda"), draft=cuda(q, torch.float16))
    layer.check_device()
    at = np.arange(B)
    took = u[:, 0] * q[at, 0, x] < p[at, 0, x]
    w = np.where(took[:, None], p[:, 1], np.maximum(p[:, 0] - q[:, 0], 0))
    w = np.where(w.sum(1, keepdims=True) == 0, p[:, 0], w)
    drawn = (np.cumsum(w, 1) <= u[:, 1:] * w.sum(1, keepdims=True)).sum(1)
    want = np.stack([np.where(took, x, drawn), np.where(took, drawn, -1)], 1)
    assert np.array_equal(accepted.cpu().numpy(), took) and np.array_equal(tokens.cpu().numpy(), want)


def test_nothing_to_do(cuda_device):
    """No rows, no tokens, no drafts: nothing is written, and nothing recorded."""
    from rank_kv_cache_gb300 import palu as P
    i32 = dict(dtype=torch.int32, device="cuda")
    layer = P.PagedAttention(n_heads=2, n_kv_heads=1, head_dim=64, dtype="f16", max_batch=2, max_tokens=4)
    pages, pool = P.KVPages8.empty(2, 16, 1, 64), P.KVPool.empty(2, 1, 2, 16)
    x = torch.ones(0, 2, 64, dtype=torch.float16, device="cuda")
    for B in (0, 2):
        rows = P.KVRows(torch.zeros(B + 1, **i32), torch.zeros(B, **i32), n_tokens=0, max_new=0, max_kv_len=16,
                        page_table=torch.zeros(B, 1, **i32))
        assert layer.append(pages, rows, x[:, :1], x[:, 1:], q=x).shape == (0, 2, 64)
        assert layer.attend(pages, rows, x).shape == (0, 2, 64)
    assert not pages.k.view(torch.uint8).any() and bool((pages.k_scale == 1).all())
    rows = P.KVRows(torch.full((3,), 5, **i32), torch.full((2,), 5, **i32), page_table=pool.page_table, n_tokens=0, max_new=4, max_kv_len=16)
    layer.plan(pool, torch.tensor([0, 3], **i32), torch.zeros(2, **i32), rows)      # no place for a token: nobody is admitted
    assert rows.tensors[0].tolist() == [0, 0, 0] and rows.tensors[1].tolist() == [0, 0] and pool.state.tolist() == [0, 2]
    p = torch.eye(3, device="cuda")[:2]
    tokens, accepted = layer.verify(p, torch.zeros(2, 0, **i32), torch.zeros(2, 1, device="cuda"), torch.tensor([0, 1, 2], **i32))
    assert tokens.tolist() == [[0], [1]] and accepted.tolist() == [0, 0]
    tokens, accepted = layer.verify(p[:0], torch.zeros(2, 1, **i32), torch.zeros(2, 2, device="cuda"), torch.zeros(3, **i32))
    assert tokens.tolist() == [[-1, -1]] * 2 and accepted.tolist() == [0, 0]
    tokens, accepted = layer.verify(p, torch.zeros(0, 1, **i32), torch.zeros(0, 2, device="cuda"), torch.zeros(1, **i32))
    assert tokens.shape == (0, 2) and accepted.shape == (0,)
    layer.check_device()


def test_calls_side_by_side_on_streams_of_their_own(cuda_device):
    """Two objects on two streams, and a third that captured its calls: each gives what it gives alone, over and over."""
    from rank_kv_cache_gb300 import palu as P
    batches = [Batch8(n=8, m=2, d=128, dtype="bf16", news=[1, 30], lens=[2000, 1500], page=16, seed=1),
               Batch8(n=8, m=2, d=128, dtype="bf16", news=[3, 2], lens=[3000, 700], page=64, seed=2),
               Batch8(n=4, m=4, d=64, dtype="f16", news=[200], lens=[900], page=48, seed=3)]
    rng = np.random.default_rng(4)
    judged = [verifications.make(rng, [4, 2, 5], 30000 + i, "bf16") for i in range(3)]
    alone = [(b.layer.attend(b.pages, b.rows, b.qd).clone(), verifications.run(c)) for b, c in zip(batches, judged)]
    torch.cuda.synchronize()
    dev = [[torch.from_numpy(c[k]).cuda() for k in ("drafts", "u", "starts")] + [c["target"].cuda(), c["draft"].cuda()] for c in judged]
    layers = [P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=3, max_tokens=11) for _ in judged]

    def both(i, stream=None):
        out = batches[i].layer.attend(batches[i].pages, batches[i].rows, batches[i].qd, stream=stream)
        drafts, u, starts, target, draft = dev[i]
        return out, *layers[i].verify(target, drafts, u, starts, draft=draft, stream=stream)

    streams = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(2)
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(both(i, s))
        graph.replay()
    torch.cuda.synchronize()
    got[2].append(held)
    for i, runs in enumerate(got):
        for out, tokens, accepted in runs:
            assert torch.equal(out, alone[i][0])
            assert np.array_equal(tokens.cpu().numpy(), alone[i][1][0]) and np.array_equal(accepted.cpu().numpy(), alone[i][1][1])
        batches[i].layer.check_device()
        layers[i].check_device()


def test_plan_and_append_on_a_side_stream(cuda_device):
    """What one stream leaves is waited for by no other: the whole step stands on the stream that is named."""
    from rank_kv_cache_gb300 import palu as P
    i32 = dict(dtype=torch.int32, device="cuda")
    layer = P.PagedAttention(n_heads=2, n_kv_heads=1, head_dim=64, dtype="bf16", max_batch=2, max_tokens=8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, 4, 64, generator=g, device="cuda").bfloat16()
    results = []
    for side in (None, torch.cuda.Stream()):
        pool, pages = P.KVPool.empty(2, 2, 4, 16), P.KVPages8.empty(4, 16, 1, 64)
        lens, new = torch.tensor([15, 0], **i32), torch.tensor([3, 5], **i32)
        pool.held[0], pool.page_table[0, 0] = 1, 0
        pool.state.copy_(torch.tensor([1, 3], **i32))
        rows = P.KVRows(torch.zeros(3, **i32), lens, page_table=pool.page_table, positions=torch.zeros(8, **i32), n_tokens=8, max_new=5,
                        max_kv_len=32)
        slots = torch.zeros(8, **i32)
        torch.cuda.synchronize()
        if side is not None:
            torch.cuda._sleep(20_000_000)                                      # the current stream is busy meanwhile
        layer.plan(pool, new, lens, rows, slots=slots, stream=side)
        q = layer.append(pages, rows, x[:, 2:3], x[:, 3:], q=x[:, :2], stream=side)
        out = layer.attend(pages, rows, q, stream=side)
        torch.cuda.synchronize()
        results.append([out, q, slots, lens, pages.k.view(torch.uint8), pages.v_scale, pool.state])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    layer.check_device()


def test_pages_of_a_derived_class_are_pages(cuda_device):
    """A program's own class of 8-bit pages, with what it keeps beside them, goes wherever the pages do."""
    from rank_kv_cache_gb300 import palu as P

    class Layered(P.KVPages8):
        layer = 3

    a = Appended(n=4, m=2, d=64, dtype="f16", x_dtype="f16", news=[3, 20], lens=[40, 33], page=16, seed=4)
    a.pages = Layered(a.pages.k, a.pages.v, a.pages.k_scale, a.pages.v_scale)
    a.run()
    a.check()
    b = Batch8(n=4, m=2, d=64, dtype="f16", news=[3, 20], lens=[40, 33], page=16, seed=5)
    b.pages = Layered(b.pages.k, b.pages.v, b.pages.k_scale, b.pages.v_scale)
    b.run_and_check()
