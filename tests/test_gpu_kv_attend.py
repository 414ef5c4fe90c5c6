"""GPU parity of the attention of new tokens over paged caches against the float64 oracle; bounds in
tests/kv_cases.py. Every slot that no row may read holds NaN (keys) or infinity (values)."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO
from tests.kv_cases import TYPES, Batch, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    return cuda_device


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("bf16", 128), ("f16", 64), ("bf16", 64)])
@pytest.mark.parametrize("n,m", [(4, 4), (8, 2), (7, 1), (6, 2)])
def test_one_token_of_ragged_rows(dtype, d, n, m):
    Batch(n=n, m=m, d=d, dtype=dtype, news=[1, 1, 1, 1, 1], lens=[1, 31, 129, 300, 17], page=16, seed=n,
          q_scale=2.0).run_and_check()


@pytest.mark.parametrize("page,table", [(1, True), (5, True), (16, True), (24, True), (64, True), (128, True),
                                        (256, True), (301, False)])
@pytest.mark.parametrize("new", [1, 3, 37, 140])
def test_page_sizes_and_chunks(page, table, new):
    Batch(n=4, m=2, d=128, dtype="f16", news=[new, max(1, new // 2)], lens=[301, max(new // 2, 1)], page=page,
          table=table, seed=page).run_and_check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,length", [(1, 1), (2, 2), (15, 15), (16, 17), (17, 400), (64, 64), (127, 127),
                                        (128, 128), (129, 129), (130, 259), (255, 256), (257, 257), (300, 511)])
def test_lengths_around_the_tiles(d, new, length):
    Batch(n=2, m=1, d=d, dtype="bf16", news=[new], lens=[length], page=32, seed=new, q_scale=2.0).run_and_check()


@pytest.mark.parametrize("n,m", [(64, 1), (33, 3), (40, 5), (3, 3), (12, 1), (28, 4)])
@pytest.mark.parametrize("new", [1, 9, 50])
def test_group_sizes(n, m, new):
    Batch(n=n, m=m, d=64, dtype="f16", news=[new, 1, new], lens=[new, 70, 150], page=16, seed=n).run_and_check()


@pytest.mark.parametrize("new", [1, 40])
def test_rows_without_new_tokens_and_tokens_of_no_row(new):
    Batch(n=4, m=2, d=128, dtype="f16", news=[0, new, 0, 2, 0], lens=[9, 200, 0, 33, 50], page=16, extra_tokens=5,
          seed=1).run_and_check()


@pytest.mark.parametrize("news,lens", [([3], [1]), ([3, 1], [0, 0]), ([40, 2], [10, 0]), ([200], [130])])
def test_tokens_that_see_nothing_are_empty(news, lens):
    b = Batch(n=4, m=2, d=128, dtype="bf16", news=news, lens=lens, page=16, seed=2)
    out, lse = b.run_and_check()
    blind = news[0] - lens[0]
    assert torch.all(out[:blind] == 0) and torch.all(torch.isneginf(lse[:blind]))


@pytest.mark.parametrize("new", [1, 64])
def test_large_scores_and_outliers(new):
    # one key far above the others (an attention sink), and queries that make the softmax nearly one-hot
    b = Batch(n=4, m=2, d=128, dtype="f16", news=[new], lens=[700], page=16, seed=3, q_scale=12.0)
    pg, off = KO.slot(b.table, 16, 0, 2)
    b.pk[pg, off] *= 6
    b.pages.k.copy_(b.pk)
    b.run_and_check()


@pytest.mark.parametrize("new", [1, 200])
def test_rising_scores_move_the_running_maximum(new):
    # each later key scores higher, so that the running maximum moves with every tile
    b = Batch(n=2, m=1, d=64, dtype="bf16", news=[new], lens=[900], page=32, seed=4)
    ramp = torch.linspace(0, 40, 900)
    u = torch.ones(64)
    for t in range(900):
        pg, off = KO.slot(b.table, 32, 0, t)
        b.pk[pg, off, 0] = (u * ramp[t] / 8 + b.pk[pg, off, 0].float() * 0.1).to(torch.bfloat16)
    b.q = (b.q.float() * 0.1 + 1).to(torch.bfloat16)
    b.qd = b.q.to(b.dev)
    b.pages.k.copy_(b.pk)
    b.run_and_check()


@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("f16", 5), ("bf16", 33), ("f16", 300)])
def test_long_caches(dtype, new):
    b = Batch(n=8, m=2, d=128, dtype=dtype, news=[new, 1], lens=[20011, 4097], page=64, seed=5, q_scale=2.0)
    out, lse = b.attend()
    b.layer.check_device()
    b.check_sampled(out, lse, sorted({0, new // 2, new - 1, new}), [0, 3, 7])


def test_mixed_chunk_and_decodes():
    news = [260, 1, 1, 7, 1, 90, 1, 1]
    lens = [1000, 1, 3000, 70, 515, 90, 129, 2000]
    b = Batch(n=8, m=2, d=128, dtype="bf16", news=news, lens=lens, page=16, seed=6, q_scale=2.0)
    out, lse = b.attend()
    b.layer.check_device()
    b.check_sampled(out, lse, [0, 100, 259, 260, 261, 262, 268, 269, 270, 300, 359, 360, 361], [0, 2, 5, 7])


@pytest.mark.parametrize("new", [1, 100])
def test_loose_bounds_and_strided_queries(new):
    b = Batch(n=4, m=2, d=128, dtype="f16", news=[new, 1], lens=[350, 20], page=16, seed=7, max_new=new + 300,
              max_kv=352)
    wide = torch.full((b.N, 6, 128), float("nan"), dtype=torch.float16, device=b.dev)
    wide[:, :4] = b.qd
    b.qd = wide[:, :4]
    b.run_and_check()


@pytest.mark.parametrize("new", [1, 30, 300])
def test_same_call_same_bits_and_clean_workspace(new):
    b = Batch(n=8, m=2, d=128, dtype="bf16", news=[new, 1, 2], lens=[5000, 3000, 40], page=16, seed=8)
    o1, l1 = b.attend()
    c = Batch(n=8, m=2, d=128, dtype="bf16", news=[1], lens=[777], page=16, seed=9)
    c.layer = b.layer                                     # another shape on the same handle in between
    c.run_and_check()
    for _ in range(5):
        o2, l2 = b.attend()
        assert torch.equal(o1, o2) and torch.equal(l1, l2)


@pytest.mark.parametrize("new", [1, 200])
def test_captured_call_replays_with_new_lengths(new):
    b = Batch(n=8, m=2, d=128, dtype="f16", news=[new, 1], lens=[2000, 900], page=16, seed=10)
    out = torch.zeros((b.N, 8, 128), dtype=torch.float16, device=b.dev)
    lse = torch.zeros((b.N, 8), dtype=torch.float32, device=b.dev)
    b.layer.attend(b.pages, b.rows, b.qd, out=out, lse=lse)   # loads the kernel before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.layer.attend(b.pages, b.rows, b.qd, out=out, lse=lse)
    for lens in ([2000, 900], [new, 1], [1500, 33]):
        b.rows.tensors[1].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref = Batch.oracle(b) if lens == b.lens else KO.attend(b.q.double().numpy(), b.pk.double().numpy(),
                                                               b.pv.double().numpy(), b.row_start, lens, b.table)
        b.check(out, lse, ref)
    b.layer.check_device()


def test_two_handles_on_two_streams():
    from rank_kv_cache_gb300 import palu as P
    a = Batch(n=8, m=2, d=128, dtype="f16", news=[1, 1], lens=[9000, 800], page=16, seed=11)
    b = Batch(n=8, m=2, d=128, dtype="f16", news=[150, 3], lens=[5000, 700], page=16, seed=12)
    ra, rb = a.attend(), b.attend()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        oa, ob = torch.empty_like(ra[0]), torch.empty_like(rb[0])
        la, lb = torch.empty_like(ra[1]), torch.empty_like(rb[1])
        torch.cuda.synchronize()
        a.layer.attend(a.pages, a.rows, a.qd, out=oa, lse=la, stream=sa)
        b.layer.attend(b.pages, b.rows, b.qd, out=ob, lse=lb, stream=sb)
        torch.cuda.synchronize()
        assert torch.equal(oa, ra[0]) and torch.equal(la, ra[1])
        assert torch.equal(ob, rb[0]) and torch.equal(lb, rb[1])


@pytest.mark.parametrize("new", [1, 40])
def test_shared_pages_and_other_rows_stay_apart(new):
    # two rows over one page table row (a shared prefix), a third with the same page twice
    b = Batch(n=4, m=2, d=64, dtype="f16", news=[new, new, new], lens=[128, 128, 128], page=16, seed=13)
    b.table[1] = b.table[0]
    b.table[2][:] = b.table[2][0]
    b.rows.tensors[2].copy_(torch.from_numpy(b.table))
    b.run_and_check()


@pytest.mark.parametrize("new", [1, 40])
def test_device_side_conditions_are_reported(new):
    from rank_kv_cache_gb300 import palu as P
    def fresh():
        return Batch(n=4, m=2, d=128, dtype="f16", news=[new, 1], lens=[100, 60], page=16, seed=14)

    def reported(b):
        b.attend()
        with pytest.raises(P.PaluError):
            b.layer.check_device()
        b.layer.check_device()

    b = fresh()
    b.rows.tensors[2][0, 2] = 10 ** 6                     # a page outside the pool
    reported(b)
    b = fresh()
    b.rows.tensors[2][1, 0] = -5
    reported(b)
    b = fresh()
    b.rows.tensors[1][0] = 10 ** 6                        # longer than the bound
    reported(b)
    b = fresh()
    b.rows.tensors[1][1] = -3
    reported(b)
    b = fresh()
    b.rows.tensors[0].copy_(torch.tensor([new, 0, 1], dtype=torch.int32))   # decreasing: the row is skipped
    reported(b)
    b = fresh()
    b.rows.tensors[0].copy_(torch.tensor([0, 1, 10 ** 6], dtype=torch.int32))
    reported(b)


def test_refusals():
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=4, m=2, d=64, dtype="f16", news=[2], lens=[20], page=16, seed=15)
    L, h, s = b.layer, b.layer.handle, torch.cuda.current_stream().cuda_stream
    p, r = b.pages.c_struct(), b.rows.c_struct()
    out = torch.zeros((2, 4, 64), dtype=torch.float16, device=b.dev)
    q, o = b.qd.data_ptr(), out.data_ptr()
    bad = P.PALU_ERR_INVALID_ARG
    assert P.palu_attend_kv(h, p, r, q, 256, o, None, s) == P.PALU_OK
    assert P.palu_attend_kv(h, p, r, q + 2, 256, o, None, s) == bad
    assert P.palu_attend_kv(h, p, r, q, 255, o, None, s) == bad
    assert P.palu_attend_kv(h, p, r, q, 260, o, None, s) == bad
    assert P.palu_attend_kv(h, p, r, q, 256, o + 8, None, s) == bad
    assert P.palu_attend_kv(h, p, r, q, 256, 0, None, s) == bad
    assert P.palu_attend_kv(h, p, r, q, 256, o, o + 2, s) == bad
    for field, value, status in (("n_pages", 0, bad), ("page_size", 0, bad), ("k", 0, bad), ("v", p.v + 8, bad),
                                 ("n_pages", 1 << 28, P.PALU_ERR_UNSUPPORTED)):
        x = P.palu_kv_pages(p.k, p.v, p.n_pages, p.page_size)
        setattr(x, field, value)
        assert P.palu_attend_kv(h, x, r, q, 256, o, None, s) == status, field
    for field, value, status in (("row_start", 0, bad), ("kv_len", 0, bad), ("batch", 2, bad), ("batch", -1, bad),
                                 ("n_tokens", 3, bad), ("n_tokens", -1, bad), ("max_new", -1, bad),
                                 ("max_kv_len", 33, bad), ("max_kv_len", -1, bad), ("table_pages", 0, bad)):
        x = P.palu_kv_rows()
        for f, _ in P.palu_kv_rows._fields_:
            setattr(x, f, getattr(r, f))
        setattr(x, field, value)
        assert P.palu_attend_kv(h, p, x, q, 256, o, None, s) == status, field
    with pytest.raises(ValueError):
        L.attend(b.pages, b.rows, b.qd, out=out.float())
    with pytest.raises(ValueError):
        L.attend(b.pages, b.rows, b.qd[:1])
    with pytest.raises(ValueError):
        L.attend(b.pages, b.rows, b.qd, lse=torch.zeros(2, 3, device=b.dev))
    f32 = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=64, dtype="f32", max_tokens=2)
    z = torch.zeros(2, 16, 2, 64, device=b.dev)
    with pytest.raises(P.PaluError):
        f32.attend(P.KVPages(z, z), b.rows, torch.zeros(2, 4, 64, device=b.dev))
    torch.cuda.synchronize()
    L.check_device()


@pytest.mark.parametrize("dtype,page,table", [("bf16", 16, True), ("f16", 200, False)])
def test_prompt_in_chunks_then_decode_steps(dtype, page, table):
    """Append and attend over two requests as a server runs them, against the oracle on the whole sequences."""
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(16)
    n, m, d, T = 8, 2, 128, 190
    full = [T, 150]
    qkv = [rounded(rng, (L, (n + 2 * m) * d), dtype) for L in full]
    wq, wk = rounded(rng, (d,), dtype).cuda(), rounded(rng, (d,), dtype).cuda()
    per = -(-T // page) if table else 1
    tab = rng.permutation(2 * per).reshape(2, per).astype(np.int32) if table else None
    n_pages = 2 * per if table else 2
    nan = torch.full((n_pages, page, m, d), float("nan"), dtype=TYPES[dtype]).cuda()
    pages = P.KVPages(nan, nan.clone())
    layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, max_batch=2, max_tokens=400)
    got = [[], []]
    queries = [[], []]
    done = [0, 0]
    for step in ((100, 0), (87, 147), (1, 1), (1, 1), (1, 1)):
        x = torch.cat([qkv[b][done[b]:done[b] + step[b]] for b in range(2)]).cuda()
        done = [done[b] + step[b] for b in range(2)]
        q, k, v = (x[:, a * d:e * d].unflatten(1, (e - a, d)) for a, e in ((0, n), (n, n + m), (n + m, n + 2 * m)))
        rows = P.KVRows(torch.tensor([0, step[0], sum(step)], dtype=torch.int32).cuda(),
                        torch.tensor(done, dtype=torch.int32).cuda(), n_tokens=sum(step), max_new=max(step),
                        max_kv_len=max(done), page_table=None if tab is None else torch.from_numpy(tab).cuda())
        qr = layer.append(pages, rows, k, v, q=q, q_weight=wq, k_weight=wk)
        o = layer.attend(pages, rows, qr)
        for b, part in enumerate(((0, step[0]), (step[0], sum(step)))):
            got[b].append(o[part[0]:part[1]])
            queries[b].append(qr[part[0]:part[1]])
    layer.check_device()
    assert done == full
    # the rotated queries and keys were checked on their own; here the oracle takes the stored ones
    b = Batch(n=n, m=m, d=d, dtype=dtype, news=full, lens=full, page=page, table=table, seed=17, slack=0)
    b.q = torch.cat([torch.cat(x) for x in queries]).cpu()
    b.pk, b.pv, b.table = pages.k.cpu(), pages.v.cpu(), tab
    ref = b.oracle()
    b.check(torch.cat([torch.cat(x) for x in got]), torch.from_numpy(ref[1]), ref)


def test_appended_sinks_and_window_feed_the_hybrid_decode():
    """The dense segment of a hybrid decode, filled by the append from unrotated keys, against the oracle."""
    from oracle import palu_oracle as O
    from rank_kv_cache_gb300 import palu as P
    from synthetic import gen
    from tests.gpu_cases import Case, assert_close
    T, D = 300, 68
    cfg = gen.ROPE_FP16.with_(T=T, batch=2)
    pos = np.stack([4 + np.arange(T)] * 2).astype(np.int32)
    q_pos = [4 + T + 63] * 2
    c = Case(cfg, positions=pos, q_pos=q_pos, max_position=T + D)
    n, d, dev = cfg.n_heads, cfg.head_dim, c.dev
    rng = np.random.default_rng(18)
    k, v = rounded(rng, (2 * D, n, d), "f32", 0.25), rounded(rng, (2 * D, n, d), "f32")
    dense_pos = np.concatenate([np.arange(4), 4 + T + np.arange(64)] * 2).astype(np.int32)
    nan = torch.full((2, D, n, d), float("nan"), dtype=torch.float16, device=dev)
    pages = P.KVPages(nan, nan.clone())
    layer = P.PagedAttention(n_heads=n, n_kv_heads=n, head_dim=d, dtype="f16", x_dtype="f32", rope_theta=cfg.theta,
                             max_batch=2, max_tokens=2 * D)
    full = torch.tensor([D, D], dtype=torch.int32, device=dev)
    rows = P.KVRows(torch.tensor([0, D, 2 * D], dtype=torch.int32, device=dev), full, n_tokens=2 * D, max_new=D,
                    max_kv_len=D, positions=torch.from_numpy(dense_pos).to(dev))
    layer.append(pages, rows, k.to(dev), v.to(dev))
    layer.check_device()
    posd = torch.from_numpy(pos).to(dev)
    out, out_d, lse = c.attn.decode_hybrid(c.q_t.to(dev), c.cache, torch.tensor([T, T], dtype=torch.int32, device=dev),
                                           pages.k, pages.v, full, max_seq_len=T, positions=posd,
                                           q_pos=torch.tensor(q_pos, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    c.attn.check_device()
    rk = KO.norm_rope(k.double().numpy(), None, dense_pos, cfg.theta, 0.0).reshape(2, D, n, d)
    ref_l, ref_d, ref_lse = O.decode_hybrid(c.q64, c.hk64, c.hv64, c.bk64, [T, T], cfg.group_size, rk,
                                           v.double().numpy().reshape(2, D, n, d), [D, D], theta=cfg.theta,
                                           positions=pos, q_pos=q_pos)
    # the stored keys' fp16 rounding moves a score by at most 2^-11 sum |q k| / sqrt(d), which the hybrid's bounds hold
    assert_close(out.cpu().double().numpy(), ref_l, lse.cpu().double().numpy(), ref_lse)
    assert_close(out_d.cpu().double().numpy(), ref_d)


@pytest.mark.parametrize("batch,new", [(33, 1), (100, 3), (1100, 1), (40, 17), (1100, 18)])
def test_many_rows(batch, new):
    # more rows than a warp's lanes (few-row cut) and than the plan's block, lengths from nothing to a few tiles
    rng = np.random.default_rng(batch)
    news = [int(x) for x in rng.integers(0, new + 1, batch)]
    news[0] = new
    lens = [int(max(n, x)) for n, x in zip(news, rng.integers(0, 300, batch))]
    Batch(n=2, m=2, d=64, dtype="f16", news=news, lens=lens, page=32, seed=batch, max_new=new).run_and_check()


def test_more_tiles_than_the_plan_weighs():
    # 4200 rows of 17 new tokens: a tile each, more than are weighed for cutting; spot checks
    news, lens = [17] * 4200, [17 + i % 40 for i in range(4200)]
    b = Batch(n=1, m=1, d=64, dtype="bf16", news=news, lens=lens, page=64, seed=21)
    out, lse = b.attend()
    b.layer.check_device()
    b.check_sampled(out, lse, [0, 16, 17 * 2049 + 5, 17 * 4199, 17 * 4200 - 1], [0])


@pytest.mark.parametrize("new,length", [(20, 9000), (200, 5000), (129, 700), (64, 30000)])
@pytest.mark.parametrize("n,m", [(2, 2), (8, 1), (6, 2)])
def test_long_rows_cut_into_many_pieces(new, length, n, m):
    b = Batch(n=n, m=m, d=128, dtype="bf16", news=[new], lens=[length], page=64, seed=new, q_scale=2.0)
    out, lse = b.attend()
    b.layer.check_device()
    b.check_sampled(out, lse, sorted({0, new // 3, new - 2, new - 1}), [0, n - 1])
    o2, l2 = b.attend()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_rows_that_overlap_in_the_packed_arrays_are_reported():
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=1, m=1, d=64, dtype="f16", news=[2048, 0, 0, 0], lens=[2048, 0, 0, 0], page=64, seed=22)
    b.rows.tensors[0].copy_(torch.tensor([0, 2048, 0, 2048, 0], dtype=torch.int32))   # rows 0 and 2 share the tokens
    b.attend()
    with pytest.raises(P.PaluError):
        b.layer.check_device()
    b.layer.check_device()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_bounded_waits_give_up_and_report_a_timeout(dtype, d):
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=4, m=2, d=d, dtype=dtype, news=[200, 20], lens=[900, 3000], page=16, seed=23)
    good = b.layer
    b.layer = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=d, dtype=dtype, max_batch=2, max_tokens=b.N,
                               flags=P.PALU_FLAG_TEST_STALL)
    b.attend()
    with pytest.raises(P.PaluError) as e:
        b.layer.check_device()
    assert e.value.status == P.PALU_ERR_TIMEOUT
    b.layer = good
    b.run_and_check()


def test_call_on_a_side_stream_allocates_there():
    b = Batch(n=4, m=2, d=128, dtype="f16", news=[1, 30], lens=[400, 90], page=16, seed=24)
    ref, _ = b.attend()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [b.layer.attend(b.pages, b.rows, b.qd, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_every_layer_of_a_step_on_one_handle_in_a_graph():
    """Append and attend of several layers, one handle and one set of rows, captured and replayed with new lengths."""
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(25)
    n, m, d, layers, B = 8, 2, 128, 3, 3
    dev = torch.device("cuda:0")
    layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype="bf16", max_batch=B, max_tokens=B)
    pages = [P.KVPages(*(rounded(rng, (B * 8, 16, m, d), "bf16").to(dev) for _ in range(2))) for _ in range(layers)]
    table = torch.from_numpy(rng.permutation(B * 8).reshape(B, 8).astype(np.int32)).to(dev)
    start, lens = torch.arange(B + 1, dtype=torch.int32, device=dev), torch.tensor([5, 60, 100], dtype=torch.int32, device=dev)
    rows = P.KVRows(start, lens, n_tokens=B, max_new=1, max_kv_len=128, page_table=table)
    x = [rounded(rng, (B, (n + 2 * m) * d), "bf16").to(dev) for _ in range(layers)]
    q_out = [torch.empty(B, n, d, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
    out = [torch.empty(B, n, d, dtype=torch.bfloat16, device=dev) for _ in range(layers)]

    def step():
        for i in range(layers):
            q, k, v = (x[i][:, a * d:e * d].unflatten(1, (e - a, d)) for a, e in ((0, n), (n, n + m), (n + m, n + 2 * m)))
            layer.append(pages[i], rows, k, v, q=q, q_out=q_out[i])
            layer.attend(pages[i], rows, q_out[i], out=out[i])

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for now in ([6, 61, 101], [128, 1, 17]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        for o in out:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for i in range(layers):
            o, s, size, reach = KO.attend(q_out[i].double().cpu().numpy(), pages[i].k.double().cpu().numpy(),
                                          pages[i].v.double().cpu().numpy(), [0, 1, 2, 3], now, table.cpu().numpy())
            b = Batch(n=n, m=m, d=d, dtype="bf16", news=[1] * B, lens=now, page=16, seed=26)
            b.pv = pages[i].v.cpu()
            b.check(out[i], torch.from_numpy(s), (o, s, size, reach))
    layer.check_device()


@pytest.mark.parametrize("n,m", [(8, 1), (6, 3)])
def test_cut_rows_behind_the_first_32(n, m):
    # the join finds its rows 32 at a time: long ones first, in the second 32 and last
    news, lens = [3] * 70, [40 + i for i in range(70)]
    for b in (1, 37, 69):
        news[b], lens[b] = 40, 9000 + b
    b = Batch(n=n, m=m, d=128, dtype="bf16", news=news, lens=lens, page=64, seed=26)
    out, lse = b.attend()
    b.layer.check_device()
    at = np.concatenate([[0], np.cumsum(news)])
    b.check_sampled(out, lse, [int(at[x]) + y for x in (1, 37, 69) for y in (0, 39)] + [int(at[36])], [0, n - 1])
    o2, l2 = b.attend()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_cut_calls_side_by_side():
    """Two handles' calls whose pieces both wait for the join, on two streams at once."""
    a = Batch(n=8, m=2, d=128, dtype="bf16", news=[64], lens=[20000], page=64, seed=27)
    b = Batch(n=8, m=8, d=64, dtype="f16", news=[300, 20], lens=[6000, 9000], page=16, seed=28)
    ra, rb = a.attend(), b.attend()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for _ in range(20):
        oa, ob = torch.empty_like(ra[0]), torch.empty_like(rb[0])
        la, lb = torch.empty_like(ra[1]), torch.empty_like(rb[1])
        torch.cuda.synchronize()
        for _ in range(5):
            a.layer.attend(a.pages, a.rows, a.qd, out=oa, lse=la, stream=sa)
            b.layer.attend(b.pages, b.rows, b.qd, out=ob, lse=lb, stream=sb)
        outs.append((oa, la, ob, lb))
    torch.cuda.synchronize()
    a.layer.check_device()
    b.layer.check_device()
    for oa, la, ob, lb in outs:
        assert torch.equal(oa, ra[0]) and torch.equal(la, ra[1])
        assert torch.equal(ob, rb[0]) and torch.equal(lb, rb[1])


@pytest.mark.parametrize("n,m,d,batch,new,extra", [(32, 32, 128, 11, 400, 0), (24, 8, 128, 9, 700, 900), (8, 8, 64, 27, 830, 0),
                                                   (28, 4, 64, 17, 600, 1), (32, 8, 128, 12, 40, 2000)])
def test_many_items_a_cta_give_the_same_bits_every_time(n, m, d, batch, new, extra):
    """Items follow each other on a CTA while a unit of the one before still runs: repeated calls agree bit for bit, and
    with float64 on a sample."""
    news = [new - i % 5 for i in range(batch)]
    b = Batch(n=n, m=m, d=d, dtype="bf16", news=news, lens=[x + extra for x in news], page=32, seed=29)
    ref, ref_lse = b.attend()
    at = np.concatenate([[0], np.cumsum(news)])
    b.check_sampled(ref, ref_lse, [int(at[x]) for x in (0, batch // 2)] + [int(at[batch]) - 1], [0, n - 1])
    diff = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        out, lse = b.attend()
        diff += (out != ref).sum() + (lse != ref_lse).sum()
    b.layer.check_device()
    assert int(diff) == 0


def test_a_handle_made_on_a_side_stream():
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=4, m=2, d=128, dtype="f16", news=[1, 30], lens=[400, 2000], page=16, seed=30)
    ref, _ = b.attend()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    layer = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=128, dtype="f16", max_batch=2, max_tokens=b.N, stream=s)
    out = layer.attend(b.pages, b.rows, b.qd, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    layer.check_device(s)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("table", [True, False])
def test_pools_past_32_bit_offsets(new, table):
    """Pages at both ends of a pool of over 2^32 elements: the same bits, written and read, as from a small pool."""
    from rank_kv_cache_gb300 import palu as P
    rng, dev = np.random.default_rng(31), torch.device("cuda:0")
    n, m, d, B, L = 16, 8, 128, 2, 300
    page, small = (64, 12) if table else (L + 20, B)
    far = 2 ** 32 // (m * d * 64) + 40 if table else B
    wide = 64 if table else 2 ** 32 // (m * d) + 64                     # without a table row 1 is page 1
    ids = torch.tensor([far - 1 - i if i % 2 else i for i in range(small)]) if table else torch.arange(B)
    pools = []
    for pages, size in ((small, page), (far, wide)):
        pools.append(P.KVPages(*(torch.empty(pages, size, m, d, dtype=torch.bfloat16, device=dev) for _ in range(2))))
    for name in ("k", "v"):
        x = rounded(rng, (small, page, m, d), "bf16").to(dev)
        getattr(pools[0], name).copy_(x)
        getattr(pools[1], name)[ids.to(dev), :page] = x
    layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype="bf16", max_batch=B, max_tokens=B * new)
    start = torch.arange(0, B * new + 1, new, dtype=torch.int32, device=dev)
    lens = torch.tensor([L, L - 7], dtype=torch.int32, device=dev)
    order = torch.from_numpy(rng.permutation(small)[:B * 5].reshape(B, 5)) if table else None
    q, k, v = (rounded(rng, (B * new, h, d), "bf16").to(dev) for h in (n, m, m))
    got = []
    for pool, where in zip(pools, (None, ids)):
        t = None if order is None else (order if where is None else where[order]).int().to(dev)
        rows = P.KVRows(start, lens, n_tokens=B * new, max_new=new, max_kv_len=L, page_table=t)
        lse = torch.empty(B * new, n, dtype=torch.float32, device=dev)
        q_rot = layer.append(pool, rows, k, v, q=q)
        got.append((q_rot, layer.attend(pool, rows, q_rot, lse=lse), lse))
    layer.check_device()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for name in ("k", "v"):
        assert torch.equal(getattr(pools[0], name), getattr(pools[1], name)[ids.to(dev), :page])
