"""GPU tests of the quantising append into the 8-bit paged KV cache."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8
from tests.kv8_cases import Appended

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,x_dtype,d,n,m,norm", [
    ("bf16", "bf16", 128, 8, 2, True), ("f16", "f32", 64, 3, 3, False), ("f16", "f16", 128, 4, 4, False),
    ("bf16", "f32", 64, 6, 1, True), ("bf16", "f16", 128, 5, 5, True), ("f16", "bf16", 64, 2, 2, False)])
@pytest.mark.parametrize("news,lens", [
    ([1], [1]), ([1, 1, 1], [1, 16, 17]), ([5, 1, 0, 16], [5, 40, 33, 16]), ([37, 3], [37, 130]), ([100, 17, 1], [129, 64, 96])])
def test_matches_the_oracle(cuda_device, dtype, x_dtype, d, n, m, norm, news, lens):
    a = Appended(n=n, m=m, d=d, dtype=dtype, x_dtype=x_dtype, news=news, lens=lens, page=16, norm=norm, seed=len(news) + d)
    a.run()
    a.check()


@pytest.mark.parametrize("page,table,news,lens", [
    (16, True, [20, 7], [150, 23]), (48, True, [20, 7], [150, 23]), (128, True, [20, 7], [150, 23]),
    (48, False, [20, 7], [45, 16]), (128, False, [20, 7], [45, 127])])
def test_page_sizes_and_contiguous_caches(cuda_device, page, table, news, lens):
    a = Appended(n=4, m=2, d=128, dtype="bf16", x_dtype="bf16", news=news, lens=lens, page=page, table=table, seed=page)
    a.run()
    a.check()


def test_token_by_token_is_as_the_oracle_step_by_step(cuda_device):
    # each step's scale is at least the block's so far: larger tokens restate the older codes
    from rank_kv_cache_gb300 import palu as P
    a = Appended(n=2, m=2, d=64, dtype="f16", x_dtype="f32", news=[1, 1], lens=[20, 40], page=32, seed=5)
    rng = np.random.default_rng(6)
    for step in range(20):
        lens = [1 + step, 20 + step]
        rows = P.KVRows(a.rows.tensors[0], torch.tensor(lens, dtype=torch.int32, device="cuda"), page_table=a.rows.tensors[2],
                        n_tokens=2, max_new=1, max_kv_len=64)
        size = float(rng.choice([0.1, 1.0, 30.0]))
        k = torch.from_numpy(rng.standard_normal((2, 2, 64)).astype(np.float32) * size)
        v = torch.from_numpy(rng.standard_normal((2, 2, 64)).astype(np.float32) * size)
        a.layer.append(a.pages, rows, k.cuda(), v.cuda())
        torch.cuda.synchronize()
        K8.append(a.codes[1], a.scales[1], v.double().numpy(), a.row_start, lens, a.table)
        assert np.array_equal(a.pages.v.view(torch.uint8).cpu().numpy(), a.codes[1])
        assert np.array_equal(a.pages.v_scale.cpu().numpy(), a.scales[1])
    a.layer.check_device()


@pytest.mark.parametrize("x", [0.0, 1.0, 448.0, 449.0, 2.0 ** -70, 1e-40, 3e38, 2.0 ** 60 * 1.75, 2.0 ** 60 * 1.7500001])
def test_scales_at_their_borders(cuda_device, x):
    a = Appended(n=1, m=1, d=64, dtype="f16", x_dtype="f32", news=[1], lens=[1], page=16, theta=0.0, with_q=False)
    v = torch.zeros(1, 1, 64)
    v[0, 0, 3], v[0, 0, 4] = x, -x / 3
    a.layer.append(a.pages, a.rows, v.cuda(), v.cuda())
    torch.cuda.synchronize()
    K8.append(a.codes[1], a.scales[1], v.double().numpy(), a.row_start, [1], a.table)
    page = a.table[0, 0]
    for codes, scales in ((a.pages.k, a.pages.k_scale), (a.pages.v, a.pages.v_scale)):
        assert np.array_equal(codes.view(torch.uint8).cpu().numpy()[page, 0], a.codes[1][page, 0])
        assert np.array_equal(scales.cpu().numpy()[page], a.scales[1][page])


def test_non_finite_values_are_stored_as_said(cuda_device):
    a = Appended(n=1, m=1, d=64, dtype="f16", x_dtype="f32", news=[2], lens=[2], page=16, theta=0.0, with_q=False)
    v = torch.zeros(2, 1, 64)
    v[0, 0, 0], v[0, 0, 1], v[0, 0, 2] = float("nan"), 5.0, -7.0
    a.layer.append(a.pages, a.rows, v.cuda(), v.cuda())
    page = int(a.table[0, 0])
    codes = a.pages.v.view(torch.uint8).cpu().numpy()[page, 0, 0]
    assert a.pages.v_scale.cpu()[page, 0, 0] == 2.0 ** -6                     # of 7: NaN does not count
    assert codes[0] & 127 == 127 and np.array_equal(codes[1:3], K8.encode(np.array([5.0, -7.0]) * 64))
    v[0, 0, 0] = float("inf")
    a.layer.append(a.pages, a.rows, v.cuda(), v.cuda())
    codes = a.pages.v.view(torch.uint8).cpu().numpy()[page, 0, 0]
    assert a.pages.v_scale.cpu()[page, 0, 0] == 2.0 ** 64 and codes[0] == 0x7e


def test_positions_rotate_and_slots_place(cuda_device):
    a = Appended(n=2, m=2, d=128, dtype="bf16", x_dtype="bf16", news=[18, 2], lens=[21, 9], page=16, seed=3,
                 positions=[1000 * i - 5000 for i in range(20)])
    a.run()
    a.check()


def test_tokens_behind_the_rows_and_many_rows(cuda_device):
    rng = np.random.default_rng(8)
    news = [int(x) for x in rng.integers(0, 4, 200)]
    lens = [int(n + x) for n, x in zip(news, rng.integers(0, 40, 200))]
    a = Appended(n=2, m=1, d=64, dtype="bf16", x_dtype="bf16", news=news, lens=lens, page=16, seed=9, extra=5)
    a.run()
    a.check()


def test_bad_rows_and_pages_are_reported_and_others_stored(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    a = Appended(n=2, m=2, d=64, dtype="f16", x_dtype="f16", news=[2, 2], lens=[3, 20], page=16, seed=4)
    table = a.table.copy()
    a.rows.tensors[2][0, 0] = 10 ** 6                                        # outside the pool
    before = a.pages.k.view(torch.uint8).clone()
    a.run()
    with pytest.raises(P.PaluError):
        a.layer.check_device()
    ref_c, ref_s = a.codes[1].copy(), a.scales[1].copy()
    K8.append(ref_c, ref_s, a.v.double().numpy()[2:], np.array([0, 2]), [20], table[1:])
    assert np.array_equal(a.pages.v.view(torch.uint8).cpu().numpy(), ref_c)
    assert np.array_equal(a.pages.v_scale.cpu().numpy(), ref_s)
    assert 2 <= int((a.pages.k.view(torch.uint8) != before).any(-1).any(-1).sum()) <= 4   # two new, two older ones
    assert bool((a.q_out != 7.0).any())                                      # the queries come back all the same
    a.rows.tensors[2][0, 0] = int(table[0, 0])
    a.rows.tensors[1].copy_(torch.tensor([1, 20], dtype=torch.int32))        # fewer cached than new: slot -1
    a.run()
    with pytest.raises(P.PaluError):
        a.layer.check_device()
    a.rows.tensors[1].copy_(torch.tensor([3, 1000], dtype=torch.int32))      # past max_kv_len and the table
    a.run()
    with pytest.raises(P.PaluError):
        a.layer.check_device()
    a.layer.check_device()                                                    # cleared


def test_in_place_queries_graphs_and_streams(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    layer = P.PagedAttention(n_heads=4, n_kv_heads=2, head_dim=64, dtype="bf16", max_batch=2, max_tokens=8)
    pages = P.KVPages8.empty(4, 32, 2, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = P.KVRows(torch.tensor([0, 3, 8], **i32), torch.tensor([3, 30], **i32), page_table=torch.tensor([[2], [0]], **i32),
                    n_tokens=8, max_new=5, max_kv_len=32)
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(8, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    want = layer.append(pages, rows, k, v, q=q)
    ref = [t.clone() for t in (pages.k.view(torch.uint8), pages.v.view(torch.uint8))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qq = q.clone()
        layer.append(pages, rows, k, v, q=qq, q_out=qq)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qq, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(graph):
        layer.append(pages, rows, k, v, q=q, q_out=out)
    for t in (pages.k.view(torch.uint8), pages.v.view(torch.uint8), pages.k_scale, pages.v_scale):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    layer.check_device()
    assert torch.equal(out, want)
    # the first row's tokens begin their block, so it is as before; the second's have older ones, zeros by now
    for got, w in zip((pages.k.view(torch.uint8), pages.v.view(torch.uint8)), ref):
        assert torch.equal(got[2, :3], w[2, :3])
