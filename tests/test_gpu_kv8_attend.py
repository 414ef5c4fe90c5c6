"""GPU tests of the attention over the 8-bit paged KV cache, on its streaming and its tensor-core kernel."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8
from tests.kv8_cases import Batch8

pytestmark = pytest.mark.gpu

SHAPES = [(8, 2, 128, "bf16"), (4, 4, 64, "f16"), (6, 1, 128, "f16"), (7, 7, 64, "bf16"), (16, 1, 64, "bf16")]


@pytest.mark.parametrize("n,m,d,dtype", SHAPES)
@pytest.mark.parametrize("lens", [[1], [16], [17, 1, 300], [128, 129, 255, 511], [1000, 33]])
def test_single_tokens(cuda_device, n, m, d, dtype, lens):
    Batch8(n=n, m=m, d=d, dtype=dtype, news=[1] * len(lens), lens=lens, page=16, seed=sum(lens)).run_and_check()


@pytest.mark.parametrize("n,m,d,dtype", SHAPES)
@pytest.mark.parametrize("news,lens", [([1, 40], [1, 40]), ([130], [130]), ([3, 0, 257], [300, 17, 300]),
                                       ([64, 1, 1, 1], [700, 1300, 15, 128]), ([20, 33], [2100, 33])])
def test_many_tokens(cuda_device, n, m, d, dtype, news, lens):
    Batch8(n=n, m=m, d=d, dtype=dtype, news=news, lens=lens, page=16, seed=sum(lens) + d).run_and_check()


@pytest.mark.parametrize("news", [1, 2, 4, 5, 17])
@pytest.mark.parametrize("page,table", [(16, True), (48, True), (128, True), (256, True), (416, False)])
def test_page_sizes_and_contiguous_caches(cuda_device, news, page, table):
    Batch8(n=8, m=2, d=128, dtype="bf16", news=[news, 1, news], lens=[400, 37, 129 + news], page=page, table=table,
           seed=page + news).run_and_check()


@pytest.mark.parametrize("news", [1, 24])
@pytest.mark.parametrize("kw", [dict(spread=12.0), dict(pow2=False), dict(q_scale=2.0 ** 12, k_scale=2.0 ** -14),
                                dict(q_scale=2.0 ** -12, k_scale=2.0 ** 12), dict(q_scale=8.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales_far_apart_and_of_any_size(cuda_device, news, kw, dtype):
    for d in (64, 128):
        Batch8(n=4, m=2, d=d, dtype=dtype, news=[news, 1], lens=[500, 260], page=32, seed=news + d, **kw).run_and_check()


@pytest.mark.parametrize("news", [1, 40])
def test_bf16_queries_past_the_range_of_fp16(cuda_device, news):
    Batch8(n=4, m=2, d=128, dtype="bf16", news=[news, 2], lens=[300, 70], page=16, seed=news, q_scale=2.0 ** 40,
           k_scale=2.0 ** -40, spread=0.5).run_and_check()


@pytest.mark.parametrize("news", [1, 30])
def test_rows_of_zero_queries_and_equal_keys(cuda_device, news):
    b = Batch8(n=4, m=2, d=64, dtype="f16", news=[news, 1], lens=[200, 64], page=16, seed=7)
    b.q.zero_()
    b.qd.zero_()
    out, lse = b.run_and_check()
    assert torch.allclose(lse[-1].cpu(), torch.log(torch.tensor(64.0)), atol=1e-5)


@pytest.mark.parametrize("news", [[3, 1], [40, 1], [5, 60]])
def test_tokens_that_see_nothing_give_zero(cuda_device, news):
    # fewer cached than new tokens: the first of them see no slot
    b = Batch8(n=4, m=2, d=64, dtype="bf16", news=news, lens=[2, 1], page=16, seed=1, max_kv=16)
    b.run_and_check()


def test_tokens_of_no_row_and_empty_caches(cuda_device):
    for news in ([1, 0, 2], [30, 0, 2]):
        b = Batch8(n=4, m=2, d=128, dtype="f16", news=news, lens=[50, 9, 0], page=16, seed=3, extra_tokens=4, max_kv=64)
        b.run_and_check()


def test_long_tails_behind_large_scores_keep_their_weight(cuda_device):
    # seven keys 18 (natural) above 30000 others, and values of zero behind them: the tail is all of the output
    for news in (1, 20):
        b = Batch8(n=2, m=2, d=64, dtype="f16", news=[news], lens=[30000], page=64, seed=2, spread=0.0)
        b.q.zero_()
        b.q[..., 0] = 8.0
        b.qd = b.q.to(b.dev)
        first = b.table[0, 0]
        b.codes[0][:, :, :, 0] = 0
        b.codes[0][first, :7, :, 0] = K8.encode(np.array(18.0 * 2))           # 8 * 36 / 2 / sqrt(64) = 18
        b.codes[1][first, :7] = 0
        b.scales[0][...] = 1.0 / 16
        b.scales[0][first, 0] = 0.5
        b.renew()
        b.run_and_check()


def test_mixed_batches_cut_and_joined(cuda_device):
    rng = np.random.default_rng(11)
    for d, dtype in ((128, "bf16"), (64, "f16")):
        lens = [int(x) for x in rng.integers(1, 3000, 12)]
        news = [int(min(L, x)) for L, x in zip(lens, [70, 1, 1, 5, 200, 1, 1, 1, 33, 1, 1, 2])]
        Batch8(n=8, m=2, d=d, dtype=dtype, news=news, lens=lens, page=32, seed=d).run_and_check()


def test_many_rows(cuda_device):
    rng = np.random.default_rng(12)
    for most in (1, 30):
        lens = [int(x) for x in rng.integers(1, 400, 70)]
        news = [int(min(L, x)) for L, x in zip(lens, rng.integers(0, most + 1, 70))]
        Batch8(n=4, m=1, d=64, dtype="bf16", news=news, lens=lens, page=16, seed=most, max_new=most).run_and_check()


@pytest.mark.parametrize("news", [1, 5])
def test_long_rows(cuda_device, news):
    b = Batch8(n=8, m=2, d=128, dtype="bf16", news=[news, 1], lens=[20000, 9000], page=64, seed=news)
    out, lse = b.attend()
    b.layer.check_device()
    b.check_sampled(out, lse, [0, news - 1, news], [0, 3, 7])


def test_the_same_call_gives_the_same_bits(cuda_device):
    for news in (1, 60):
        b = Batch8(n=8, m=2, d=128, dtype="bf16", news=[news, 1, 1], lens=[5000, 700, 2900], page=16, seed=4)
        a = b.attend()
        for _ in range(5):
            c = b.attend()
            assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_strided_queries_and_no_lse(cuda_device):
    for news in (2, 40):
        b = Batch8(n=4, m=2, d=128, dtype="bf16", news=[news, 1], lens=[300, 90], page=16, seed=news)
        want, _ = b.run_and_check()
        wide = torch.zeros(b.N, 6 * 128 + 8, dtype=torch.bfloat16, device="cuda")
        q = wide[:, 8:8 + 4 * 128].unflatten(1, (4, 128))
        q.copy_(b.qd)
        assert torch.equal(b.layer.attend(b.pages, b.rows, q), want)


def test_device_side_conditions_are_reported(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    for news in (1, 30):
        b = Batch8(n=4, m=2, d=64, dtype="f16", news=[news, 1], lens=[100, 50], page=16, seed=5)
        good = b.attend()
        b.rows.tensors[2][0, 2] = -3                                          # read as zeros
        b.attend()
        with pytest.raises(P.PaluError):
            b.layer.check_device()
        b.rows.tensors[2].copy_(torch.from_numpy(b.table))
        b.rows.tensors[1].copy_(torch.tensor([100, 5000], dtype=torch.int32))
        b.attend()
        with pytest.raises(P.PaluError):
            b.layer.check_device()
        b.rows.tensors[1].copy_(torch.tensor([100, 50], dtype=torch.int32))
        again = b.attend()
        b.layer.check_device()
        assert torch.equal(good[0], again[0])


def test_bounded_waits_give_up_and_report_a_timeout(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    b = Batch8(n=4, m=2, d=128, dtype="bf16", news=[40], lens=[300], page=16, seed=6, flags=P.PALU_FLAG_TEST_STALL)
    b.attend()
    with pytest.raises(P.PaluError) as e:
        b.layer.check_device()
    assert e.value.status == P.PALU_ERR_TIMEOUT
    Batch8(n=4, m=2, d=128, dtype="bf16", news=[40], lens=[300], page=16, seed=6).run_and_check()


def test_graphs_streams_and_two_handles(cuda_device):
    for news in (1, 40):
        x = Batch8(n=4, m=2, d=128, dtype="f16", news=[news, 1], lens=[900, 70], page=16, seed=1)
        y = Batch8(n=4, m=2, d=128, dtype="f16", news=[news, 1], lens=[900, 70], page=16, seed=2)
        want = [b.attend() for b in (x, y)]
        outs = [torch.zeros_like(x.qd), torch.zeros_like(y.qd)]
        graphs = []
        for b, o in zip((x, y), outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                b.layer.attend(b.pages, b.rows, b.qd, out=o)
            graphs.append(g)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w[0])
        # lengths change between replays
        x.rows.tensors[1].copy_(torch.tensor([300, 20], dtype=torch.int32))
        graphs[0].replay()
        torch.cuda.synchronize()
        z, _ = x.attend()
        assert torch.equal(outs[0], z)


def test_codes_of_every_value(cuda_device):
    # a first token sees itself alone: its codes come back, every finite one, exactly
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    for news in (1, 17):
        for part in range(4):
            b = Batch8(n=1, m=1, d=64, dtype="f16", news=[news], lens=[news], page=16, seed=0, spread=0.0)
            first = b.table[0, 0]
            b.codes[1][first, 0, 0] = np.resize(codes[64 * part:64 * part + 64], 64)
            b.scales[1][first] = 2.0 ** -3
            b.renew()
            out, _ = b.run_and_check()
            assert torch.equal(out[0, 0].double().cpu(), b.pv[first, 0, 0])
