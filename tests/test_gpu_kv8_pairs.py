"""GPU tests of the attention over the 8-bit cache by pairs of CTAs (heads of 128, much work by the call's bounds), at sizes where it
can go wrong: the calls here have page tables, and bounds, far longer than their rows."""
import pytest
import torch

from rank_kv_cache_gb300 import palu as P
from tests.kv8_cases import Batch8

pytestmark = pytest.mark.gpu

FAR = 1 << 19       # cached tokens by the bound: steps enough for 76 pairs, whatever the rows


class Wide(Batch8):
    """Rows over a page table for FAR tokens, whose entries behind their own are no page."""

    def __init__(self, **kw):
        super().__init__(**kw)
        start, lens, table, _ = self.rows.tensors
        wide = torch.full((len(self.lens), -(-FAR // self.page)), 1 << 30, dtype=torch.int32, device=self.dev)
        wide[:, :table.shape[1]] = table
        self.rows = P.KVRows(start, lens, page_table=wide, n_tokens=self.N, max_new=self.rows.max_new, max_kv_len=FAR)


# query rows of a key/value head: pairs take averages whose last 512 are more than half full
@pytest.mark.parametrize("n,m,dtype", [(8, 2, "bf16"), (4, 4, "f16"), (6, 1, "f16"), (7, 1, "bf16"), (3, 3, "bf16")])
@pytest.mark.parametrize("rows,at", [(384, 0), (510, 0), (300, 1), (430, 2000), (1800, 77)])
@pytest.mark.parametrize("page", [16, 48])
def test_one_prompt_or_chunk(cuda_device, n, m, dtype, rows, at, page):
    new = -(-rows // (n // m))
    Wide(n=n, m=m, d=128, dtype=dtype, news=[new], lens=[new + at], page=page, seed=rows + at).run_and_check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("news,lens", [([1, 200], [300, 200]), ([130, 0, 257, 1], [130, 40, 900, 2000]),
                                       ([64, 300, 1, 127, 129, 128], [700, 1300, 15, 128, 129, 3000]),
                                       ([400, 2], [450, 4000]), ([110] * 40, [110 + 13 * i for i in range(40)])])
def test_batches(cuda_device, news, lens, dtype):
    Wide(n=8, m=2, d=128, dtype=dtype, news=news, lens=lens, page=32, seed=len(news)).run_and_check()


@pytest.mark.parametrize("page", [64, 80, 128, 256, 1024])
def test_pages_that_end_inside_and_behind_a_tile(cuda_device, page):
    Wide(n=8, m=2, d=128, dtype="bf16", news=[100, 96], lens=[1111, 96], page=page, seed=page).run_and_check()


def test_contiguous_caches(cuda_device):
    Batch8(n=8, m=8, d=128, dtype="f16", news=[300, 400], lens=[5000, 400], page=40960, max_kv=40960, table=False, seed=3).run_and_check()


@pytest.mark.parametrize("kw", [dict(spread=12.0), dict(pow2=False), dict(q_scale=2.0 ** 12, k_scale=2.0 ** -14),
                                dict(q_scale=2.0 ** 100, k_scale=2.0 ** -100)])
def test_scales_far_apart_and_of_any_size(cuda_device, kw):
    Wide(n=8, m=2, d=128, dtype="bf16", news=[120], lens=[700], page=16, seed=11, **kw).run_and_check()


def test_tokens_that_see_nothing_give_zero(cuda_device):
    """More new tokens than cached ones: the first see no slot."""
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[100, 150], lens=[60, 150], page=16, seed=5)
    out, lse = b.run_and_check()
    assert not out[:40].any() and bool(torch.isneginf(lse[:40]).all())


def test_tokens_of_no_row_are_left(cuda_device):
    Wide(n=8, m=2, d=128, dtype="f16", news=[100, 101], lens=[333, 101], page=16, seed=6, extra_tokens=37).run_and_check()


def test_cut_rows_are_joined(cuda_device):
    """A few long rows, whose pieces all pairs share, beside short ones."""
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[100, 70, 128], lens=[20000, 500, 9000], page=64, seed=8)
    out, lse = b.run_and_check()
    for _ in range(3):
        again, again_lse = b.attend()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_many_items_a_pair_give_the_same_bits_every_time(cuda_device):
    b = Wide(n=32, m=16, d=128, dtype="f16", news=[450] * 6, lens=[450 + 90 * i for i in range(6)], page=32, seed=9)
    out, lse = b.attend()
    for _ in range(5):
        again, again_lse = b.attend()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)
    b.layer.check_device()


def test_a_query_that_is_not_a_number_stays_by_itself(cuda_device):
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[120], lens=[600], page=16, seed=10)
    want, _ = b.run_and_check()
    b.qd[77, 3, 5] = float("nan")
    got, _ = b.attend()
    assert torch.isnan(got[77, 3]).all()
    got[77, 3] = want[77, 3]
    assert torch.equal(got, want)


def test_pairs_and_single_ctas_agree_within_the_bounds_of_both(cuda_device):
    """The same rows by a bound that is theirs and by one that is far, captured one behind the other, over and over."""
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[56, 200], lens=[1000, 200], page=16, seed=12)
    start, lens, table, _ = b.rows.tensors
    tight = P.KVRows(start, lens, page_table=table, n_tokens=b.N, max_new=200, max_kv_len=1000)
    outs = [torch.empty_like(b.qd) for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, rows in enumerate((b.rows, tight, tight, b.rows)):
            b.layer.attend(b.pages, rows, b.qd, out=outs[i])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[3]) and torch.equal(outs[1], outs[2])
    _, lse = b.run_and_check()
    for out in outs[:2]:
        b.check(out, lse, b.oracle())


def test_bad_pages_and_lengths_are_reported(cuda_device):
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[125], lens=[900], page=16, seed=13)
    want, _ = b.run_and_check()
    b.rows.tensors[2][0, 3] = 1 << 20                                          # slots 48 .. 63: no page, read as zeros
    got, _ = b.attend()
    with pytest.raises(P.PaluError):
        b.layer.check_device()
    assert torch.isfinite(got.float()).all() and not torch.equal(got, want)
    b.layer.check_device()


def test_bounded_waits_give_up_and_report_a_timeout(cuda_device):
    b = Wide(n=8, m=2, d=128, dtype="f16", news=[125], lens=[900], page=16, seed=14, flags=P.PALU_FLAG_TEST_STALL)
    b.attend()
    with pytest.raises(P.PaluError) as e:
        b.layer.check_device()
    assert e.value.status == P.PALU_ERR_TIMEOUT
    plain = Wide(n=8, m=2, d=128, dtype="f16", news=[125], lens=[900], page=16, seed=14)
    plain.run_and_check()


def test_two_calls_at_once_on_streams_of_their_own(cuda_device):
    """Pairs of two calls, cut and joined, that share the GPU."""
    batches = [Wide(n=8, m=2, d=128, dtype="bf16", news=[100, 70, 128], lens=[20000, 500, 9000], page=64, seed=21),
               Wide(n=32, m=8, d=128, dtype="f16", news=[120, 100], lens=[9000, 30000], page=32, seed=22)]
    want = [b.attend() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[], []]
    for _ in range(8):
        for b, s, g in zip(batches, streams, got):
            g.append(b.layer.attend(b.pages, b.rows, b.qd, stream=s))
    torch.cuda.synchronize()
    for b, w, g in zip(batches, want, got):
        b.layer.check_device()
        assert all(torch.equal(w[0], x) for x in g)
