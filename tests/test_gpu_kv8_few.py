"""GPU tests of the 8-bit cache's streaming attention where 13 to 24 query rows share a key/value head: by bounds that promise much
work (page tables far longer than the rows) on the streaming kernel, by the rows' own on the other."""
import pytest
import torch

from rank_kv_cache_gb300 import palu as P
from tests.kv8_cases import Batch8
from tests.test_gpu_kv8_pairs import Wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [Wide, Batch8])
@pytest.mark.parametrize("n,m,d,dtype,new", [(8, 2, 128, "bf16", 5), (8, 2, 128, "f16", 6), (4, 4, 64, "f16", 17), (4, 4, 128, "bf16", 24),
                                             (6, 1, 128, "f16", 3), (7, 7, 64, "bf16", 20), (16, 1, 64, "bf16", 1), (12, 4, 128, "bf16", 8),
                                             (23, 1, 128, "f16", 1), (13, 1, 128, "bf16", 1)])
@pytest.mark.parametrize("lens", [[25], [300, 24, 1000], [129, 4000]])
def test_rows_of_two_and_three_eights(cuda_device, kind, n, m, d, dtype, new, lens):
    news = [min(new, L) for L in lens]
    news[-1] = max(1, news[-1] - 1)                                            # ragged; the most is `new`
    news[0] = min(new, lens[0])
    kind(n=n, m=m, d=d, dtype=dtype, news=news, lens=lens, page=16, seed=sum(lens) + n, max_new=new).run_and_check()


@pytest.mark.parametrize("page", [48, 128, 256])
def test_pages(cuda_device, page):
    Wide(n=8, m=2, d=128, dtype="bf16", news=[6, 5], lens=[700, 257], page=page, seed=page).run_and_check()


@pytest.mark.parametrize("kw", [dict(spread=12.0), dict(pow2=False), dict(q_scale=2.0 ** 100, k_scale=2.0 ** -100)])
def test_scales(cuda_device, kw):
    Wide(n=8, m=2, d=128, dtype="bf16", news=[6], lens=[500], page=16, seed=3, **kw).run_and_check()


def test_rows_that_see_nothing_and_tokens_of_no_row(cuda_device):
    b = Wide(n=8, m=2, d=128, dtype="f16", news=[6, 5], lens=[2, 40], page=16, seed=4, extra_tokens=3)
    out, lse = b.run_and_check()
    assert not out[:4].any() and bool(torch.isneginf(lse[:4]).all())


def test_many_and_long_rows(cuda_device):
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[6, 1, 5, 4] * 10, lens=[100 + 37 * i for i in range(40)], page=16, seed=5)
    b.run_and_check()
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[6], lens=[30000], page=64, seed=6)
    out, lse = b.run_and_check()
    for _ in range(3):
        again, again_lse = b.attend()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_both_kernels_in_one_graph(cuda_device):
    """The same rows by a far bound and by their own, one behind the other."""
    b = Wide(n=8, m=2, d=128, dtype="bf16", news=[6, 4], lens=[1000, 90], page=16, seed=7)
    start, lens, table, _ = b.rows.tensors
    near = P.KVRows(start, lens, page_table=table, n_tokens=b.N, max_new=6, max_kv_len=1000)
    outs = [torch.empty_like(b.qd) for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, rows in enumerate((b.rows, near, b.rows, near)):
            b.layer.attend(b.pages, rows, b.qd, out=outs[i])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    _, lse = b.run_and_check()
    for out in outs[:2]:
        b.check(out, lse, b.oracle())
