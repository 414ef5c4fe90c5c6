"""GPU tests of the paged KV cache's calls at the corners of what the header allows: addresses, score ranges, batches
of many rows, far positions, bounds that the rows break, and a window that rolls."""
import numpy as np
import pytest
import torch

from tests.kv_cases import TYPES, Batch, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    return cuda_device


def _at_16(t):
    """A copy of t whose address is 16 modulo 32."""
    pad = 16 // t.element_size()
    buf = torch.empty(t.numel() + 2 * pad, dtype=t.dtype, device=t.device)
    x = buf[pad if buf.data_ptr() % 32 == 0 else 0:][:t.numel()].view(t.shape)
    x.copy_(t)
    assert x.data_ptr() % 32 == 16
    return x


@pytest.mark.parametrize("dtype,d,n,m", [("f16", 128, 4, 2), ("bf16", 64, 7, 1), ("bf16", 128, 6, 2)])
@pytest.mark.parametrize("news,lens", [([1, 1], [300, 17]), ([40, 3], [90, 200]), ([40, 200], [9000, 5000])])
def test_outputs_and_queries_at_16_modulo_32(dtype, d, n, m, news, lens):
    # one token (the streaming kernel), whole tiles and cut ones (the tensor-core kernel's two ways to its output)
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=n, m=m, d=d, dtype=dtype, news=news, lens=lens, page=16, seed=40)
    ref, ref_lse = b.attend()
    b.check_sampled(ref, ref_lse, [0, news[0] - 1, b.N - 1], [0, n - 1])
    q = _at_16(b.qd)
    pages = P.KVPages(_at_16(b.pages.k), _at_16(b.pages.v))
    out = _at_16(torch.full_like(ref, 7.0))
    lse = torch.empty_like(ref_lse)
    b.layer.attend(pages, b.rows, q, out=out, lse=lse)
    b.layer.check_device()
    # the address changes how the output is stored, not what is computed
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
