"""GPU tests of the attention over the 8-bit cache where a score's factor, a query row's own power of two times a block's scale, leaves
fp32's range: queries next to nothing against blocks of zero keys (whose scale is the least, 2^-64), and queries and scales next to
the largest, whose products are zero."""
import numpy as np
import pytest
import torch

from tests.kv8_cases import Batch8
from tests.kv_cases import TYPES
from tests.test_gpu_kv8_pairs import Wide

pytestmark = pytest.mark.gpu

# each kernel: one to three eights of query rows on the streaming one, single CTAs and pairs on the other
KERNELS = [(Batch8, dict(n=8, d=128, news=[2, 1], lens=[300, 77])), (Batch8, dict(n=8, d=128, news=[3, 2], lens=[301, 16])),
           (Wide, dict(n=8, d=128, news=[6, 1], lens=[333, 40])), (Batch8, dict(n=8, d=64, news=[4, 3], lens=[300, 77])),
           (Batch8, dict(n=4, d=64, news=[70, 1], lens=[300, 77])), (Batch8, dict(n=4, d=128, news=[70, 1], lens=[700, 77])),
           (Wide, dict(n=8, d=128, news=[120, 3], lens=[700, 3]))]


def _used(b, side):
    return b.codes[side] & 0x7f != 0x7f


@pytest.mark.parametrize("kind,kw", KERNELS)
@pytest.mark.parametrize("q_scale", [2.0 ** -66, 2.0 ** -80, 2.0 ** -110])
@pytest.mark.parametrize("every", [1, 2])
def test_queries_next_to_nothing_and_zero_keys(cuda_device, kind, kw, q_scale, every):
    b = kind(m=2, dtype="bf16", page=16, seed=1, q_scale=q_scale, **kw)
    codes, scales = b.codes[0], b.scales[0]
    codes[_used(b, 0) & (np.arange(len(codes)) % every == 0)[:, None, None, None]] = 0   # pages, which are blocks here
    scales[::every][np.isfinite(scales[::every])] = 2.0 ** -64
    b.renew()
    b.run_and_check()


@pytest.mark.parametrize("kind,kw", KERNELS)
@pytest.mark.parametrize("q_scale,scale", [(2.0 ** 120, 2.0 ** 64), (2.0 ** 85, 2.0 ** 64), (2.0 ** 120, 2.0 ** 20)])
def test_products_of_zero_under_the_largest_scales(cuda_device, kind, kw, q_scale, scale):
    b = kind(m=2, dtype="bf16", page=16, seed=2, q_scale=q_scale, **kw)
    b.q[..., 0] = 0                                                          # the keys have nothing but this element
    b.qd.copy_(b.q)
    assert b.q.dtype == TYPES["bf16"] and bool(torch.isfinite(b.q).all())
    codes = b.codes[0]
    used = _used(b, 0)
    codes[used] = 0
    codes[:, ::5, :, 0] = np.where(used[:, ::5, :, 0], 0x7e, codes[:, ::5, :, 0])
    b.scales[0][np.isfinite(b.scales[0])] = scale
    b.renew()
    b.run_and_check()
