"""CPU tests of the paged KV cache's entry points: descriptors and arguments are refused on the host, before any
CUDA call."""
import ctypes

import pytest

from rank_kv_cache_gb300 import palu as P


def _desc(**kw):
    base = dict(n_heads=32, n_kv_heads=8, head_dim=128, dtype=P.PALU_BF16, x_dtype=P.PALU_BF16, rope_theta=1e4,
                norm_eps=1e-6, max_batch=4, max_tokens=64, flags=0)
    base.update(kw)
    return P.palu_kv_desc(P.PALU_ABI_VERSION, *[base[f] for f, _ in P.palu_kv_desc._fields_[1:]])


@pytest.mark.parametrize("kw", [{}, dict(dtype=P.PALU_F16), dict(head_dim=64), dict(rope_theta=0.0),
                                dict(n_kv_heads=32), dict(n_heads=64, n_kv_heads=1), dict(dtype=P.PALU_F32),
                                dict(x_dtype=P.PALU_F32), dict(n_heads=7, n_kv_heads=7),
                                dict(flags=P.PALU_FLAG_TEST_STALL)])
def test_descriptors_accepted(kw):
    st, n = P.palu_kv_workspace_size(_desc(**kw))
    assert st == P.PALU_OK and n > 0 and n % 256 == 0


@pytest.mark.parametrize("kw,status", [
    (dict(n_heads=0), P.PALU_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), P.PALU_ERR_INVALID_ARG),
    (dict(n_kv_heads=5), P.PALU_ERR_INVALID_ARG),
    (dict(n_heads=65, n_kv_heads=1), P.PALU_ERR_UNSUPPORTED),
    (dict(head_dim=96), P.PALU_ERR_UNSUPPORTED),
    (dict(head_dim=0), P.PALU_ERR_INVALID_ARG),
    (dict(dtype=P.PALU_INT4), P.PALU_ERR_UNSUPPORTED),
    (dict(x_dtype=P.PALU_INT4), P.PALU_ERR_UNSUPPORTED),
    (dict(x_dtype=9), P.PALU_ERR_INVALID_ARG),
    (dict(rope_theta=-1.0), P.PALU_ERR_INVALID_ARG),
    (dict(rope_theta=float("nan")), P.PALU_ERR_INVALID_ARG),
    (dict(norm_eps=-1e-6), P.PALU_ERR_INVALID_ARG),
    (dict(norm_eps=float("inf")), P.PALU_ERR_INVALID_ARG),
    (dict(max_batch=0), P.PALU_ERR_INVALID_ARG),
    (dict(max_batch=65536), P.PALU_ERR_UNSUPPORTED),
    (dict(max_tokens=0), P.PALU_ERR_INVALID_ARG),
    (dict(max_tokens=1 << 31), P.PALU_ERR_UNSUPPORTED),
    (dict(flags=P.PALU_FLAG_ALIBI), P.PALU_ERR_INVALID_ARG),
])
def test_descriptors_refused(kw, status):
    assert P.palu_kv_workspace_size(_desc(**kw))[0] == status


def test_abi_version_and_null_pointers_refused():
    d = _desc()
    d.abi_version = 2
    assert P.palu_kv_workspace_size(d)[0] == P.PALU_ERR_INVALID_ARG
    assert P._lib.palu_kv_workspace_size(ctypes.byref(_desc()), None) == P.PALU_ERR_INVALID_ARG
    assert P._lib.palu_kv_workspace_size(None, None) == P.PALU_ERR_INVALID_ARG
    st, h = P.palu_kv_create(_desc(), 0, 0, 0)
    assert st == P.PALU_ERR_WORKSPACE and h is None
    st, h = P.palu_kv_create(_desc(), 0x1100, 16, 0)
    assert st == P.PALU_ERR_WORKSPACE and h is None
    st, h = P.palu_kv_create(_desc(), 0x1010, 1 << 40, 0)      # misaligned
    assert st == P.PALU_ERR_WORKSPACE and h is None
    pages, rows = P.palu_kv_pages(), P.palu_kv_rows()
    assert P.palu_attend_kv(None, pages, rows, 0, 0, 0, None, 0) == P.PALU_ERR_INVALID_ARG
    assert P.palu_append_kv(None, pages, rows, None, 0, 0, 0, 0, 0, None, None, None, 0) == P.PALU_ERR_INVALID_ARG
    assert P.palu_norm_rope(None, 0, 0, None, 0, None, None, None, 1, 0, 0, None, 0, 0) == P.PALU_ERR_INVALID_ARG
    assert P.palu_kv_check(None, 0) == P.PALU_ERR_INVALID_ARG
    assert P.palu_kv_destroy(None) == P.PALU_OK


def test_fp32_handles_need_no_split_workspace():
    assert P.palu_kv_workspace_size(_desc(dtype=P.PALU_F32))[1] < P.palu_kv_workspace_size(_desc())[1]


def test_binding_refuses_mismatched_tensors():
    import torch
    k = torch.zeros(2, 4, 2, 64)
    with pytest.raises(ValueError):
        P.KVPages(k, torch.zeros(2, 4, 2, 32))
    with pytest.raises(ValueError):
        P.KVPages(k.transpose(1, 2), k.transpose(1, 2))
    i32 = torch.int32
    with pytest.raises(ValueError):       # row_start holds batch + 1 entries
        P.KVRows(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), n_tokens=1, max_new=1, max_kv_len=1)
    with pytest.raises(ValueError):       # int64 lengths
        P.KVRows(torch.zeros(3, dtype=i32), torch.zeros(2, dtype=torch.int64), n_tokens=1, max_new=1, max_kv_len=1)
    with pytest.raises(ValueError):
        P.KVRows(torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), n_tokens=1, max_new=1, max_kv_len=1,
                 page_table=torch.zeros(3, 2, dtype=i32))
    with pytest.raises(ValueError):
        P.KVRows(torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), n_tokens=4, max_new=1, max_kv_len=1,
                 positions=torch.zeros(3, dtype=i32))
