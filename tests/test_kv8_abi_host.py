"""CPU tests of the 8-bit paged cache's, the plan's and the verification's entry points: refused on the host, before any CUDA
call."""
import pytest
import torch

from rank_kv_cache_gb300 import palu as P

BAD = P.PALU_ERR_INVALID_ARG


def test_null_handles_refused():
    pages, rows, pool = P.palu_kv8_pages(), P.palu_kv_rows(), P.palu_kv_pool()
    assert P.palu_append_kv8(None, pages, rows, None, 0, 0, 0, 0, 0, None, None, None, 0) == BAD
    assert P.palu_attend_kv8(None, pages, rows, 0, 0, 0, None, 0) == BAD
    assert P.palu_plan_kv_rows(None, pool, 0, 0, 1, 1, 1, 1, 0, 0, None, None, None, None, 0) == BAD
    assert P.palu_verify_drafts(None, 0, 0, None, 0, P.PALU_F32, 1, 0, 1, 1, 0, 0, 0, 0, 0, None, None, 0) == BAD


def test_pages_of_codes():
    k = torch.zeros(2, 32, 2, 64, dtype=torch.uint8)
    s = torch.ones(2, 2, 2)
    assert P.KVPages8(k, k, s, s).page_size == 32
    f = k.view(torch.float8_e4m3fn)
    assert P.KVPages8(f, f, s, s).heads == (2, 64)
    for bad in ((k, f, s, s), (k, k[:1], s, s), (k.bfloat16(), k.bfloat16(), s, s), (k, k, s[:, :1], s), (k, k, s, s.double()),
                (k.transpose(1, 2), k.transpose(1, 2), s, s)):
        with pytest.raises(ValueError):
            P.KVPages8(*bad)
    k = torch.zeros(2, 24, 2, 64, dtype=torch.uint8)                          # no whole blocks of 16
    with pytest.raises(ValueError):
        P.KVPages8(k, k, s, s)
    with pytest.raises(ValueError):
        P.KVPages8.empty(2, 24, 2, 64, device="cpu")
    e = P.KVPages8.empty(3, 48, 2, 64, device="cpu")
    assert e.k_scale.shape == (3, 3, 2) and not e.k.view(torch.uint8).any()


def test_pools():
    pool = P.KVPool.empty(3, 4, 10, 16, device="cpu")
    assert pool.state.tolist() == [0, 10] and sorted(pool.free_pages.tolist()) == list(range(10))
    i = dict(dtype=torch.int32)
    good = [torch.zeros(3, 4, **i), torch.zeros(3, **i), torch.zeros(9, **i), torch.zeros(2, **i)]
    P.KVPool(*good, page_size=16)
    for at, bad in ((0, torch.zeros(12, **i)), (1, torch.zeros(4, **i)), (2, torch.zeros(3, 3, **i)), (3, torch.zeros(3, **i)),
                    (1, torch.zeros(3, dtype=torch.int64))):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            P.KVPool(*args, page_size=16)
