"""CPU pins of the paged KV cache's oracle against closed forms, identities and the decode oracle."""
import math

import numpy as np
import pytest

from oracle import kv_oracle as KO
from oracle import palu_oracle as O


def test_norm_gives_unit_mean_square_and_weights_scale_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    y = KO.norm_rope(x, np.ones(64), [0, 5, 900], 10000.0, 0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0, atol=1e-12)          # a rotation keeps the length
    w = rng.standard_normal(64)
    z = KO.norm_rope(x, w, [0, 0, 0], 10000.0, 0.0)
    assert np.allclose(z, x / np.sqrt((x ** 2).mean(-1, keepdims=True)) * w, atol=1e-12)
    assert np.array_equal(KO.norm_rope(x, None, [7, 7, 7], 0.0, 0.0), x)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))
    a = [float((KO.norm_rope(q, None, [p + 11], 1e4, 0)[0, 0] * KO.norm_rope(k, None, [p], 1e4, 0)[0, 0]).sum())
         for p in (0, 3, 1000, -40)]
    assert np.allclose(a, a[0], atol=1e-9)


def test_one_new_token_over_a_contiguous_cache_is_full_rank_decode():
    # G-LRD decode with identity factors (rank = d_h, one head a group) is decode over the keys themselves
    rng = np.random.default_rng(2)
    n, d, T = 3, 64, 9
    k, v = rng.standard_normal((T, n, d)), rng.standard_normal((T, n, d))
    q = rng.standard_normal((1, n, d))
    pk, pv = np.zeros((1, T, n, d)), np.zeros((1, T, n, d))
    KO.append(pk, pv, k, v, [0, T], [T], None)
    o, lse, _, _ = KO.attend(KO.norm_rope(q, None, [T - 1], 1e4, 0), pk, pv, [0, 1], [T], None)
    bk = np.stack([np.eye(d)] * n)
    ref, ref_lse = O.decode(q, k[None], v[None], bk, [T], 1, mode="rope", theta=1e4)
    assert np.allclose(o, ref, atol=1e-10) and np.allclose(lse, ref_lse, atol=1e-10)


@pytest.mark.parametrize("page_size", [1, 3, 8])
def test_pages_in_any_order_and_chunks_give_the_contiguous_answer(page_size):
    rng = np.random.default_rng(3)
    n, m, d, T = 4, 2, 64, 13
    k, v, q = (rng.standard_normal((T, h, d)) for h in (m, m, n))
    ck, cv = np.zeros((1, T, m, d)), np.zeros((1, T, m, d))
    KO.append(ck, cv, k, v, [0, T], [T], None)
    whole, lse, _, _ = KO.attend(q, ck, cv, [0, T], [T], None)
    per = -(-T // page_size)
    table = rng.permutation(per + 2)[None, :per]
    pk, pv = np.full((per + 2, page_size, m, d), np.nan), np.full((per + 2, page_size, m, d), np.nan)
    got, got_lse = [], []
    for lo, hi in ((0, 5), (5, 12), (12, 13)):
        KO.append(pk, pv, k[lo:hi], v[lo:hi], [0, hi - lo], [hi], table)
        o, s, _, _ = KO.attend(q[lo:hi], pk, pv, [0, hi - lo], [hi], table)
        got.append(o)
        got_lse.append(s)
    assert np.allclose(np.concatenate(got), whole, atol=1e-12)
    assert np.allclose(np.concatenate(got_lse), lse, atol=1e-12)


def test_first_token_returns_its_value_and_unseen_rows_are_empty():
    rng = np.random.default_rng(4)
    k, v, q = (rng.standard_normal((2, 1, 64)) for _ in range(3))
    o, lse, _, _ = KO.attend(q, k[None], v[None], [0, 2], [2], None)
    assert np.allclose(o[0], v[0])
    assert math.isclose(lse[0, 0], float(k[0, 0] @ q[0, 0]) / 8.0, rel_tol=1e-12)
    o, lse, _, _ = KO.attend(q, k[None], v[None], [0, 2], [1], None)   # two new tokens, one cached
    assert np.all(o[0] == 0) and lse[0, 0] == -np.inf and np.allclose(o[1], v[0])
