"""CPU pins of the 8-bit paged cache's oracle, and of the oracles of the plan and the verification, against other sources."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8
from oracle import kv_oracle as KO


def test_codes_are_torchs_e4m3():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(K8.decode(np.arange(256)), every, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2.6, 20000), every[np.isfinite(every)],
                        [0.0, -0.0, 432.0, 447.99, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K8.encode(x), want)
    assert list(K8.encode([1e9, -1e9, np.inf, -np.inf])) == [0x7e, 0xfe, 0x7e, 0xfe] and K8.encode(np.nan) & 127 == 127


def test_scales_are_the_least_powers():
    assert K8.scale_for(448.0) == 1.0 and K8.scale_for(448.0001) == 2.0 and K8.scale_for(224.0) == 0.5
    assert K8.scale_for(0.0) == 2.0 ** -64 and K8.scale_for(1e30) == 2.0 ** 64
    for x in np.random.default_rng(1).uniform(-40, 40, 200):
        s = K8.scale_for(2.0 ** x)
        assert 224 * s < 2.0 ** x <= 448 * s


def test_a_growing_scale_keeps_older_values_and_new_blocks_begin_anew():
    codes, scales = np.zeros((2, 32, 1, 8), np.uint8), np.full((2, 2, 1), 2.0 ** 50, np.float32)
    table = np.array([[1]])
    rng = np.random.default_rng(2)
    x = rng.standard_normal((20, 1, 8)) * np.concatenate([np.ones(10), np.full(10, 100.0)])[:, None, None]
    stored = []
    for t in range(20):
        K8.append(codes, scales, x[t:t + 1], [0, 1], [t + 1], table)
        stored.append(K8.values(codes, scales)[1, :t + 1].copy())
    assert scales[1, 0, 0] == K8.scale_for(np.abs(x[:16]).max()) and scales[1, 1, 0] == K8.scale_for(np.abs(x[16:]).max())
    # a power of two moves the exponents alone: only values that fell below 2^-6 of a scale may have changed
    end = K8.values(codes, scales)[1]
    for t, was in enumerate(stored):
        s = np.repeat(scales[1, :, 0], 16)[:t + 1, None, None]
        assert np.all((end[:t + 1] == was) | (np.abs(was) < 2.0 ** -6 * s))
    # a value's own rounding, and one below 2^-6 of each scale that came after, all but the last together as much as the last
    s = np.repeat(scales[1, :, 0].astype(np.float64), 16)[:20, None, None]
    assert np.all(np.abs(end[:20] - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s)
    assert np.all(codes[0] == 0) and np.all(scales[0] == 2.0 ** 50)


def test_whole_blocks_at_once_are_as_the_dense_cache_rounded():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((37, 2, 8))
    codes, scales = np.zeros((3, 16, 2, 8), np.uint8), np.ones((3, 1, 2), np.float32)
    K8.append(codes, scales, x, [0, 37], [37], np.array([[2, 0, 1]]))
    dense_k, dense_v = np.zeros((3, 16, 2, 8)), np.zeros((3, 16, 2, 8))
    KO.append(dense_k, dense_v, x, x, [0, 37], [37], np.array([[2, 0, 1]]), theta=0.0)
    got = K8.values(codes, scales)
    assert np.all(np.abs(got - dense_v) <= np.maximum(2.0 ** -4 * np.abs(dense_v), 2.0 ** -10 * np.repeat(scales, 16, 1)[..., None]))


def test_a_plan_is_the_scan_of_the_lengths():
    new, lens, held = [3, -1, 0, 20], [14, 33, 7, 0], [1, 3, 1, 0]
    table = np.full((4, 3), -1)
    table[0, 0], table[1], table[2, 0] = 9, [1, 2, 3], 4
    ring = np.array([6, 7, 8, 0, 0, 0, 0, 0, 0, 5])
    start, kv, hold, state, pos, slots, tab, after = K8.plan(new, lens, held, table, ring, [9, 4], 16, 25)
    assert start == [0, 3, 3, 3, 23] and kv == [17, 0, 7, 20] and hold == [2, 0, 1, 2] and state == [2, 4]
    assert list(tab[0]) == [9, 5, -1] and list(tab[3]) == [6, 7, -1] and list(after[2:6]) == [8, 1, 2, 3]
    assert pos[:4] == [14, 15, 16, 0] and slots[:4] == [9 * 16 + 14, 9 * 16 + 15, 80, 96]
    assert pos[23:] == [0, 0] and slots[23:] == [-1, -1]
    # a page less, and the last row and all behind it get nothing
    start, kv, hold, state, *_ = K8.plan(new + [1], lens + [0], held + [1], np.vstack([table, table[:1]]), ring, [9, 2], 16, 25)
    assert start == [0, 3, 3, 3, 3, 3] and kv == [17, 0, 7, 0, 0] and hold == [2, 0, 1, 0, 1] and state == [0, 4]


def test_verified_tokens_are_distributed_as_the_target():
    # over the drafts' distribution and a grid of uniforms, the first token's shares are the target's: what the rule is for
    p, q = np.array([0.5, 0.25, 0.125, 0.125]), np.array([0.125, 0.5, 0.25, 0.125])
    grid = (np.arange(64) + 0.5) / 64
    count = np.zeros(4)
    for x in range(4):
        for u in grid:
            for v in grid:
                a, token = K8.verify(np.stack([p, p]), q[None], [x], [u, v])
                count[x if a else token] += q[x] / 64 ** 2
    assert np.allclose(count, p, atol=1 / 64)


@pytest.mark.parametrize("u,v,want", [(0.0, 0.0, (1, 0)), (0.99, 0.0, (0, 1)), (0.99, 0.99, (0, 2))])
def test_certain_drafts(u, v, want):
    p = np.array([[0.5, 0.25, 0.25], [1.0, 0.0, 0.0]])
    assert K8.verify(p, None, [0], [u, v]) == want


@pytest.mark.parametrize("u,want", [(1.0, 2), (7.5, 2), (float("inf"), 2), (float("nan"), 2), (-1.0, 2), (1 - 2.0 ** -24, 2)])
def test_uniforms_are_brought_into_range(u, want):
    # the target and the draft agree, so that every uniform below 1 accepts; behind the drafts 0 draws the first, the largest the last
    p = np.array([[0.5, 0.5, 0.0], [0.25, 0.75, 0.0], [0.0, 0.125, 0.875]])
    assert K8.verify(p, p[:2], [0, 1], [u, u, u]) == (want, 1 if u < 0 else 2)
    # a certain draft of less than all is rejected by the largest
    assert K8.verify(p[:2], None, [0], [u, 0.0]) == ((1, 0) if u < 0 else (0, 1))


@pytest.mark.parametrize("state,whole", [([9, 4], True), ([9, 7], True), ([9, 8], False), ([10, 4], False), ([-1, 4], False), ([9, -1], False)])
def test_a_ring_that_does_not_add_up_is_left(state, whole):
    new, lens, held = [3, -1, 0, 20], [14, 33, 7, 0], [1, 3, 1, 0]
    table = np.full((4, 3), -1)
    table[0, 0], table[1], table[2, 0] = 9, [1, 2, 3], 4
    ring = np.array([6, 7, 8, 0, 0, 0, 0, 0, 0, 5])
    start, kv, hold, after, pos, slots, tab, out = K8.plan(new, lens, held, table, ring, state, 16, 25)
    if whole:
        assert kv == [17, 0, 7, 20] and hold == [2, 0, 1, 2] and after == [2, state[1]]
    else:                                                                     # no page is taken or given back
        assert start == [0] * 5 and kv == lens and hold == held and after == state
        assert np.array_equal(tab, table) and np.array_equal(out, ring)
    # an ended row whose pages cannot be right is left
    start, kv, hold, after, *_ = K8.plan(new, lens, [1, 4, 1, 0], table, ring, [9, 4], 16, 25)
    assert kv == [17, 33, 7, 20] and hold == [2, 4, 1, 2] and after == [2, 1]
