"""GPU tests of the plan of a step's rows and pages."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8

pytestmark = pytest.mark.gpu


def make(rng, batch, page, most_kv, most_new, ended, spare, empty=0.1):
    lens = rng.integers(0, most_kv + 1, batch)
    held = -(-lens // page) + rng.integers(0, 2, batch)                        # some hold a page to spare
    new = np.where(rng.random(batch) < empty, 0, rng.integers(1, most_new + 1, batch))
    new[rng.permutation(batch)[:ended]] = -1
    need = np.maximum(0, -(-(lens + new) // page) - held) * (new > 0)
    per = int(max((held + need).max(), 1))
    free = max(0, int(need.sum()) + spare)
    pages = int(held.sum()) + free + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((batch, per), -1, dtype=np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    ring = np.full(pages, -1, dtype=np.int32)
    head = int(rng.integers(0, pages))
    ring[(head + np.arange(free)) % pages] = order[at:at + free]
    return dict(new=new.astype(np.int32), kv_len=lens.astype(np.int32), held=held.astype(np.int32), table=table, ring=ring,
                state=np.array([head, free], dtype=np.int32), page=page)


def run(c, n_tokens, in_place=False, layer=None, max_new=None, positions=True, slots=True):
    from rank_kv_cache_gb300 import palu as P
    B = len(c["new"])
    layer = layer or P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B, max_tokens=max(1, n_tokens))
    d = {k: torch.from_numpy(v.copy()).cuda() for k, v in c.items() if k != "page"}
    pool = P.KVPool(d["table"], d["held"], d["ring"], d["state"], page_size=c["page"])

    def fill(n):
        return torch.full((n,), 99, dtype=torch.int32, device="cuda")

    kv_out = d["kv_len"] if in_place else fill(B)
    pos, slot = fill(n_tokens) if positions else None, fill(n_tokens) if slots else None
    rows = P.KVRows(fill(B + 1), kv_out, page_table=d["table"], positions=pos, n_tokens=n_tokens,
                    max_new=int(max(1, c["new"].max())) if max_new is None else max_new,
                    max_kv_len=c["table"].shape[1] * c["page"])
    out = dict(held_out=None, state_out=None) if in_place else dict(held_out=fill(B), state_out=fill(2))
    layer.plan(pool, d["new"], d["kv_len"], rows, slots=slot, **out)
    torch.cuda.synchronize()
    held, state = (d["held"], d["state"]) if in_place else (out["held_out"], out["state_out"])
    got = [rows.tensors[0], kv_out, held, state, pos, slot, d["table"], d["ring"]]
    return [None if t is None else t.cpu().numpy() for t in got], layer


def check(c, got, n_tokens):
    want = K8.plan(c["new"], c["kv_len"], c["held"], c["table"], c["ring"], c["state"], c["page"], n_tokens)
    for name, g, w in zip(("row_start", "kv_len", "held", "state", "positions", "slots", "table", "ring"), got, want):
        if g is not None:
            assert np.array_equal(g, np.asarray(w)), name


@pytest.mark.parametrize("batch,page,most_kv,most_new,ended", [
    (1, 16, 0, 1, 0), (1, 1, 5, 7, 0), (3, 16, 100, 40, 1), (64, 16, 1000, 6, 5), (65, 24, 300, 50, 0), (512, 32, 400, 100, 40),
    (700, 7, 90, 20, 700), (2047, 16, 200, 3, 100), (2048, 64, 100, 3, 9), (5000, 16, 60, 9, 500)])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_the_oracle(cuda_device, batch, page, most_kv, most_new, ended, in_place):
    rng = np.random.default_rng(batch + page)
    c = make(rng, batch, page, most_kv, most_new, ended, 5)
    n = int(np.maximum(c["new"], 0).sum()) + 3
    got, layer = run(c, n, in_place)
    layer.check_device()
    check(c, got, n)


@pytest.mark.parametrize("batch", [5, 300, 4500])
def test_rows_are_admitted_while_pages_and_places_last(cuda_device, batch):
    rng = np.random.default_rng(batch)
    for spare, share in ((-batch // 2, 1.0), (4, 0.5), (-batch // 3, 0.8), (-10 ** 6, 1.0), (4, 0.0)):
        c = make(rng, batch, 16, 100, 40, batch // 10, spare)
        n = int(np.maximum(c["new"], 0).sum() * share)
        got, layer = run(c, n)
        layer.check_device()
        check(c, got, n)


def test_a_plan_elsewhere_can_be_repeated(cuda_device):
    rng = np.random.default_rng(3)
    c = make(rng, 40, 16, 300, 30, 6, 2)
    n = int(np.maximum(c["new"], 0).sum())
    first, layer = run(c, n)
    again, _ = run({**c, "table": first[6], "ring": first[7]}, n, layer=layer)
    for a, b in zip(first, again):
        assert np.array_equal(a, b)


def test_steps_follow_each_other_in_place_and_keep_every_page(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(4)
    B, ps, pages, per = 12, 16, 90, 20
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B, max_tokens=256)
    pool = P.KVPool.empty(B, per, pages, ps)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = P.KVRows(torch.zeros(B + 1, dtype=torch.int32, device="cuda"), lens, page_table=pool.page_table, n_tokens=256,
                    max_new=64, max_kv_len=per * ps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.plan(pool, new, lens, rows)
    state = dict(table=pool.page_table.cpu().numpy(), ring=pool.free_pages.cpu().numpy(), held=np.zeros(B, int), lens=np.zeros(B, int),
                 state=[0, pages])
    for step in range(40):
        n = rng.integers(0, 30, B)
        n[state["lens"] + n > per * ps] = -1
        n[rng.random(B) < 0.1] = -1
        new.copy_(torch.from_numpy(n.astype(np.int32)))
        graph.replay()
        start, kv, held, st, _, _, table, ring = K8.plan(n, state["lens"], state["held"], state["table"], state["ring"],
                                                         state["state"], ps, 256)
        state = dict(table=table, ring=ring, held=np.array(held), lens=np.array(kv), state=st)
        assert np.array_equal(rows.tensors[0].cpu().numpy(), start) and np.array_equal(lens.cpu().numpy(), kv)
        assert np.array_equal(pool.held.cpu().numpy(), held) and np.array_equal(pool.state.cpu().numpy(), st)
        assert np.array_equal(pool.page_table.cpu().numpy(), table)
        free = [int(ring[(st[0] + i) % pages]) for i in range(st[1])]
        assert sorted(free + [int(p) for b in range(B) for p in table[b, :held[b]]]) == list(range(pages))
    layer.check_device()


def test_rows_that_do_not_add_up_are_reported_and_left(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(5)
    base = make(rng, 6, 16, 100, 10, 0, 8, empty=0.0)
    base["new"][:] = 4
    base["held"][:] = -(-base["kv_len"] // 16)
    per = base["table"].shape[1]
    for field, row, value in (("kv_len", 2, -1), ("held", 1, per + 1), ("held", 4, -2), ("new", 3, 1000), ("kv_len", 0, per * 16 - 1),
                              ("held", 5, int(base["held"][5]) - 1)):
        c = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in base.items()}
        c[field][row] = value
        if field == "kv_len" and row == 0:
            c["held"][0] = per
        got, layer = run(c, 64, max_new=50)
        with pytest.raises(P.PaluError):
            layer.check_device()
        # as a plan in which that row brings nothing
        c["new"][row] = 0
        want = K8.plan(c["new"], c["kv_len"], c["held"], c["table"], c["ring"], c["state"], 16, 64)
        for k in (0, 1, 2, 3, 4, 5):
            assert np.array_equal(got[k], np.asarray(want[k])), (field, k)
    _, layer = run({**base, "state": np.array([0, 10 ** 6], dtype=np.int32)}, 64)
    with pytest.raises(P.PaluError):
        layer.check_device()


def test_without_positions_or_slots(cuda_device):
    rng = np.random.default_rng(6)
    c = make(rng, 30, 16, 100, 10, 2, 8)
    n = int(np.maximum(c["new"], 0).sum())
    for positions, slots in ((False, True), (True, False), (False, False)):
        got, layer = run(c, n, positions=positions, slots=slots)
        layer.check_device()
        check(c, got, n)


@pytest.mark.parametrize("batch", [6, 512, 700, 2048, 5000])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_ring_that_does_not_add_up_is_reported_and_left(cuda_device, batch, in_place):
    """With requests that end, others that need pages, and others that do not."""
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(batch)
    base = make(rng, batch, 16, 60, 9, max(2, batch // 10), 5)
    pages, back = len(base["ring"]), int(base["held"][base["new"] < 0].sum())
    base["ring"] = rng.permutation(pages).astype(np.int32)
    n = int(np.maximum(base["new"], 0).sum()) + 3
    for head, count, whole in ((0, 10 ** 6, False), (3, -1, False), (-1, 4, False), (pages, 4, False), (2, pages + 1, False),
                               (pages - 1, pages - back + 1, False), (5, pages - back, True), (0, 2 ** 31 - 1, False)):
        c = {**base, "state": np.array([head, count], dtype=np.int32)}
        got, layer = run(c, n, in_place)
        check(c, got, n)
        if whole:
            layer.check_device()
        else:
            assert np.array_equal(got[7], base["ring"]) and np.array_equal(got[6], base["table"]) and list(got[3]) == [head, count]
            with pytest.raises(P.PaluError):
                layer.check_device()


@pytest.mark.parametrize("batch", [6, 2100])
def test_ended_rows_that_hold_more_than_the_table_are_left(cuda_device, batch):
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(batch)
    for value in (-1, 10 ** 6, 2 ** 31 - 1):
        c = make(rng, batch, 16, 100, 10, batch // 2, 4)
        ended = np.flatnonzero(c["new"] < 0)[::2]
        c["held"][ended] = value
        n = int(np.maximum(c["new"], 0).sum())
        got, layer = run(c, n)
        check(c, got, n)
        assert np.array_equal(got[1][ended], c["kv_len"][ended]) and np.all(got[2][ended] == value)
        with pytest.raises(P.PaluError):
            layer.check_device()


def test_as_many_tokens_as_a_pool_has_slots(cuda_device):
    """Two rows that fill a pool of nearly 2^31 slots in one step: the places' numbers end next to the largest int."""
    from rank_kv_cache_gb300 import palu as P
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("wants 20 GB")
    i32 = dict(dtype=torch.int32, device="cuda")
    ps, pages, L = 64, (1 << 25) - 1, (1 << 30) - 64
    N = 2 * L + 5
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=2, max_tokens=N)
    pool = P.KVPool.empty(2, 1 << 24, pages, ps)
    positions, slots = (torch.full((N + 64,), 99, **i32) for _ in range(2))
    lens = torch.zeros(2, **i32)
    rows = P.KVRows(torch.zeros(3, **i32), lens, page_table=pool.page_table, positions=positions[:N], n_tokens=N, max_new=L, max_kv_len=L)
    layer.plan(pool, torch.full((2,), L, **i32), lens, rows, slots=slots[:N])
    layer.check_device()
    assert rows.tensors[0].tolist() == [0, L, 2 * L] and lens.tolist() == [L, L] and pool.held.tolist() == [L // ps] * 2
    assert pool.state.tolist() == [2 * L // ps, pages - 2 * L // ps]
    for lo in range(0, N, 1 << 28):                                           # pages come in order: a token's slot is its number
        t = torch.arange(lo, min(lo + (1 << 28), 2 * L), **i32)
        assert torch.equal(slots[lo:lo + len(t)], t) and torch.equal(positions[lo:lo + len(t)], torch.where(t < L, t, t - L))
    assert slots[2 * L:].tolist() == [-1] * 5 + [99] * 64 and positions[2 * L:].tolist() == [0] * 5 + [99] * 64
