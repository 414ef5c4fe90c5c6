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


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (64, "f16"), (128, "bf16")])
def test_long_tails_behind_attention_sinks_keep_their_weight(new, d, dtype):
    """Seven sinks with a score of 18 above 65529 tokens of score 0, which hold all the values: each of those weighs
    2^-26 of a sink, together 1.4e-4 of the output. The sinks stand where every warp, unit and tile of the kernels' first
    steps has one, and the rows are as many as leave them whole.

    Bound: the score 18 is a sum of d products accumulated in fp32 (2^-16 of it), the exponential 2^-20, both of them in
    the sinks' weights and the others'; a weight's rounding u, or half an fp16 step (2^-25) of weights that are lifted so
    that a sink's is 2^7 at least: 2^-32 of it for each of the others; the sums 2^-20; the output u and half its smallest
    step."""
    from rank_kv_cache_gb300 import palu as P
    B, m, L, page = 38, 8, 65536, 256
    dev, t = torch.device("cuda:0"), TYPES[dtype]
    sinks = torch.tensor([0, 16, 32, 48, 64, 96, 128], device=dev)
    k, v = torch.zeros(L // page, page, m, d, dtype=t, device=dev), torch.full((L // page, page, m, d), 64.0, dtype=t, device=dev)
    each = torch.tensor(18.0 * d ** 0.5 / d).to(t)
    k.view(L, m, d)[sinks] = each.to(dev)
    v.view(L, m, d)[sinks] = 0
    score = float(each) * d / d ** 0.5
    table = torch.arange(L // page, dtype=torch.int32, device=dev).expand(B, -1).contiguous()   # all rows read the same
    rows = P.KVRows(torch.arange(0, B * new + 1, new, dtype=torch.int32, device=dev),
                    torch.full((B,), L, dtype=torch.int32, device=dev), n_tokens=B * new, max_new=new, max_kv_len=L,
                    page_table=table)
    layer = P.PagedAttention(n_heads=m, n_kv_heads=m, head_dim=d, dtype=dtype, max_batch=B, max_tokens=B * new)
    q = torch.ones(B * new, m, d, dtype=t, device=dev)
    lse = torch.empty(B * new, m, dtype=torch.float32, device=dev)
    out = layer.attend(P.KVPages(k, v), rows, q, lse=lse)
    layer.check_device()
    others = L - new + 1 + np.arange(new, dtype=np.float64) - 7      # of new token i
    total = others + 7 * np.exp(score)
    ref = np.tile(64 * others / total, B)[:, None, None]
    ref_lse = np.tile(np.log(total), B)[:, None]
    f = torch.finfo(t)
    e = 2.0 ** -16 * score + 2.0 ** -20
    steps = 2.0 ** -32 * 64 * L / 7 if dtype == "f16" else 0.0
    tol = (f.eps + 2 * e + 2.0 ** -20) * ref + steps + f.smallest_normal * f.eps / 2
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3f} of the bound"
    assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= e + 2.0 ** -20 * (1 + ref_lse))


@pytest.mark.parametrize("new", [1, 40])
def test_scores_past_the_lifted_range_stay_finite(new):
    # every score is 4.5e6 or more (log2 units 6.5e6), and the first of all by 2^-3 of that: one-hot rows
    from rank_kv_cache_gb300 import palu as P
    dev, d, L = torch.device("cuda:0"), 128, 700
    k = torch.full((1, L, 1, d), 1000.0, dtype=torch.float16, device=dev)
    k[0, 0] = 1125.0
    v = torch.randn(1, L, 1, d, generator=torch.Generator(dev).manual_seed(41), device=dev).half()
    q = torch.full((new, 2, d), 400.0, dtype=torch.float16, device=dev)
    rows = P.KVRows(torch.tensor([0, new], dtype=torch.int32, device=dev), torch.tensor([L], dtype=torch.int32, device=dev),
                    n_tokens=new, max_new=new, max_kv_len=L)
    layer = P.PagedAttention(n_heads=2, n_kv_heads=1, head_dim=d, dtype="f16", max_tokens=new)
    lse = torch.empty(new, 2, dtype=torch.float32, device=dev)
    out = layer.attend(P.KVPages(k, v), rows, q, lse=lse)
    layer.check_device()
    # the base is a multiple of 1/2 at this size, so the one weight left is 2^x, |x| <= 1/4, not 1: it is rounded to fp16
    # (u) for the product and not for the sum, and the quotient is rounded once more (u)
    ref, u = v[0, 0, 0].double(), 2.0 ** -11
    assert torch.all((out.double() - ref).abs() <= (2 * u + 2.0 ** -20) * ref.abs() + 2.0 ** -25)
    s = 400.0 * 1125 * d / d ** 0.5
    assert torch.all((lse.double() - s).abs() <= 2.0 ** -16 * s)


@pytest.mark.parametrize("new,q_scale", [(1, 12.0), (50, 2.0), (200, 12.0)])
def test_fp16_rows_whose_maximum_rises(new, q_scale):
    # scores that rise and fall by more and by less than the threshold, over cut and whole tiles
    b = Batch(n=4, m=2, d=128, dtype="f16", news=[new, new], lens=[1500, 400], page=16, seed=42, q_scale=q_scale)
    wave = 1 + torch.sin(torch.arange(b.pk.shape[0] * 16) / 200).reshape(-1, 16, 1, 1)
    b.pk = (b.pk.float() * wave).half()
    b.pages.k.copy_(b.pk)
    b.run_and_check()


def _turns(theta, d, k, digits=60):
    """theta^(-2k/d) / 2 pi, as a Decimal."""
    from decimal import Decimal, getcontext
    getcontext().prec = digits

    def arctan_inverse(n):
        term, total, i = Decimal(1) / n, Decimal(1) / n, 1
        while abs(term) > Decimal(10) ** -digits:
            term, i = -term / (n * n), i + 2
            total += term / i
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))           # Machin
    return (Decimal(theta).ln() * (Decimal(-2 * k) / d)).exp() / (2 * pi)


@pytest.mark.parametrize("theta", [1e4, 1e5])
@pytest.mark.parametrize("d,sign", [(128, 1), (64, 1), (64, -1)])
def test_far_positions_against_sixty_digits(theta, d, sign):
    """Of the 2^20 farthest positions, each pair's whose angle comes nearest to whole turns: there fp32 holds the sine to
    2^-24 of itself, and an error of the frequency shows. Bound: half of 2^-64 turns, times the position, in radians; four
    roundings of the sine."""
    from decimal import Decimal
    from rank_kv_cache_gb300 import palu as P
    half, dev = d // 2, torch.device("cuda:0")
    pos = sign * (np.int64(2 ** 31 - 1) - np.arange(2 ** 20))
    exact = [_turns(theta, d, k) for k in range(half)]
    at, sines = [], []
    for f in exact:
        turn = np.uint64(int((f % 1) * 2 ** 64))                     # to find the positions; the angles are exact
        with np.errstate(over="ignore"):
            phase = (pos.astype(np.uint64) * turn).view(np.int64)
        i = int(np.argmin(np.abs(phase.astype(np.float64))))
        x = (f * int(pos[i])) % 1
        x = float(x - 1 if x > Decimal("0.5") else x + 1 if x < Decimal("-0.5") else x)
        at.append(int(pos[i]))
        sines.append(np.sin(2 * np.pi * x))
    x = torch.zeros(half, 1, d, device=dev)
    x[:, :, :half] = 1.0                                             # pairs (1, 0) turn into (cos, sin)
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=d, dtype="f32", rope_theta=theta, max_tokens=half)
    y, _ = layer.norm_rope(x, positions=torch.tensor(at, dtype=torch.int32, device=dev))
    got = y[:, 0].diagonal(half).double().cpu().numpy()              # token k's sine of pair k
    sines = np.array(sines)
    assert np.abs(sines).max() < 2.0 ** -9
    tol = 2.0 ** -65 * 2.0 ** 31 * 2 * np.pi + 2.0 ** -22 * np.abs(sines)
    assert np.all(np.abs(got - sines) <= tol), np.max(np.abs(got - sines) / tol)


@pytest.mark.parametrize("what,row_start,lens,max_new,max_kv", [
    ("a length past the bound, with pages for it", [0, 2, 4], [9, 5], 2, 8),
    ("a negative length of a row without new tokens", [0, 4, 4], [9, -1], 4, 12),
    ("more new tokens than the bound", [0, 3, 4], [9, 5], 2, 12),
    ("a bound of no new tokens", [0, 3, 4], [9, 5], 0, 12),
    ("a row that starts before the one ahead of it", [0, 3, 1], [9, 5], 4, 12),
    ("a row that ends behind the tokens", [0, 3, 5], [9, 5], 4, 12),
    ("the last of many rows", [0, 2, 4] + [4] * 40, [9, 5] + [4] * 39 + [13], 2, 12),
])
def test_append_reports_rows_that_break_their_bounds(what, row_start, lens, max_new, max_kv):
    """What attend reports of the rows, append does too: not every cache that is filled here is read by attend."""
    from rank_kv_cache_gb300 import palu as P
    rng, dev, batch = np.random.default_rng(43), torch.device("cuda:0"), len(lens)
    k, v = rounded(rng, (4, 1, 64), "f16").to(dev), rounded(rng, (4, 1, 64), "f16").to(dev)
    layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f16", max_batch=batch, max_tokens=4)
    table = torch.arange(batch * 4, dtype=torch.int32, device=dev).view(batch, 4)

    def run(row_start, lens, max_new, max_kv):
        pages = P.KVPages(*(torch.zeros(batch * 4, 4, 1, 64, dtype=torch.float16, device=dev) for _ in range(2)))
        rows = P.KVRows(torch.tensor(row_start, dtype=torch.int32, device=dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                        n_tokens=4, max_new=max_new, max_kv_len=max_kv, page_table=table)
        layer.append(pages, rows, k, v)
        return pages

    run([0, 2, 4] + [4] * (batch - 2), [9, 5] + [4] * (batch - 2), 2, 12)
    layer.check_device()                                             # rows that keep their bounds
    pages = run(row_start, lens, max_new, max_kv)
    with pytest.raises(P.PaluError):
        layer.check_device()
    layer.check_device()                                             # reported once
    # tokens 0 and 1 have a row and a slot in every case: they are stored
    n = row_start[1]
    assert torch.equal(pages.v.view(batch, 16, 64)[0, 9 - n:11 - n], v[:2, 0])


def test_attend_reports_new_tokens_past_a_bound_of_none():
    from rank_kv_cache_gb300 import palu as P
    b = Batch(n=4, m=2, d=64, dtype="f16", news=[2, 0], lens=[20, 30], page=16, seed=44, max_new=0)
    out, lse = b.attend()
    with pytest.raises(P.PaluError):
        b.layer.check_device()
    assert torch.all(out == 7.0) and torch.all(lse == 7.0)           # clamped to no new tokens
    b.rows.tensors[0].zero_()                                        # rows that keep the bound
    b.attend()
    b.layer.check_device()


class Rows:
    """A ragged batch made on the GPU, its rows' pages scattered over one pool; float64 references of single tokens."""

    def __init__(self, *, n, m, d, dtype, news, lens, page, seed):
        from rank_kv_cache_gb300 import palu as P
        g = torch.Generator("cuda:0").manual_seed(seed)
        dev, t = torch.device("cuda:0"), TYPES[dtype]
        self.n, self.m, self.d, self.dtype, self.news, self.lens, self.page = n, m, d, dtype, news, lens, page
        per = [-(-x // page) for x in lens]
        order = torch.randperm(sum(per), generator=g, device=dev).int()
        self.table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device=dev)    # past a row's end: no page
        at = 0
        for b, x in enumerate(per):
            self.table[b, :x] = order[at:at + x]
            at += x
        self.start = np.concatenate([[0], np.cumsum(news)])
        N = int(self.start[-1])
        self.k, self.v = (torch.randn(sum(per), page, m, d, generator=g, device=dev).to(t) for _ in range(2))
        self.q = torch.randn(N, n, d, generator=g, device=dev).to(t)
        self.layer = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=dtype, max_batch=len(lens), max_tokens=N)
        self.pages = P.KVPages(self.k, self.v)
        self.rows = P.KVRows(torch.from_numpy(self.start).int().to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                             page_table=self.table, n_tokens=N, max_new=max(news), max_kv_len=max(lens))
        self.out = torch.empty(N, n, d, dtype=t, device=dev)
        self.lse = torch.empty(N, n, dtype=torch.float32, device=dev)

    def attend(self):
        self.layer.attend(self.pages, self.rows, self.q, out=self.out, lse=self.lse)

    def check(self, tokens, heads):
        """(row, new token) pairs against float64; the bounds of Batch.check."""
        g, u = self.n // self.m, torch.finfo(TYPES[self.dtype]).eps / 2
        for b, i in tokens:
            L, n = self.lens[b], self.news[b]
            t = torch.arange(L - n + i + 1, device=self.k.device)
            at = self.table[b, t // self.page].long() * self.page + t % self.page
            tok = int(self.start[b]) + i
            for h in heads:
                K, V = (x.flatten(0, 1)[at, h // g].double() for x in (self.k, self.v))
                q = self.q[tok, h].double()
                s = K @ q / self.d ** 0.5
                p = torch.softmax(s, 0)
                e = 2.0 ** -16 * float((K.abs() @ q.abs()).max()) / self.d ** 0.5 + 2.0 ** -20
                o = p @ V
                tol = u * o.abs() + (u + 2 * e + 2.0 ** -20) * (p @ V.abs())
                if self.dtype == "f16":
                    tol = tol + 2.0 ** -25 * L * 8 + 2.0 ** -25
                assert bool(((self.out[tok, h].double() - o).abs() <= tol).all()), (b, i, h)
                lse = torch.logsumexp(s, 0)
                assert abs(float(self.lse[tok, h].double() - lse)) <= e + 2.0 ** -20 * (1 + abs(float(lse)))

    def time(self, passes=15):
        """Median of several passes, in microseconds."""
        for _ in range(3):
            self.attend()
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2 * passes)]
        torch.cuda.synchronize()
        for i in range(passes):
            ev[2 * i].record()
            self.attend()
            ev[2 * i + 1].record()
        torch.cuda.synchronize()
        return float(np.median([1e3 * ev[2 * i].elapsed_time(ev[2 * i + 1]) for i in range(passes)]))


def test_more_pieces_than_the_workspace_holds_are_cut_coarser():
    """33 rows on one key/value head: a prompt of 7400, a decode at 57000 and 31 at 1000. An SM's share is 50 steps of
    128 tokens; in shares the prompt's 232 pairs of tiles and the decode make 473 pieces, the workspace holds 456. With 32
    rows the pieces are weighed instead. The 33rd row adds 8 steps to 7600, and a cut a quarter coarser lets the last wave
    last a quarter longer: 1.6 times the 32 rows' time leaves room for both. Whole, the decode's 446 steps alone are nine
    shares."""
    news, lens = [7400, 1] + [1] * 31, [7400, 57000] + [1000] * 31
    shape = dict(n=8, m=1, d=128, dtype="bf16", page=64, seed=45)
    many, few = Rows(news=news, lens=lens, **shape), Rows(news=news[:-1], lens=lens[:-1], **shape)
    for x in (many, few):
        x.attend()
        x.layer.check_device()
        x.check([(0, 0), (0, 3700), (0, 7399), (1, 0), (2, 0), (len(x.lens) - 1, 0)], [0, 7])
    a, b = many.time(), few.time()
    print(f"33 rows {a:.1f} us, 32 rows {b:.1f} us")
    assert a <= 1.6 * b, f"{a:.1f} us against {b:.1f}"


@pytest.mark.parametrize("n,m,news,lens", [
    (4, 4, [2560] * 6 + [1] + [0] * 26, [2560] * 6 + [5120] + [9] * 26),         # 492 pieces of one-share prompts
    (2, 2, [40] * 30 + [300] * 30, [40 + 977 * i % 9000 for i in range(60)]),
    (1, 1, [17] * 4190 + [500] * 10, [17 + i % 40 for i in range(4190)] + [500 + 3000 * i for i in range(10)]),
])
def test_many_rows_with_cut_ones(n, m, news, lens):
    lens = [max(a, b) for a, b in zip(news, lens)]
    x = Rows(n=n, m=m, d=128, dtype="f16", news=news, lens=lens, page=32, seed=46)
    x.attend()
    x.layer.check_device()
    longest = int(np.argmax(lens))
    live = [b for b in range(len(news)) if news[b]]
    x.check([(b, i) for b in {live[0], live[len(live) // 2], longest, live[-1]} for i in (0, news[b] - 1)], [0, n - 1])
    first = x.out.clone(), x.lse.clone()
    for _ in range(5):
        x.attend()
        assert torch.equal(x.out, first[0]) and torch.equal(x.lse, first[1])


def test_the_time_of_many_short_rows_grows_with_their_number():
    """Decode of rows of 16 tokens, 8 heads: four times the rows are four times the pieces, and each CTA walks the rows'
    lengths a fixed number of times. 6.5 times the time leaves room for that; a search from the first row for each piece
    is 16 times as long."""
    shape = dict(n=8, m=8, d=64, dtype="f16", page=16, seed=47)
    a, b = (Rows(news=[1] * B, lens=[16] * B, **shape) for B in (2048, 8192))
    for x in (a, b):
        x.attend()
        x.layer.check_device()
        last = len(x.lens) - 1
        x.check([(0, 0), (31, 0), (32, 0), (last // 2, 0), (last, 0)], [0, 7])
    ta, tb = a.time(), b.time()
    print(f"2048 rows {ta:.1f} us, 8192 rows {tb:.1f} us")
    assert tb <= 6.5 * ta, f"{tb:.1f} us against {ta:.1f}"


@pytest.mark.parametrize("batch,top", [(33, 4000), (100, 700), (1100, 90)])
def test_many_ragged_rows_of_one_token(batch, top):
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(top), batch))]
    lens[batch // 2] = top * 20                                       # one that is cut
    x = Rows(n=8, m=4, d=128, dtype="bf16", news=[1] * batch, lens=lens, page=16, seed=48)
    x.attend()
    x.layer.check_device()
    x.check([(b, 0) for b in sorted({0, 1, 31, 32, batch // 2 - 1, batch // 2, batch // 2 + 1, batch - 1})], [0, 7])


@pytest.mark.parametrize("capacity,new", [(20, 20), (3, 3), (20, 2), (130, 40)])
def test_contiguous_caches_smaller_than_a_tile(capacity, new):
    Batch(n=24, m=1, d=64, dtype="f16", news=[new], lens=[capacity], page=capacity, table=False, seed=49).run_and_check()
    Batch(n=24, m=3, d=128, dtype="bf16", news=[1, new, new], lens=[1, new, capacity], page=capacity, table=False,
          seed=50).run_and_check()


@pytest.mark.parametrize("new", [1, 40])
def test_empty_caches_with_a_bound_of_no_length(new):
    b = Batch(n=4, m=2, d=128, dtype="bf16", news=[new, 0], lens=[0, 0], page=16, seed=51, max_kv=0)
    out, lse = b.run_and_check()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("news,lens", [([1, 3], [40, 2000]), ([60, 5], [300, 9000])])
def test_a_query_that_is_not_a_number_stays_by_itself(news, lens):
    b = Batch(n=4, m=2, d=128, dtype="f16", news=news, lens=lens, page=16, seed=52)
    ref, ref_lse = b.attend()
    b.qd[0, 1, 5] = float("nan")
    b.qd[news[0], 2] = float("inf")
    out, lse = b.attend()
    bad = torch.zeros(b.N, 4, dtype=torch.bool, device=b.dev)
    bad[0, 1] = bad[news[0], 2] = True
    assert torch.all(torch.isnan(out[bad])) and torch.all(torch.isnan(lse[bad]))
    assert torch.all(torch.isfinite(out[~bad])) and torch.all(torch.isfinite(lse[~bad]))
    # rows of a warp are rescaled together, by factors of one: their neighbours' bits stay
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], ref_lse[~bad])


@pytest.mark.parametrize("news,lens", [([1], [30000]), ([40], [30000]), ([5, 1], [64, 9])])
def test_outputs_without_the_log_sum(news, lens):
    b = Batch(n=4, m=2, d=64, dtype="bf16", news=news, lens=lens, page=64, seed=53)
    ref, _ = b.attend()
    assert torch.equal(b.layer.attend(b.pages, b.rows, b.qd), ref)


def test_queries_rotated_in_place_by_the_append():
    from rank_kv_cache_gb300 import palu as P
    rng, dev = np.random.default_rng(54), torch.device("cuda:0")
    q, k, v = (rounded(rng, (5, h, 64), "bf16").to(dev) for h in (8, 2, 2))
    w = rounded(rng, (64,), "bf16").to(dev)
    rows = P.KVRows(torch.tensor([0, 2, 5], dtype=torch.int32, device=dev), torch.tensor([20, 7], dtype=torch.int32, device=dev),
                    n_tokens=5, max_new=3, max_kv_len=32)
    layer = P.PagedAttention(n_heads=8, n_kv_heads=2, head_dim=64, dtype="bf16", max_batch=2, max_tokens=5)
    got = []
    for out in (None, q.clone()):
        pages = P.KVPages(*(torch.zeros(2, 32, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)))
        given = q if out is None else out
        got.append((layer.append(pages, rows, k, v, q=given, q_weight=w, k_weight=w, q_out=out), pages.k, pages.v))
    layer.check_device()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_graphs_of_one_handle_replayed_in_turn():
    """A step's graph and a prompt's share the handle's workspace; they follow each other on a stream, any way round."""
    a = Batch(n=8, m=2, d=128, dtype="bf16", news=[1, 1], lens=[9000, 700], page=16, seed=55)
    b = Batch(n=8, m=2, d=128, dtype="bf16", news=[150, 40], lens=[5000, 9000], page=16, seed=56)
    b.layer.close()
    a.layer.close()
    from rank_kv_cache_gb300 import palu as P
    a.layer = b.layer = P.PagedAttention(n_heads=8, n_kv_heads=2, head_dim=128, dtype="bf16", max_batch=2, max_tokens=190)
    refs, graphs, outs = [], [], []
    for x in (a, b):
        refs.append(x.attend())
        x.check_sampled(*refs[-1], [0, x.news[0] - 1, x.N - 1], [0, 7])
        outs.append((torch.empty_like(refs[-1][0]), torch.empty_like(refs[-1][1])))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.layer.attend(x.pages, x.rows, x.qd, out=outs[-1][0], lse=outs[-1][1])
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1), (1, 0, 1, 0, 1)):
        for o, s in outs:
            o.fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i][0], refs[i][0]) and torch.equal(outs[i][1], refs[i][1])
    a.layer.check_device()


def test_two_handles_side_by_side_against_float64():
    a = Batch(n=8, m=2, d=128, dtype="f16", news=[1, 1], lens=[9000, 800], page=16, seed=57)
    b = Batch(n=8, m=2, d=128, dtype="f16", news=[150, 3], lens=[5000, 700], page=16, seed=58)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, o in zip((a, b), streams, outs):
            lse = torch.empty(x.N, 8, dtype=torch.float32, device=x.dev)
            o.append((x.layer.attend(x.pages, x.rows, x.qd, lse=lse, stream=s), lse))
    torch.cuda.synchronize()
    for x, s, o in zip((a, b), streams, outs):
        x.layer.check_device(s)
        x.check_sampled(*o[0], [0, x.news[0] // 2, x.news[0], x.N - 1], [0, 3, 7])
        assert all(torch.equal(y[0], o[0][0]) and torch.equal(y[1], o[0][1]) for y in o)


def test_a_hybrid_window_that_rolls():
    """The window of a hybrid decode over several steps: each new token takes the oldest window slot (one new token with
    kv_len = slot + 1, at its own position), the token that leaves moves to the latent middle. Against the oracle."""
    from oracle import kv_oracle as KO
    from oracle import palu_oracle as O
    from rank_kv_cache_gb300 import palu as P
    from synthetic import gen
    from tests.gpu_cases import Case, assert_close
    sinks, window, T, steps, B = 4, 8, 300, 11, 2
    D = sinks + window
    cfg = gen.ROPE_FP16.with_(T=T, batch=B)
    latent_pos = np.stack([sinks + np.arange(T)] * B).astype(np.int32)
    c = Case(cfg, positions=latent_pos, q_pos=[0] * B, max_position=T + D + steps)
    n, d, dev = cfg.n_heads, cfg.head_dim, c.dev
    rng = np.random.default_rng(59)
    pages = P.KVPages(*(torch.full((B, D, n, d), float("nan"), dtype=torch.float16, device=dev) for _ in range(2)))
    layer = P.PagedAttention(n_heads=n, n_kv_heads=n, head_dim=d, dtype="f16", x_dtype="f32", rope_theta=cfg.theta,
                             max_batch=B, max_tokens=B * D)
    full = torch.full((B,), D, dtype=torch.int32, device=dev)
    middle = T - steps                                                # latent tokens when the decode begins
    dense_pos = np.concatenate([np.arange(sinks), sinks + middle + np.arange(window)])
    k, v = rounded(rng, (B * D, n, d), "f32", 0.25), rounded(rng, (B * D, n, d), "f32")
    rows = P.KVRows(torch.tensor([0, D, 2 * D], dtype=torch.int32, device=dev), full, n_tokens=B * D, max_new=D,
                    max_kv_len=D, positions=torch.from_numpy(np.tile(dense_pos, B).astype(np.int32)).to(dev))
    layer.append(pages, rows, k.to(dev), v.to(dev))
    rk = KO.norm_rope(k.double().numpy(), None, np.tile(dense_pos, B), cfg.theta, 0.0).reshape(B, D, n, d)
    rv = v.double().numpy().reshape(B, D, n, d).copy()
    start = torch.arange(B + 1, dtype=torch.int32, device=dev)
    posd = torch.from_numpy(latent_pos).to(dev)
    for step in range(steps):
        slot, now = sinks + step % window, sinks + middle + window + step
        k1, v1 = rounded(rng, (B, n, d), "f32", 0.25), rounded(rng, (B, n, d), "f32")
        rows = P.KVRows(start, torch.full((B,), slot + 1, dtype=torch.int32, device=dev), n_tokens=B, max_new=1, max_kv_len=D,
                        positions=torch.full((B,), now, dtype=torch.int32, device=dev))
        layer.append(pages, rows, k1.to(dev), v1.to(dev))
        rk[:, slot] = KO.norm_rope(k1.double().numpy(), None, [now] * B, cfg.theta, 0.0)
        rv[:, slot] = v1.double().numpy()
        if step not in (0, 1, window - 1, window, steps - 1):
            continue
        seen = middle + step + 1                                      # the token that left the window is latent now
        out, out_d, lse = c.attn.decode_hybrid(c.q_t.to(dev), c.cache, torch.full((B,), seen, dtype=torch.int32, device=dev),
                                               pages.k, pages.v, full, max_seq_len=T, positions=posd,
                                               q_pos=torch.full((B,), now, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        ref_l, ref_d, ref_lse = O.decode_hybrid(c.q64, c.hk64, c.hv64, c.bk64, [seen] * B, cfg.group_size, rk, rv, [D] * B,
                                               theta=cfg.theta, positions=latent_pos, q_pos=[now] * B)
        assert_close(out.cpu().double().numpy(), ref_l, lse.cpu().double().numpy(), ref_lse)
        assert_close(out_d.cpu().double().numpy(), ref_d)
    c.attn.check_device()
    layer.check_device()
