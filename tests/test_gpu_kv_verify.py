"""GPU tests of the verification of drafted tokens."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(rng, news, vocab, dtype, certain=False, near=1.0):
    B, K = len(news), max(max(n - 1 for n in news), 0)
    N = sum(news)
    p = torch.from_numpy(rng.standard_normal((N, vocab)).astype(np.float32)) * 3.0
    q = torch.from_numpy(rng.standard_normal((B, K, vocab)).astype(np.float32)) * near
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    drafts = np.zeros((B, K), dtype=np.int32)
    for b, n in enumerate(news):
        for i in range(max(n - 1, 0)):
            q[b, i] += p[starts[b] + i]
    p, q = torch.softmax(p, -1), torch.softmax(q, -1)
    for b in range(B):
        for i in range(K):
            w = q[b, i].double().numpy()
            drafts[b, i] = rng.choice(vocab, p=w / w.sum())
    return dict(target=p.to(TYPES[dtype]), draft=None if certain else q.to(TYPES[dtype]), drafts=drafts, starts=starts,
                u=rng.random((B, K + 1)).astype(np.float32), kv=rng.integers(K + 1, 100, B).astype(np.int32))


def run(c, layer=None, **kw):
    from rank_kv_cache_gb300 import palu as P
    B = len(c["starts"]) - 1
    layer = layer or P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B,
                                      max_tokens=max(1, len(c["target"])))
    kv = torch.from_numpy(c["kv"]).cuda()
    tokens, accepted = layer.verify(c["target"].cuda(), torch.from_numpy(c["drafts"]).cuda(), torch.from_numpy(c["u"]).cuda(),
                                    torch.from_numpy(c["starts"]).cuda(), draft=None if c["draft"] is None else c["draft"].cuda(),
                                    kv_len=kv, **kw)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), accepted.cpu().numpy(), kv.cpu().numpy(), layer


def check(c, tokens, accepted, kv):
    for b in range(len(accepted)):
        lo, hi = int(c["starts"][b]), int(c["starts"][b + 1])
        if hi == lo:
            assert accepted[b] == 0 and np.all(tokens[b] == -1) and kv[b] == c["kv"][b]
            continue
        n = hi - lo
        u = np.concatenate([c["u"][b, :n - 1], c["u"][b, -1:]])
        a, token = K8.verify(c["target"][lo:hi].double().numpy(), None if c["draft"] is None else c["draft"][b].double().numpy(),
                             c["drafts"][b], u)
        want = np.full(tokens.shape[1], -1)
        want[:a] = c["drafts"][b, :a]
        want[a] = token
        assert accepted[b] == a and np.array_equal(tokens[b], want), b
        assert kv[b] == c["kv"][b] - (n - 1 - a)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("news,vocab", [([1], 1), ([2, 1, 0, 3], 7), ([5, 5, 2], 512), ([4, 1, 6], 513), ([3, 3], 1000),
                                        ([2, 9, 1], 5003), ([3], 20000)])
@pytest.mark.parametrize("certain", [False, True])
def test_matches_rational_arithmetic(cuda_device, dtype, news, vocab, certain):
    rng = np.random.default_rng(vocab + len(news))
    for _ in range(3):
        c = make(rng, news, vocab, dtype, certain)
        tokens, accepted, kv, layer = run(c)
        layer.check_device()
        check(c, tokens, accepted, kv)


def test_many_rows_and_forty_drafts(cuda_device):
    rng = np.random.default_rng(1)
    for news in ([int(x) for x in rng.integers(0, 4, 700)], [41, 35, 3]):
        c = make(rng, news, 65, "f32", near=0.05)
        tokens, accepted, kv, layer = run(c)
        layer.check_device()
        check(c, tokens, accepted, kv)
    assert accepted.max() > 32


def test_shares_of_a_draw_follow_the_residual(cuda_device):
    # one distribution, many uniforms on a grid: the counts are the residual's shares to one step
    V, B = 300, 4096
    rng = np.random.default_rng(2)
    p, q = rng.random(V) ** 3, rng.random(V) ** 3
    p, q = (p / p.sum()).astype(np.float32), (q / q.sum()).astype(np.float32)
    x = int(np.argmax(q - p))
    c = dict(target=torch.from_numpy(np.tile(p, (2 * B, 1))), draft=torch.from_numpy(np.tile(q, (B, 1, 1)).reshape(B, 1, V)),
             drafts=np.full((B, 1), x, dtype=np.int32), starts=(2 * np.arange(B + 1)).astype(np.int32),
             u=np.stack([np.full(B, 0.99999), (np.arange(B) + 0.5) / B], 1).astype(np.float32), kv=np.full(B, 9, dtype=np.int32))
    tokens, accepted, kv, layer = run(c)
    assert np.all(accepted == 0) and np.all(kv == 8)
    r = np.maximum(p.astype(np.float64) - q, 0)
    count = np.bincount(tokens[:, 0], minlength=V)
    assert np.all(np.abs(count - B * r / r.sum()) <= 1 + 1e-6)


def test_borders_of_acceptance_and_of_a_draw(cuda_device):
    # u q = p is a rejection; u = 0 draws the first possible token, the largest u the last
    V = 1200
    p = torch.zeros(4, V)
    p[:, [5, 600, 1100]] = 0.25
    q = torch.zeros(2, 1, V)
    q[:, 0, 5] = 0.5
    c = dict(target=p, draft=q, drafts=np.full((2, 1), 5, dtype=np.int32), starts=np.array([0, 2, 4], dtype=np.int32),
             u=np.array([[0.5, 0.0], [np.nextafter(np.float32(0.5), np.float32(0)), 1.0]], dtype=np.float32),
             kv=np.array([3, 3], dtype=np.int32))
    tokens, accepted, _, layer = run(c)
    layer.check_device()
    assert list(accepted) == [0, 1]
    assert tokens[0, 0] == 600                                               # 5 has nothing left of it
    assert list(tokens[1]) == [5, 1100]


def test_nothing_left_falls_back_to_the_target_and_nothing_at_all_is_reported(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    V = 700
    p = torch.zeros(2, V)
    p[0, 650] = 1.0
    p[1, 3] = 1.0
    q = p[:1].clone().view(1, 1, V)
    c = dict(target=p, draft=q, drafts=np.array([[2]], dtype=np.int32), starts=np.array([0, 2], dtype=np.int32),
             u=np.array([[0.3, 0.9]], dtype=np.float32), kv=np.array([3], dtype=np.int32))
    tokens, accepted, _, layer = run(c)
    layer.check_device()
    assert accepted[0] == 0 and list(tokens[0]) == [650, -1]                  # p - q is zero throughout
    c["target"] = torch.zeros(2, V)
    tokens, accepted, _, _ = run(c, layer)
    assert accepted[0] == 0 and list(tokens[0]) == [-1, -1]
    with pytest.raises(P.PaluError):
        layer.check_device()
    c["target"] = torch.full((2, V), float("nan"))
    c["target"][0, 4], c["target"][0, 7] = -1.0, 0.125
    tokens, _, _, _ = run(c, layer)
    layer.check_device()
    assert tokens[0, 0] == 7


def test_bad_drafts_and_rows_are_reported(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(3)
    c = make(rng, [3, 2], 50, "f32", near=0.01)
    c["drafts"][0, 1] = 50
    c["u"][:, :-1] = 0.0
    tokens, accepted, _, layer = run(c)
    assert accepted[0] == 1 and accepted[1] == 1 and 0 <= tokens[0, 1] < 50
    with pytest.raises(P.PaluError):
        layer.check_device()
    c = make(rng, [3, 2], 50, "f32")
    c["starts"] = np.array([0, 4, 2], dtype=np.int32)                         # four rows for two drafts; then back
    _, accepted, kv, _ = run(c, layer)
    assert accepted[1] == 0 and kv[1] == c["kv"][1]
    with pytest.raises(P.PaluError):
        layer.check_device()


def test_large_vocabularies_strides_and_alignment(cuda_device):
    from rank_kv_cache_gb300 import palu as P
    for dtype, vocab, pad, off in (("f32", 131072, 0, 0), ("bf16", 50257, 3, 1), ("f16", 262144, 8, 0), ("f32", 1 << 20, 0, 0)):
        g = torch.Generator().manual_seed(vocab)
        B, K = 3, 2
        p = torch.softmax(torch.randn(B * 3, vocab, generator=g) * 2, -1).to(TYPES[dtype])
        q = torch.softmax(torch.randn(B, K, vocab, generator=g) * 2, -1).to(TYPES[dtype])
        wide_p = torch.zeros(B * 3, vocab + pad + off, dtype=TYPES[dtype], device="cuda")
        wide_q = torch.zeros(B, K, vocab + pad + off, dtype=TYPES[dtype], device="cuda")
        tp, tq = wide_p[:, off:off + vocab], wide_q[:, :, off:off + vocab]
        tp.copy_(p)
        tq.copy_(q)
        drafts = torch.stack([torch.multinomial(q[b].float(), 1, generator=g)[:, 0] for b in range(B)]).int()
        u = torch.rand(B, K + 1, generator=g)
        layer = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=B, max_tokens=9)
        tokens, accepted = layer.verify(tp, drafts.cuda(), u.cuda(), torch.tensor([0, 3, 6, 9], dtype=torch.int32, device="cuda"), draft=tq)
        layer.check_device()
        for b in range(B):
            a = 0
            while a < K and float(u[b, a]) * float(q[b, a, drafts[b, a]]) < float(p[3 * b + a, drafts[b, a]]):
                a += 1
            w = p[3 * b + a].double()
            if a < K:
                w = (w - q[b, a].double()).clamp(min=0)
            run_ = torch.cumsum(w, 0)
            want = int((run_ <= float(u[b, K]) * float(run_[-1])).sum())
            assert int(accepted[b]) == a and int(tokens[b, a]) == want, (vocab, b)


def test_graphs_and_lengths_elsewhere(cuda_device):
    rng = np.random.default_rng(5)
    c = make(rng, [3, 1, 4], 2999, "bf16")
    tokens, accepted, kv, layer = run(c)
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    t2, a2, kv2, _ = run(c, layer, kv_len_out=out)
    assert np.array_equal(tokens, t2) and np.array_equal(accepted, a2)
    assert np.array_equal(kv2, c["kv"]) and np.array_equal(out.cpu().numpy(), kv)
    dev = [torch.from_numpy(x).cuda() for x in (c["drafts"], c["u"], c["starts"])]
    target, draft = c["target"].cuda(), c["draft"].cuda()
    t3, a3 = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.verify(target, dev[0], dev[1], dev[2], draft=draft, tokens=t3, accepted=a3)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(t3.cpu().numpy(), tokens) and np.array_equal(a3.cpu().numpy(), accepted)


# Weights whose sum is subnormal, next to it, or past the largest number. The sums' and products' 48 bits decide each of these draws as
# rational arithmetic does: none lies nearer to a border than 2^-25 of the sum, but those on it (u = 1/2), which are exact.
@pytest.mark.parametrize("name,dtype,vocab,weights", [
    ("one-least", "f32", 700, {650: 2.0 ** -149}), ("seventy-least", "f32", 1300, {5: 30 * 2.0 ** -149, 600: 2.0 ** -149, 1299: 39 * 2.0 ** -149}),
    ("least-normal", "f32", 6000, {3: 2.0 ** -127, 5900: 2.0 ** -127}), ("above-it", "f32", 9000, {1: 3 * 2.0 ** -120, 4100: 2.0 ** -140, 8999: 2.0 ** -119}),
    ("largest", "f32", 9000, {0: 3.0e38, 2000: 3.25e38, 8999: 1.0e38}), ("largest-one", "f32", 600, {9: 3.4028234663852886e38}),
    ("bf16-least", "bf16", 700, {4: 2.0 ** -133, 699: 2.0 ** -132}), ("bf16-largest", "bf16", 700, {4: 2.0 ** 127, 699: 2.0 ** 127}),
    ("f16-least", "f16", 700, {4: 2.0 ** -24, 699: 2.0 ** -23})])
@pytest.mark.parametrize("residual", [False, True])
def test_sums_outside_the_range_draw_a_token(cuda_device, name, dtype, vocab, weights, residual):
    u = np.float32([0.0, 0.25, 0.5, np.nextafter(np.float32(0.5), np.float32(1)), 0.625, 0.75, 0.995, 1 - 2.0 ** -24])
    B, rows = len(u), 2 if residual else 1
    p = torch.zeros(B * rows, vocab, dtype=torch.float64)
    for v, w in weights.items():
        p[::rows, v] = w
    draft, drafts = None, np.zeros((B, rows - 1), dtype=np.int32)
    if residual:                                                              # a draft of token 2, whose p is 0
        draft = torch.zeros(B, 1, vocab)
        draft[:, 0, 2] = 1.0
        draft[:, 0, 8:200] = 2.0 ** -100
        drafts[:] = 2
    c = dict(target=p.to(TYPES[dtype]), draft=None if draft is None else draft.to(TYPES[dtype]), drafts=drafts,
             starts=(rows * np.arange(B + 1)).astype(np.int32), u=np.stack([u] * rows, 1), kv=np.full(B, 9, dtype=np.int32))
    assert np.array_equal(c["target"].double().numpy(), p.float().double().numpy())
    tokens = torch.full((B, rows), 12345, dtype=torch.int32, device="cuda")
    got, accepted, kv, layer = run(c, tokens=tokens)
    layer.check_device()
    assert np.all(accepted == 0)
    check(c, got, accepted, kv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("certain", [False, True])
def test_uniforms_outside_the_range_are_brought_to_its_ends(cuda_device, dtype, certain):
    # two drafts that the target agrees with to the bit (every number below 1 accepts), and one that it gives half as much
    V = 600
    odd = np.float32([1.0, np.nextafter(np.float32(1), np.float32(2)), 2.0, 1e30, np.inf, np.nan, -1.0, -np.inf, -0.0, 1 - 2.0 ** -24])
    B, K = len(odd), 3
    p = torch.zeros(B, K + 1, V)
    p[:, :, [5, 300, 599]] = torch.tensor([0.5, 0.25, 0.25])
    p[:, 2] *= 0.5
    q = torch.zeros(B, K, V)
    q[:, :, [5, 599]] = 0.5
    if certain:
        p[:, :2, 5] = 1.0                                                     # as much as a certain draft's
    for col in range(K + 1):
        u = np.full((B, K + 1), 0.25, dtype=np.float32)
        u[:, col] = odd
        c = dict(target=p.view(-1, V).to(TYPES[dtype]), draft=None if certain else q.to(TYPES[dtype]),
                 drafts=np.full((B, K), 5, dtype=np.int32), starts=((K + 1) * np.arange(B + 1)).astype(np.int32), u=u,
                 kv=np.full(B, 9, dtype=np.int32))
        tokens, accepted, kv, layer = run(c)
        layer.check_device()
        check(c, tokens, accepted, kv)
        if col == 0:
            assert np.all(accepted > 0)


def test_drafts_past_the_bound_leave_the_length(cuda_device):
    # six target rows for two drafts: the first two are judged, and what is not judged is not kept
    from rank_kv_cache_gb300 import palu as P
    rng = np.random.default_rng(6)
    c = make(rng, [3, 3], 50, "f32")
    c["target"] = torch.cat([c["target"], c["target"][:3]])
    c["starts"] = np.array([0, 6, 9], dtype=np.int32)
    c["kv"] = np.array([20, 30], dtype=np.int32)
    for n in (0, 2):                                                          # accepted of the two
        c["u"][:, :2] = 0.0 if n else 0.75
        c["target"][[0, 1, 6, 7], c["drafts"].reshape(-1)] = 0.5
        c["draft"][[0, 0, 1, 1], [0, 1, 0, 1], c["drafts"].reshape(-1)] = 1.0
        tokens, accepted, kv, layer = run(c)
        assert list(accepted) == [n, n] and list(kv) == [20 - (5 - n), 30 - (2 - n)]
        for b, lo in ((0, 0), (1, 6)):
            a, token = K8.verify(c["target"][lo:lo + 3].double().numpy(), c["draft"][b].double().numpy(), c["drafts"][b], c["u"][b])
            assert a == n and list(tokens[b]) == [*c["drafts"][b, :a], token] + [-1] * (2 - a)
        with pytest.raises(P.PaluError):
            layer.check_device()
