"""GPU test of the operators together, as a server would run them: plan, append into 8-bit pages, attend, verify, and the next
step from what was accepted, without the host in between; and the same from one captured graph."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8
from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu


class Server:
    """A toy model of one layer: embedded tokens are queries, keys and values, the output's products with a vocabulary the
    logits. Requests draft K tokens each (random ones, of known probabilities) and judge them in one pass."""

    B, K, V, n, m, d, page, pages, per = 5, 3, 97, 4, 2, 64, 16, 40, 12

    def __init__(self, seed):
        from rank_kv_cache_gb300 import palu as P
        i32 = dict(dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gen = g
        N = self.B * (self.K + 1)
        width = (self.n + 2 * self.m) * self.d
        self.embed = torch.randn(self.V, width, generator=g, device="cuda").bfloat16()
        self.head = (torch.randn(self.n * self.d, self.V, generator=g, device="cuda") * 0.3)
        self.layer = P.PagedAttention(n_heads=self.n, n_kv_heads=self.m, head_dim=self.d, dtype="bf16", max_batch=self.B, max_tokens=N)
        self.pool = P.KVPool.empty(self.B, self.per, self.pages, self.page)
        self.cache = P.KVPages8.empty(self.pages, self.page, self.m, self.d)
        self.lens, self.new = torch.zeros(self.B, **i32), torch.full((self.B,), self.K + 1, **i32)
        self.positions, self.slots = torch.zeros(N, **i32), torch.zeros(N, **i32)
        self.rows = P.KVRows(torch.zeros(self.B + 1, **i32), self.lens, page_table=self.pool.page_table, positions=self.positions,
                             n_tokens=N, max_new=self.K + 1, max_kv_len=self.per * self.page)
        self.last = torch.arange(self.B, **i32)                              # the tokens that each request ended with
        self.drafts, self.u = torch.zeros(self.B, self.K, **i32), torch.zeros(self.B, self.K + 1, device="cuda")
        self.q_probs = torch.zeros(self.B, self.K, self.V, device="cuda")
        self.tokens, self.accepted = torch.zeros(self.B, self.K + 1, **i32), torch.zeros(self.B, **i32)
        self.out = torch.zeros(N, self.n, self.d, dtype=torch.bfloat16, device="cuda")
        self.q_rot = torch.zeros_like(self.out)

    def draft(self):
        """New drafts and random numbers, in place: what a draft model would leave."""
        self.q_probs.copy_(torch.softmax(torch.randn(self.q_probs.shape, generator=self.gen, device="cuda"), -1))
        flat = self.q_probs.view(-1, self.V)
        self.drafts.copy_(torch.multinomial(flat, 1, generator=self.gen).view(self.B, self.K))
        self.u.copy_(torch.rand(self.u.shape, generator=self.gen, device="cuda"))

    def step(self):
        L = self.layer
        L.plan(self.pool, self.new, self.lens, self.rows, slots=self.slots)
        x = self.embed[torch.cat([self.last[:, None], self.drafts], 1).reshape(-1).long()]
        q, k, v = (t.unflatten(1, (-1, self.d)) for t in x.split([self.n * self.d, self.m * self.d, self.m * self.d], 1))
        L.append(self.cache, self.rows, k, v, q=q, q_out=self.q_rot)
        L.attend(self.cache, self.rows, self.q_rot, out=self.out)
        self.target = torch.softmax(self.out.float().flatten(1) @ self.head, -1)
        L.verify(self.target, self.drafts, self.u, self.rows.tensors[0], draft=self.q_probs, kv_len=self.lens, tokens=self.tokens,
                 accepted=self.accepted)
        self.last.copy_(self.tokens.gather(1, self.accepted[:, None].long())[:, 0])


def test_steps_match_the_oracles_and_the_graph_the_steps(cuda_device):
    a, b = Server(7), Server(7)
    for s in (a, b):
        s.draft()
    a.step()                                                                  # outside the graph
    b.step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        b.step()
    for t in range(20):                                                       # each leaves one token at least
        for s in (a, b):
            s.draft()
        before, held = a.lens.cpu().numpy().copy(), a.pool.held.cpu().numpy().copy()
        table, ring, state = (x.cpu().numpy().copy() for x in (a.pool.page_table, a.pool.free_pages, a.pool.state))
        drafts, u, q = a.drafts.cpu().numpy(), a.u.cpu().numpy(), a.q_probs.double().cpu().numpy()
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        a.layer.check_device()
        b.layer.check_device()
        for x, y in ((a.tokens, b.tokens), (a.accepted, b.accepted), (a.lens, b.lens), (a.out, b.out), (a.last, b.last),
                     (a.cache.k.view(torch.uint8), b.cache.k.view(torch.uint8)), (a.pool.page_table, b.pool.page_table)):
            assert torch.equal(x, y)
        # the plan
        new = np.full(a.B, a.K + 1)
        start, lens, hold, st, pos, slots, tab, _ = K8.plan(new, before, held, table, ring, state, a.page, a.B * (a.K + 1))
        assert np.array_equal(a.pool.page_table.cpu().numpy(), tab) and np.array_equal(a.slots.cpu().numpy(), slots)
        assert np.array_equal(a.positions.cpu().numpy(), pos)
        # the attention, over the codes as they are now
        vals = [K8.values(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
                for c, s in ((a.cache.k, a.cache.k_scale), (a.cache.v, a.cache.v_scale))]
        o, _, size, reach = KO.attend(a.q_rot.double().cpu().numpy(), *vals, start, lens, tab)
        e = 2.0 ** -16 * reach + 2.0 ** -20 + 2.0 ** -22 * 65
        big = max(float(a.cache.v_scale.max()), 1.0)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * e + 2.0 ** -19) * size + max(lens) * 2.0 ** -32 * big * 448 + 1e-38
        assert np.all(np.abs(a.out.double().cpu().numpy() - o) <= tol)
        # the verification, and what it leaves cached
        p = a.target.double().cpu().numpy()
        for r in range(a.B):
            n_acc, tok = K8.verify(p[start[r]:start[r + 1]], q[r], drafts[r], u[r])
            assert int(a.accepted[r]) == n_acc and int(a.tokens[r, n_acc]) == tok == int(a.last[r])
            assert int(a.lens[r]) == lens[r] - (a.K - n_acc)
    assert int(a.lens.max()) > a.page                                         # pages were taken on the way


def test_a_request_ends_and_another_takes_its_row(cuda_device):
    s = Server(3)
    for t in range(6):
        s.draft()
        s.new.fill_(s.K + 1)
        if t == 3:
            s.new[2] = -1                                                     # ends: its pages go back
        s.layer.plan(s.pool, s.new, s.lens, s.rows, slots=s.slots)
        if t == 3:
            torch.cuda.synchronize()
            assert int(s.lens[2]) == 0 and int(s.pool.held[2]) == 0
            assert int(s.rows.tensors[0][3] - s.rows.tensors[0][2]) == 0
        # tokens of the rows that are there, packed
        n = (s.rows.tensors[0][1:] - s.rows.tensors[0][:-1]).cpu()
        x = s.embed[torch.randint(0, s.V, (s.B * (s.K + 1),), generator=s.gen, device="cuda")]
        q, k, v = (y.unflatten(1, (-1, s.d)) for y in x.split([s.n * s.d, s.m * s.d, s.m * s.d], 1))
        s.layer.append(s.cache, s.rows, k, v, q=q, q_out=s.q_rot)
        s.layer.attend(s.cache, s.rows, s.q_rot, out=s.out)
        target = torch.softmax(s.out.float().flatten(1) @ s.head, -1)
        s.layer.verify(target, s.drafts, s.u, s.rows.tensors[0], draft=s.q_probs, kv_len=s.lens, tokens=s.tokens, accepted=s.accepted)
        torch.cuda.synchronize()
        s.layer.check_device()
        assert [int(c) == 0 for c in n] == [t == 3 and b == 2 for b in range(s.B)]
        if t == 3:
            assert int(s.accepted[2]) == 0 and bool((s.tokens[2] == -1).all())
    free = int(s.pool.state[1])
    assert free + int(s.pool.held.sum()) == s.pages
