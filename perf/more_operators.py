"""Cases of the operators of a serving step over a paged KV cache held in 8 bits: the plan of the step's rows and pages, the
append that quantises, the attention over the codes, and the verification of drafted tokens.

  plan     from each request's new tokens and cached length: the packed rows (row_start), the lengths behind the step, the
           page table's new entries from a ring of free pages (pages of ended requests, new = -1, go to its end), and the
           position and slot of every packed token. Requests are admitted in order; the first whose pages or tokens are
           not there, and all behind it, get none.
  append   keys normed and rotated as in the dense cache, then held as e4m3 codes with one scale, a power of two, for every
           16 slots and head: the least that brings the new tokens' largest magnitude to 448 or below, and no less than the
           old one where older tokens are in the 16 slots, whose codes are restated when it grows. Values likewise, without
           norm and rotation. Queries come back normed and rotated.
  attend   o = softmax(q K^T / sqrt(d)) V over the slots 0 .. L - n + i of the query's row, K and V being codes times scales;
           grouped heads; and the natural log-sum-exp of the scaled scores.
  verify   drafts of a row are accepted while u_i q_i(x_i) < p_i(x_i). Behind the first rejected one a token is drawn from
           max(p - q, 0) (where that is nowhere positive: from p), behind the last accepted one from p: the first whose
           running sum exceeds u times the whole. The cached length loses the rejected tokens.
"""
import math
import random

import torch

own = False

THETA, EPS, BLOCK, TOP = 10000.0, 1e-6, 16, 448.0
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# a drawn case stays below the largest listed ones: padded scores (32 heads x 2048 new tokens), cached elements, tokens,
# probabilities
MOST_SCORES, MOST_CACHE, MOST_TOKENS, MOST_PROBS = 32 * 2048 * 64000, 1 << 29, 1 << 14, 1 << 26


def listed():
    return [
        # a step of 64 requests that decode with five drafts each
        dict(name="plan-drafts", op="plan", batch=64, new=6, kv=16384, page=16, ended=0),
        # a step of 512 requests: some end, some bring chunks of prompts, the others decode
        dict(name="plan-mixed", op="plan", batch=512, new=1024, kv=8192, page=32, ended=20),
        # one decode step of eight requests at unlike lengths
        dict(name="append-step", op="append", dtype="bf16", x_dtype="bf16", heads=32, kv_heads=8, dim=128, page=16,
             table=True, batch=8, new=1, kv=4096, rows="ragged", norm=False),
        # drafts of 16 requests in a layer of small heads, from fp32 projections
        dict(name="append-drafts", op="append", dtype="f16", x_dtype="f32", heads=16, kv_heads=16, dim=64, page=32,
             table=True, batch=16, new=6, kv=2048, rows="ragged", norm=False),
        # four prompts of unlike length at once, grouped heads with normed queries and keys
        dict(name="append-prompt", op="append", dtype="bf16", x_dtype="bf16", heads=32, kv_heads=8, dim=128, page=64,
             table=True, batch=4, new=4096, kv=4096, rows="ragged", norm=True),
        # one token of one request of a small layer: latency
        dict(name="decode-small", op="attend", dtype="f16", heads=8, kv_heads=8, dim=64, page=16, table=True, batch=1,
             new=1, kv=512, rows="same"),
        # one token of four requests at 64K, grouped heads
        dict(name="decode-64k", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, table=True, batch=4,
             new=1, kv=65536, rows="same"),
        # eight requests at unlike lengths, up to five drafted tokens of each to be judged at once
        dict(name="drafts-ragged", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=16, table=True, batch=8,
             new=5, kv=16384, rows="ragged"),
        # four whole prompts of 4K in contiguous caches
        dict(name="prompt-4k", op="attend", dtype="f16", heads=32, kv_heads=32, dim=128, page=4096, table=False, batch=4,
             new=4096, kv=4096, rows="same"),
        # the last chunk of a 64K prompt
        dict(name="chunk-64k", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, table=True, batch=1,
             new=2048, kv=65536, rows="same"),
        # four requests with up to four drafts each, over 32000 tokens
        dict(name="verify-few", op="verify", p_dtype="f32", batch=4, drafts=4, vocab=32000, draft_probs=True),
        # 64 requests with up to six drafts each, over 128K tokens
        dict(name="verify-batch", op="verify", p_dtype="f32", batch=64, drafts=6, vocab=131072, draft_probs=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "verify"])
    if op == "plan":
        batch = _spread(rng, 1, 2048)
        return dict(op=op, batch=batch, new=_spread(rng, 1, min(4096, (1 << 17) // batch)), kv=_spread(rng, 64, 32768),
                    page=rng.choice([8, 16, 24, 32, 64, 128]), ended=rng.choice([0, 0, batch // 16]))
    if op == "verify":
        vocab = rng.choice([_spread(rng, 1000, 1 << 18), 8 * _spread(rng, 500, 1 << 14), 32000, 131072])
        drafts = _spread(rng, 1, 12)
        return dict(op=op, p_dtype=rng.choice(["f32", "f32", "f16", "bf16"]), drafts=drafts, vocab=vocab,
                    batch=_spread(rng, 1, min(256, MOST_PROBS // (vocab * (drafts + 1)))), draft_probs=rng.random() < 0.8)
    heads, kv_heads = rng.choice([(8, 8), (32, 32), (32, 8), (32, 4), (16, 2), (24, 8), (12, 4), (28, 4)])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]))
    if op == "append":
        case["x_dtype"] = rng.choice([case["dtype"], case["dtype"], "f32"])
        case["norm"] = rng.random() < 0.5
    batch = _spread(rng, 1, 32)
    kv = _spread(rng, 1, 65536)
    new = min(kv, 1 if rng.random() < 0.3 else _spread(rng, 1, 4096))
    kv = min(kv, max(1, MOST_CACHE // (batch * kv_heads * case["dim"] * 2)))
    if op == "append":
        kv = min(kv, 8192)
    new = min(new, kv, MOST_TOKENS // batch if op == "append" else max(1, MOST_SCORES // (batch * heads * kv)))
    case.update(page=rng.choice([16, 32, 48, 64, 128, 256]), table=True, batch=batch, new=new, kv=kv,
                rows=rng.choice(["same", "ragged", "ragged", "mixed"]))
    if rng.random() < 0.15:
        case.update(page=-(-kv // BLOCK) * BLOCK + BLOCK * rng.randrange(3), table=False)
    return case


def _rows(case):
    """The new tokens and cached lengths of each row: the same for every seed, so that the work is."""
    b, new, kv = case["batch"], case["new"], case["kv"]
    rng = random.Random(b * 1000003 + new * 1009 + kv)
    if case["rows"] == "same":
        return [new] * b, [kv] * b
    if case["rows"] == "mixed":
        news = [new] + [1] * (b - 1)
    else:
        news = [new] + [rng.randint(max(1, new // 4), new) for _ in range(b - 1)]
    return news, [kv] + [rng.randint(max(n, kv // 4), max(n, kv)) for n in news[1:]]


def _requests(case):
    """The new tokens (-1: the request has ended) and cached lengths of a plan's requests: the same for every seed."""
    b, new, kv = case["batch"], case["new"], case["kv"]
    rng = random.Random(b * 1000003 + new * 1009 + kv + case["ended"])
    news = [rng.randint(max(1, new // 2), new) if rng.random() < 0.1 else rng.randint(1, min(new, 6)) for _ in range(b)]
    for i in rng.sample(range(b), case["ended"]):
        news[i] = -1
    return news, [rng.randint(1, kv) for _ in range(b)]


def _cpu_ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _scale_of(top):
    """2^k with the least k for which top <= 448 * 2^k, k within -64 .. 64."""
    m, e = torch.frexp(top)
    return torch.exp2((e - 9 + (m > 0.875)).clamp(-64, 64).to(top.dtype))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"]}

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    if case["op"] == "plan":
        news, lens = _requests(case)
        b, ps = case["batch"], case["page"]
        held = [-(-L // ps) for L in lens]
        need = [max(0, -(-(L + n) // ps) - h) for n, L, h in zip(news, lens, held)]
        per = max(h + a for h, a in zip(held, need))
        pages = sum(held) + sum(need) + 8
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.full((b, per), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(per, device="cuda")[None] < _cpu_ints(held)[:, None]
        table[at] = order[:sum(held)]
        ring, head = torch.full((pages,), -1, dtype=torch.int32, device="cuda"), pages - pages // 3
        free = order[sum(held):]
        ring[(head + torch.arange(len(free), device="cuda")) % pages] = free
        s.update(table=table, ring=ring, held=_cpu_ints(held), state=_cpu_ints([head, len(free)]), new=_cpu_ints(news),
                 kv_len=_cpu_ints(lens), page=ps, pages=pages, n_tokens=sum(max(0, n) for n in news) + 5,
                 max_kv=max(max(lens), max(L + n for n, L in zip(news, lens))), max_new=max(1, max(news)))
        n = s["n_tokens"]
        for name, size in (("row_start", b + 1), ("kv_out", b), ("held_out", b), ("state_out", 2), ("positions", n), ("slots", n)):
            s[name] = torch.zeros(size, dtype=torch.int32, device="cuda")
    elif case["op"] == "verify":
        b, k, vocab, dt = case["batch"], case["drafts"], case["vocab"], TYPES[case["p_dtype"]]
        rng = random.Random(b * 1009 + k)
        n = [1 + (k if i == 0 else rng.randint(0, k)) for i in range(b)]
        starts = [sum(n[:i]) for i in range(b + 1)]
        s["row_start"], s["k"] = _cpu_ints(starts), k
        target = normal(starts[-1], vocab, scale=2.0)
        of = (s["row_start"][:-1, None] + torch.arange(k, device="cuda")).clamp(max=starts[-1] - 1).long()
        draft = normal(b, k, vocab).add_(target[of])                             # a draft model that is near the target
        noise = torch.rand(b, k, vocab, generator=g, device="cuda").clamp_(min=1e-20).log_().neg_().log_().neg_()
        s["draft_tokens"] = noise.add_(draft).argmax(-1).int()
        s["target"] = torch.softmax(target, -1).to(dt)
        s["draft"] = torch.softmax(draft, -1).to(dt) if case["draft_probs"] else None
        s["u"] = torch.rand(b, k + 1, generator=g, device="cuda")
        s["kv_len"] = torch.randint(k + 1, 4096, (b,), generator=g, device="cuda").int()
        s["kv_out"], s["accepted"] = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))
        s["tokens"] = torch.zeros(b, k + 1, dtype=torch.int32, device="cuda")
    else:
        n, m, d, dt = case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
        news, lens = _rows(case)
        starts = [sum(news[:b]) for b in range(len(news) + 1)]
        N, ps = starts[-1], case["page"]
        per = -(-max(lens) // ps) if case["table"] else 1
        pages = case["batch"] * per + (3 if case["table"] else 0)
        for side in "kv":
            x = normal(pages, ps // BLOCK, BLOCK, m, d)
            x *= normal(pages, ps // BLOCK, 1, m, 1, scale=0.5).exp_()         # blocks of unlike magnitude
            scale = _scale_of(x.abs().amax((2, 4)))
            x /= scale[:, :, None, :, None]
            s["codes_" + side] = x.to(torch.float8_e4m3fn).view(pages, ps, m, d)
            s["scale_" + side] = scale
            del x
        s["table"] = None
        if case["table"]:
            order = torch.randperm(pages, generator=g, device="cuda")[:case["batch"] * per]
            s["table"] = order.int().view(case["batch"], per).contiguous()
        s["row_start"], s["kv_len"] = _cpu_ints(starts), _cpu_ints(lens)
        s.update(n=n, m=m, d=d, dtype=dt, page=ps, max_new=max(news), max_kv=max(lens), N=N)
        if case["op"] == "attend":
            s["q"] = normal(N, n, d, scale=2.0).to(dt)
            s["out"] = torch.zeros(N, n, d, dtype=dt, device="cuda")
            s["lse"] = torch.zeros(N, n, dtype=torch.float32, device="cuda")
        else:
            # queries, keys and values are column blocks of one fused projection's output
            qkv = normal(N, (n + 2 * m) * d, dtype=TYPES[case["x_dtype"]])
            s["q"] = qkv[:, :n * d].unflatten(1, (n, d))
            s["k"] = qkv[:, n * d:(n + m) * d].unflatten(1, (m, d))
            s["v"] = qkv[:, (n + m) * d:].unflatten(1, (m, d))
            s["wq"] = s["wk"] = None
            if case["norm"]:
                s["wq"], s["wk"] = (1 + normal(d, dtype=qkv.dtype, scale=0.2) for _ in range(2))
            s["q_out"] = torch.zeros(N, n, d, dtype=dt, device="cuda")
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program of the framework keeps: the handle and the views of its tensors."""
    from rank_kv_cache_gb300 import palu as P
    if case["op"] == "verify":
        s["layer"] = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=case["batch"],
                                      max_tokens=s["target"].shape[0])
    elif case["op"] == "plan":
        s["layer"] = P.PagedAttention(n_heads=1, n_kv_heads=1, head_dim=64, dtype="f32", max_batch=case["batch"],
                                      max_tokens=s["n_tokens"])
        s["pool"] = P.KVPool(s["table"], s["held"], s["ring"], s["state"], page_size=s["page"])
        s["rows"] = P.KVRows(s["row_start"], s["kv_out"], page_table=s["table"], positions=s["positions"],
                             n_tokens=s["n_tokens"], max_new=s["max_new"], max_kv_len=s["max_kv"])
    else:
        s["layer"] = P.PagedAttention(n_heads=s["n"], n_kv_heads=s["m"], head_dim=s["d"], dtype=case["dtype"],
                                      x_dtype=case.get("x_dtype", case["dtype"]), rope_theta=THETA, norm_eps=EPS,
                                      max_batch=case["batch"], max_tokens=s["N"])
        s["pages"] = P.KVPages8(s["codes_k"], s["codes_v"], s["scale_k"], s["scale_v"])
        s["rows"] = P.KVRows(s["row_start"], s["kv_len"], page_table=s["table"], n_tokens=s["N"], max_new=s["max_new"],
                             max_kv_len=s["max_kv"])


# ---------------------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    ps, cap, T = s["page"], s["pages"], s["n_tokens"]
    new, L, held = s["new"].long(), s["kv_len"].long(), s["held"].long()
    ended, n = new < 0, new.clamp(min=0)
    need = torch.where(n > 0, (-(-(L + n) // ps) - held).clamp(min=0), 0)
    taken, tokens = need.cumsum(0), n.cumsum(0)
    fits = (taken <= s["state"][1]) & (tokens <= T)
    n, need = n * fits, need * fits
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    # pages for the admitted, from the ring's head; those of ended requests behind its end
    row = torch.repeat_interleave(torch.arange(len(n), device=n.device), need, output_size=None)
    j = torch.arange(len(row), device=n.device)
    s["table"][row, held[row] + j - (need.cumsum(0) - need)[row]] = s["ring"][(s["state"][0] + j) % cap]
    back = held * ended
    row = torch.repeat_interleave(torch.arange(len(n), device=n.device), back)
    f = torch.arange(len(row), device=n.device)
    s["ring"][(s["state"][0] + s["state"][1] + f) % cap] = s["table"][row, f - (back.cumsum(0) - back)[row]]
    t = torch.arange(T, device=n.device)
    row = torch.searchsorted(start[1:], t, right=True)
    live = row < len(n)
    row = row.clamp(max=len(n) - 1)
    pos = torch.where(live, L[row] + t - start[row], 0)
    page = s["table"][row, torch.where(live, pos // ps, 0)].long()
    slot = torch.where(live, page * ps + pos % ps, -1)
    all_need, all_back = need.sum(), back.sum()
    state = torch.stack([(s["state"][0] + all_need) % cap, s["state"][1] - all_need + all_back])
    return [x.int() for x in (start, torch.where(ended, 0, L + n), torch.where(ended, 0, held + need), state, pos, slot)] + [
        s["table"], s["ring"]]


def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, pos):
    h = x.shape[-1] // 2
    rate = THETA ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    turn = pos.double()[:, None, None] * rate
    c, s = turn.cos().float(), turn.sin().float()
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


def _row_of_token(s, N):
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    row = torch.searchsorted(s["row_start"][1:].contiguous(), t, right=True)
    return row, t.long() - s["row_start"][row]


def _slots(s, row, t):
    if s["table"] is None:
        return row * s["page"] + t
    return s["table"][row, t // s["page"]].long() * s["page"] + t % s["page"]


def _bytes(codes, m, d):
    return codes.view(torch.uint8).view(-1, m, d)


def _plain_append(s):
    m, d = s["m"], s["d"]
    row, i = _row_of_token(s, s["N"])
    n_new = s["row_start"][1:] - s["row_start"][:-1]
    first = (s["kv_len"] - n_new)[row].long()                                  # slot of the row's first new token
    pos = first + i
    q = _rotate(_norm(s["q"].float(), s["wq"]), pos)
    at = _slots(s, row, pos)
    block = at // BLOCK
    old = (first > pos - pos % BLOCK) & (first - first % BLOCK == pos - pos % BLOCK)   # older tokens share the block
    ids, of = torch.unique(block, return_inverse=True)
    keep = torch.zeros(len(ids), dtype=torch.bool, device="cuda").index_put_((of,), old, accumulate=False)
    begin = torch.full((len(ids),), BLOCK, device="cuda").index_reduce_(0, of, pos % BLOCK, "amin")
    for side, x in (("k", _rotate(_norm(s["k"].float(), s["wk"]), pos)), ("v", s["v"].float())):
        codes, scale = _bytes(s["codes_" + side], m, d), s["scale_" + side].view(-1, m)
        top = torch.zeros(len(ids), m, device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")
        was = scale[ids]
        now = _scale_of(top)
        now = torch.where(keep[:, None], torch.maximum(now, was), now)
        # the older tokens' codes under the new scale
        t = torch.arange(BLOCK, device="cuda")
        older = (keep[:, None] & (t < begin[:, None])).nonzero(as_tuple=True)
        spot = ids[older[0]] * BLOCK + older[1]
        c = codes[spot].view(torch.float8_e4m3fn).float() * (was / now)[older[0]][..., None]
        codes[spot] = c.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[at] = (x / now[of][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[ids] = now
    return [q.to(s["dtype"]), s["codes_k"], s["codes_v"], s["scale_k"], s["scale_v"]]


def _plain_attend(s):
    n, m, d, T, M = s["n"], s["m"], s["d"], s["max_kv"], s["max_new"]
    B, N, g = s["kv_len"].shape[0], s["N"], n // m
    n_new = (s["row_start"][1:] - s["row_start"][:-1]).long()
    t = torch.arange(T, device="cuda")
    short = t < s["kv_len"][:, None]
    at = _slots(s, torch.arange(B, device="cuda")[:, None], t[None, :])

    def values(side):
        x = _bytes(s["codes_" + side], m, d)[at].view(torch.float8_e4m3fn).float()
        return x.mul_(s["scale_" + side].view(-1, m)[at // BLOCK][..., None])  # [B, T, m, d]

    K = values("k").permute(0, 2, 3, 1)
    i = torch.arange(M, device="cuda")
    of = (s["row_start"][:-1, None] + i).clamp(max=N - 1).long()
    q = s["q"][of].float().view(B, M, m, g, d).permute(0, 2, 3, 1, 4).reshape(B, m, g * M, d)
    x = torch.matmul(q, K).mul_(1.0 / math.sqrt(d)).view(B, m, g, M, T)
    del K
    last = (s["kv_len"].long() - n_new)[:, None] + i                          # [B, M]
    x.masked_fill_((t > last[..., None])[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(top.clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    V = values("v").masked_fill_(~short[..., None, None], 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, m, g * M, T), V).view(B, m, g, M, d) / total
    lse = (top + total.log())[..., 0]
    row, j = _row_of_token(s, N)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, n, d)[row, j]
    lse = lse.permute(0, 3, 1, 2).reshape(B, M, n)[row, j]
    return [o.to(s["dtype"]), lse]


def _plain_verify(s):
    k, N = s["k"], s["target"].shape[0]
    first = s["row_start"][:-1].long()
    n = (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(k, device="cuda")
    at, x = (first[:, None] + i).clamp(max=N - 1), s["draft_tokens"].long()
    p = s["target"][at, x].double()
    b = torch.arange(len(n), device="cuda")
    q = torch.ones_like(p) if s["draft"] is None else s["draft"][b[:, None], i, x].double()
    taken = (s["u"][:, :k].double() * q < p) & (i < n[:, None] - 1)
    a = taken.long().cumprod(1).sum(1)
    rejected = a < n - 1
    w = s["target"][first + a].double()
    c = a.clamp(max=k - 1)
    if s["draft"] is None:
        less = w.clone().scatter_(1, x[b, c][:, None], 0.0)
    else:
        less = (w - s["draft"][b, c].double()).clamp_(min=0.0)
    less = torch.where(rejected[:, None], less, w)
    less = torch.where(less.sum(1, keepdim=True) > 0, less, w)
    run_ = less.cumsum(1)
    drawn = torch.searchsorted(run_, s["u"][:, k:].double() * run_[:, -1:], right=True).clamp(max=w.shape[1] - 1)
    j = torch.arange(k + 1, device="cuda")
    tokens = torch.cat([x, x.new_zeros(len(n), 1)], 1)
    tokens = torch.where(j < a[:, None], tokens, torch.where(j == a[:, None], drawn, -1))
    return [tokens.int(), a.int(), (s["kv_len"] - (n - 1 - a)).int()]


def run(s):
    if own:
        if s["op"] == "plan":
            s["layer"].plan(s["pool"], s["new"], s["kv_len"], s["rows"], slots=s["slots"], held_out=s["held_out"],
                            state_out=s["state_out"])
            return [s["row_start"], s["kv_out"], s["held_out"], s["state_out"], s["positions"], s["slots"], s["table"], s["ring"]]
        if s["op"] == "append":
            s["layer"].append(s["pages"], s["rows"], s["k"], s["v"], q=s["q"], q_weight=s["wq"], k_weight=s["wk"],
                              q_out=s["q_out"])
            return [s["q_out"], s["codes_k"], s["codes_v"], s["scale_k"], s["scale_v"]]
        if s["op"] == "attend":
            s["layer"].attend(s["pages"], s["rows"], s["q"], out=s["out"], lse=s["lse"])
            return [s["out"], s["lse"]]
        s["layer"].verify(s["target"], s["draft_tokens"], s["u"], s["row_start"], draft=s["draft"], kv_len=s["kv_len"],
                          tokens=s["tokens"], accepted=s["accepted"], kv_len_out=s["kv_out"])
        return [s["tokens"], s["accepted"], s["kv_out"]]
    if s["op"] == "plan":
        return _plain_plan(s)
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s) if s["op"] == "attend" else _plain_verify(s)


def work(case):
    if case["op"] == "plan":
        news, lens = _requests(case)
        held = [-(-L // case["page"]) for L in lens]
        pages = sum(max(0, -(-(L + n) // case["page"]) - h) if n > 0 else h if n < 0 else 0 for n, L, h in zip(news, lens, held))
        N = sum(max(0, n) for n in news)
        return {"bytes": 4 * (6 * case["batch"] + 5 + 2 * pages + 2 * N), "flops": 0}
    if case["op"] == "verify":
        b, k, e = case["batch"], case["drafts"], BYTES[case["p_dtype"]]
        rows = b * (2 if case["draft_probs"] else 1)                           # p, and q where a draft is rejected
        return {"bytes": rows * case["vocab"] * e + b * k * (2 * e + 8) + 4 * b * (k + 5), "flops": 3 * b * case["vocab"]}
    n, m, d, e = case["heads"], case["kv_heads"], case["dim"], BYTES[case["dtype"]]
    news, lens = _rows(case)
    N = sum(news)
    table = 4 * sum(-(-L // case["page"]) for L in lens) if case["table"] else 0
    if case["op"] == "append":
        b = N * (n + 2 * m) * d * BYTES[case["x_dtype"]] + N * n * d * e + 2 * N * m * d + 8 * m * sum(-(-k // BLOCK) for k in news)
        return {"bytes": b, "flops": N * (n + m) * d * (7 if case["norm"] else 3)}
    seen = sum(k * (L - k) + k * (k + 1) // 2 for k, L in zip(news, lens))
    cache = 2 * m * sum(L * d + 4 * -(-L // BLOCK) for L in lens)
    return {"bytes": 2 * N * n * d * e + 4 * N * n + cache + table, "flops": 4 * seen * n * d}


# ---------------------------------------------------------------------------------------- 64 bits

def _turned(x, w, at):
    """The normed head vectors x [N, h, d] as complex pairs, multiplied by e^(i at rate)."""
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    h = x.shape[-1] // 2
    rate = torch.exp(torch.arange(h, device=x.device).double() * (-math.log(THETA) / h))
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones((), device=x.device, dtype=torch.float64),
                                                            at.double()[:, None] * rate)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _places(s, b, lo, hi):
    if s["table"] is None:
        return torch.arange(b * s["page"] + lo, b * s["page"] + hi, device="cuda")
    flat = (s["table"][b].long()[:, None] * s["page"] + torch.arange(s["page"], device="cuda")).reshape(-1)
    return flat[lo:hi]


def _exact_plan(case, s):
    news, lens, held = s["new"].tolist(), s["kv_len"].tolist(), s["held"].tolist()
    table, ring, (head, count) = s["table"].tolist(), s["ring"].tolist(), s["state"].tolist()
    ps, cap, tail = s["page"], s["pages"], head + count
    start, pos, slot, got, given, full = [0], [], [], 0, 0, False
    for b, n in enumerate(news):
        if n < 0:
            for p in table[b][:held[b]]:
                ring[(tail + given) % cap] = p
                given += 1
            lens[b] = held[b] = n = 0
        want = max(0, -(-(lens[b] + n) // ps) - held[b]) if n else 0
        full = full or got + want > count or start[-1] + n > s["n_tokens"]
        if full:
            n = want = 0
        for _ in range(want):
            table[b][held[b]] = ring[(head + got) % cap]
            held[b] += 1
            got += 1
        for t in range(lens[b], lens[b] + n):
            pos.append(t)
            slot.append(table[b][t // ps] * ps + t % ps)
        lens[b] += n
        start.append(start[-1] + n)
    rest = s["n_tokens"] - len(pos)
    return [torch.tensor(x, dtype=torch.int32) for x in (start, lens, held, [(head + got) % cap, count - got + given],
                                                         pos + [0] * rest, slot + [-1] * rest, table, ring)]


def _exact_verify(case, s):
    k, starts = s["k"], s["row_start"].tolist()
    tokens, accepted, lens = torch.full((case["batch"], k + 1), -1, dtype=torch.int32), [], s["kv_len"].tolist()
    for b in range(case["batch"]):
        p = s["target"][starts[b]:starts[b + 1]].double()
        u, x, n = s["u"][b].double().tolist(), s["draft_tokens"][b].tolist(), len(p) - 1
        a = 0
        while a < n and u[a] * (1.0 if s["draft"] is None else float(s["draft"][b, a, x[a]])) < float(p[a, x[a]]):
            tokens[b, a] = x[a]
            a += 1
        w = p[a]
        if a < n:
            q = torch.zeros_like(w)
            if s["draft"] is None:
                q[x[a]] = math.inf
            else:
                q = s["draft"][b, a].double()
            rest = torch.relu(w - q)
            w = rest if float(rest.sum()) > 0 else w
        passed = torch.cumsum(w, 0)
        tokens[b, a] = int((passed <= u[k] * passed[-1]).sum())
        accepted.append(a)
        lens[b] -= n - a
    return [tokens, torch.tensor(accepted, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)]


def _exact_append(s, news, lens):
    m, d, at, q = s["m"], s["d"], 0, []
    held = {x: s["codes_" + x].double().flatten(0, 1) for x in "kv"}
    scales = {x: s["scale_" + x].double().flatten(0, 1) for x in "kv"}
    for b, (k, L) in enumerate(zip(news, lens)):
        pos, to = torch.arange(L - k, L, device="cuda"), _places(s, b, L - k, L)
        q.append(_turned(s["q"][at:at + k], s["wq"], pos))
        for x, y in (("k", _turned(s["k"][at:at + k], s["wk"], pos)), ("v", s["v"][at:at + k].double())):
            front = (L - k) % BLOCK                                             # older tokens of the first block
            whole = torch.zeros(front + k + -(front + k) % BLOCK, m, d, dtype=torch.float64, device="cuda")
            whole[front:front + k] = y
            block = _places(s, b, L - k - front, L)[::BLOCK] // BLOCK
            top = whole.abs().view(-1, BLOCK, m, d).amax((1, 3))
            to_scale = 2.0 ** torch.ceil(torch.log2((top / TOP).clamp(min=2.0 ** -64))).clamp(-64, 64)
            if front:
                to_scale[0] = torch.maximum(to_scale[0], scales[x][block[0]])
                older = _places(s, b, L - k - front, L - k)
                held[x][older] *= (scales[x][block[0]] / to_scale[0])[:, None]
            scales[x][block] = to_scale
            held[x][to] = y / to_scale.repeat_interleave(BLOCK, 0)[front:front + k, :, None]
        at += k
    return [torch.cat(q)] + [held[x].view(s["codes_" + x].shape) for x in "kv"] + [scales[x].view(s["scale_" + x].shape) for x in "kv"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, s)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    news, lens = _rows(case)
    if case["op"] == "append":
        return _exact_append(s, news, lens)
    n, m, d = s["n"], s["m"], s["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (k, L) in enumerate(zip(news, lens)):
        to = _places(s, b, 0, L)
        hidden = torch.ones(k, L, dtype=torch.bool, device="cuda").triu(L - k + 1)
        for h in range(n):
            kv = h // (n // m)
            K, V = (s["codes_" + x].view(torch.uint8).flatten(0, 1)[to, kv].view(torch.float8_e4m3fn).double()
                    * s["scale_" + x].double().flatten(0, 1)[to // BLOCK, kv][:, None] for x in "kv")
            x = (s["q"][at:at + k, h].double() @ K.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[at:at + k, h] = torch.logsumexp(x, -1)
            o[at:at + k, h] = torch.softmax(x, -1) @ V
        at += k
    return [o, lse]
