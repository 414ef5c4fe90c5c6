"""Cases of the paged KV cache's operators: the norm and rotation of queries and keys, the append that writes
rotated keys and values into the pages, and the attention of new tokens over them.

Three operators, each over packed new tokens of a batch (row b's tokens are row_start[b] .. row_start[b + 1] - 1):

  norm_rope  y = R(pos) (x * rsqrt(mean(x^2) + eps) * w) for every head of the queries and keys; without weights the
             norm is left out. R is the rotate-half rotation of pairs (k, k + d/2) by pos * theta^(-2k/d).
  append     the same for the keys, written with the values to their slots of the paged cache, and for the queries,
             which come back packed. Token i of a row with n new tokens and a cached length L (the new ones counted)
             has slot and position L - n + i.
  attend     o = softmax(q K^T / sqrt(d)) V over the slots 0 .. L - n + i of the query's row, grouped heads, and the
             natural log-sum-exp of the scaled scores.
"""
import math
import random

import torch

own = False

THETA, EPS = 10000.0, 1e-6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# a drawn case stays below the largest listed ones: padded scores (32 heads x 2048 new tokens), cached bytes, tokens
MOST_SCORES, MOST_CACHE, MOST_TOKENS = 32 * 2048 * 64000, 1 << 30, 1 << 14


def listed():
    return [
        # one decode step's queries and keys of eight requests in a layer of 32 heads
        dict(name="rope-step", op="norm_rope", dtype="f16", x_dtype="f16", heads=32, kv_heads=32, dim=128, tokens=8,
             norm=False),
        # a packed prompt of 16384 tokens, grouped heads with normed queries and keys
        dict(name="norm-rope-prompt", op="norm_rope", dtype="bf16", x_dtype="bf16", heads=32, kv_heads=8, dim=128,
             tokens=16384, norm=True),
        # the four sink and 64 window tokens of a small dense cache without a page table, from fp32 projections
        dict(name="append-window", op="append", dtype="f16", x_dtype="f32", heads=8, kv_heads=8, dim=64, page=68,
             table=False, batch=2, new=68, kv=68, rows="same", norm=False),
        # one decode step of eight requests at unlike lengths
        dict(name="append-step", op="append", dtype="f16", x_dtype="f16", heads=32, kv_heads=32, dim=128, page=16,
             table=True, batch=8, new=1, kv=4096, rows="ragged", norm=False),
        # four prompts of unlike length at once, grouped heads with normed queries and keys
        dict(name="append-prompt", op="append", dtype="bf16", x_dtype="bf16", heads=32, kv_heads=8, dim=128, page=64,
             table=True, batch=4, new=4096, kv=4096, rows="ragged", norm=True),
        # one token of one request of a small layer: latency
        dict(name="decode-small", op="attend", dtype="f16", heads=8, kv_heads=8, dim=64, page=16, table=True, batch=1,
             new=1, kv=512, rows="same"),
        # one token of one request in a layer of 32 heads at 4K
        dict(name="decode-4k", op="attend", dtype="f16", heads=32, kv_heads=32, dim=128, page=16, table=True, batch=1,
             new=1, kv=4096, rows="same"),
        # one token of four requests at 64K, grouped heads
        dict(name="decode-64k", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, table=True,
             batch=4, new=1, kv=65536, rows="same"),
        # eight requests at unlike lengths, up to five drafted tokens of each to be judged at once
        dict(name="draft-ragged", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=16, table=True,
             batch=8, new=5, kv=16384, rows="ragged"),
        # a batch of one 512-token chunk among 15 requests that decode
        dict(name="mixed-batch", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=16, table=True,
             batch=16, new=512, kv=16384, rows="mixed"),
        # four whole prompts of 4K in contiguous caches
        dict(name="prompt-4k", op="attend", dtype="f16", heads=32, kv_heads=32, dim=128, page=4096, table=False,
             batch=4, new=4096, kv=4096, rows="same"),
        # the last chunk of a 64K prompt
        dict(name="chunk-64k", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128, page=64, table=True, batch=1,
             new=2048, kv=65536, rows="same"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    heads, kv_heads = rng.choice([(8, 8), (32, 32), (32, 8), (32, 4), (16, 2), (24, 8), (12, 4), (28, 4)])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]))
    if op != "attend":
        case["x_dtype"] = rng.choice([case["dtype"], case["dtype"], "f32"])
        case["norm"] = rng.random() < 0.5
    if op == "norm_rope":
        if rng.random() < 0.2:
            case["dtype"] = case["x_dtype"] = "f32"
        case["tokens"] = _spread(rng, 1, MOST_TOKENS // (2 if case["x_dtype"] == "f32" else 1))
        return case
    batch = _spread(rng, 1, 32)
    kv = _spread(rng, 1, 65536)
    new = min(kv, 1 if rng.random() < 0.3 else _spread(rng, 1, 4096))
    kv = min(kv, max(1, MOST_CACHE // (batch * kv_heads * case["dim"] * 4)))
    if op == "append":
        kv = min(kv, 8192)
    new = min(new, kv, MOST_TOKENS // batch if op == "append" else max(1, MOST_SCORES // (batch * heads * kv)))
    case.update(page=rng.choice([8, 16, 24, 32, 64, 128, 256]), table=True, batch=batch, new=new, kv=kv,
                rows=rng.choice(["same", "ragged", "ragged", "mixed"]))
    if rng.random() < 0.15:
        case.update(page=kv + rng.randrange(8), table=False)
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


def _tokens(case):
    return case["tokens"] if case["op"] == "norm_rope" else sum(_rows(case)[0])


def _cpu_ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, m, d, dt = case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    N = _tokens(case)

    def normal(*shape, dtype=dt, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = {"op": case["op"], "n": n, "m": m, "d": d, "dtype": dt}
    if case["op"] == "attend":
        s["q"] = normal(N, n, d, scale=2.0)
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
    if case["op"] == "norm_rope":
        s["k_out"] = torch.zeros(N, m, d, dtype=dt, device="cuda")
        s["positions"] = torch.randint(0, 131072, (N,), generator=g, device="cuda").int()
    else:
        news, lens = _rows(case)
        starts = [sum(news[:b]) for b in range(len(news) + 1)]
        per = -(-max(lens) // case["page"]) if case["table"] else 1
        pages = case["batch"] * per + (3 if case["table"] else 0)
        s["pages_k"], s["pages_v"] = (normal(pages, case["page"], m, d) for _ in range(2))
        s["table"] = None
        if case["table"]:
            order = torch.randperm(pages, generator=g, device="cuda")[:case["batch"] * per]
            s["table"] = order.int().view(case["batch"], per).contiguous()
        s["row_start"], s["kv_len"] = _cpu_ints(starts), _cpu_ints(lens)
        s["max_new"], s["max_kv"], s["page"] = max(news), max(lens), case["page"]
    if own:
        from rank_kv_cache_gb300 import palu as P
        names = {v: k for k, v in TYPES.items()}
        s["layer"] = P.PagedAttention(n_heads=n, n_kv_heads=m, head_dim=d, dtype=names[dt],
                                      x_dtype=case.get("x_dtype", case["dtype"]), rope_theta=THETA, norm_eps=EPS,
                                      max_batch=case.get("batch", 1), max_tokens=N)
        if case["op"] != "norm_rope":
            s["pages"] = P.KVPages(s["pages_k"], s["pages_v"])
            s["rows"] = P.KVRows(s["row_start"], s["kv_len"], page_table=s["table"], n_tokens=N,
                                 max_new=s["max_new"], max_kv_len=s["max_kv"])
    return s


# ---------------------------------------------------------------------------------------- plain forms

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


def _plain_append(s):
    row, i = _row_of_token(s, s["q"].shape[0])
    n_new = s["row_start"][1:] - s["row_start"][:-1]
    pos = s["kv_len"][row] - n_new[row] + i
    q = _rotate(_norm(s["q"].float(), s["wq"]), pos)
    k = _rotate(_norm(s["k"].float(), s["wk"]), pos)
    at = _slots(s, row, pos)
    s["pages_k"].view(-1, s["m"], s["d"])[at] = k.to(s["dtype"])
    s["pages_v"].view(-1, s["m"], s["d"])[at] = s["v"].to(s["dtype"])
    return q.to(s["dtype"])


def _plain_attend(s):
    n, m, d, T, M = s["n"], s["m"], s["d"], s["max_kv"], s["max_new"]
    B, N, g = s["kv_len"].shape[0], s["q"].shape[0], n // m
    n_new = (s["row_start"][1:] - s["row_start"][:-1]).long()
    t = torch.arange(T, device="cuda")
    at = _slots(s, torch.arange(B, device="cuda")[:, None], t[None, :])
    K = s["pages_k"].view(-1, m, d)[at].float().permute(0, 2, 3, 1)            # [B, m, d, T]
    V = s["pages_v"].view(-1, m, d)[at].float().permute(0, 2, 1, 3)            # [B, m, T, d]
    i = torch.arange(M, device="cuda")
    of = (s["row_start"][:-1, None] + i).clamp(max=N - 1).long()
    q = s["q"][of].float().view(B, M, m, g, d).permute(0, 2, 3, 1, 4).reshape(B, m, g * M, d)
    x = torch.matmul(q, K).mul_(1.0 / math.sqrt(d)).view(B, m, g, M, T)
    last = (s["kv_len"].long() - n_new)[:, None] + i                          # [B, M]
    x.masked_fill_((t > last[..., None])[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(top.clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, m, g * M, T), V).view(B, m, g, M, d) / total
    lse = (top + total.log())[..., 0]
    row, j = _row_of_token(s, N)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, n, d)[row, j]
    lse = lse.permute(0, 3, 1, 2).reshape(B, M, n)[row, j]
    return o.to(s["dtype"]), lse


def run(s):
    if s["op"] == "norm_rope":
        if own:
            return list(s["layer"].norm_rope(s["q"], s["k"], s["positions"], q_weight=s["wq"], k_weight=s["wk"],
                                             q_out=s["q_out"], k_out=s["k_out"]))
        return [_rotate(_norm(s["q"].float(), s["wq"]), s["positions"]).to(s["dtype"]),
                _rotate(_norm(s["k"].float(), s["wk"]), s["positions"]).to(s["dtype"])]
    if s["op"] == "append":
        if own:
            s["layer"].append(s["pages"], s["rows"], s["k"], s["v"], q=s["q"], q_weight=s["wq"], k_weight=s["wk"],
                              q_out=s["q_out"])
            return [s["q_out"], s["pages_k"], s["pages_v"]]
        return [_plain_append(s), s["pages_k"], s["pages_v"]]
    if own:
        s["layer"].attend(s["pages"], s["rows"], s["q"], out=s["out"], lse=s["lse"])
        return [s["out"], s["lse"]]
    return list(_plain_attend(s))


def work(case):
    n, m, d, N = case["heads"], case["kv_heads"], case["dim"], _tokens(case)
    e = BYTES[case["dtype"]]
    if case["op"] == "norm_rope":
        b = N * (n + m) * d * (BYTES[case["x_dtype"]] + e) + 4 * N
        return {"bytes": b, "flops": N * (n + m) * d * (7 if case["norm"] else 3)}
    news, lens = _rows(case)
    table = 4 * sum(-(-L // case["page"]) for L in lens) if case["table"] else 0
    if case["op"] == "append":
        b = N * (n + 2 * m) * d * (BYTES[case["x_dtype"]] + e) + 8 * len(lens) + 4
        return {"bytes": b, "flops": N * (n + m) * d * (7 if case["norm"] else 3)}
    seen = sum(k * (L - k) + k * (k + 1) // 2 for k, L in zip(news, lens))
    return {"bytes": 2 * N * n * d * e + 4 * N * n + 2 * sum(lens) * m * d * e + table, "flops": 4 * seen * n * d}


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_turned(s["q"], s["wq"], s["positions"]), _turned(s["k"], s["wk"], s["positions"])]
    news, lens = _rows(case)

    def places(b, lo, hi):
        if s["table"] is None:
            return torch.arange(b * s["page"] + lo, b * s["page"] + hi, device="cuda")
        flat = (s["table"][b].long()[:, None] * s["page"] + torch.arange(s["page"], device="cuda")).reshape(-1)
        return flat[lo:hi]

    if case["op"] == "append":
        K, V = s["pages_k"].double().flatten(0, 1), s["pages_v"].double().flatten(0, 1)
        q, at = [], 0
        for b, (k, L) in enumerate(zip(news, lens)):
            pos, to = torch.arange(L - k, L, device="cuda"), places(b, L - k, L)
            q.append(_turned(s["q"][at:at + k], s["wq"], pos))
            K[to] = _turned(s["k"][at:at + k], s["wk"], pos)
            V[to] = s["v"][at:at + k].double()
            at += k
        return [torch.cat(q), K.view(s["pages_k"].shape), V.view(s["pages_v"].shape)]
    n, m, d = s["n"], s["m"], s["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (k, L) in enumerate(zip(news, lens)):
        to = places(b, 0, L)
        hidden = torch.ones(k, L, dtype=torch.bool, device="cuda").triu(L - k + 1)
        for h in range(n):
            kv = h // (n // m)
            K, V = s["pages_k"].flatten(0, 1)[to, kv].double(), s["pages_v"].flatten(0, 1)[to, kv].double()
            x = (s["q"][at:at + k, h].double() @ K.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[at:at + k, h] = torch.logsumexp(x, -1)
            o[at:at + k, h] = torch.softmax(x, -1) @ V
        at += k
    return [o, lse]
