"""Cases for the serving operators: page tables, cache writes, shared-prefix attention, sampling.

Each case is one call (attention: a step's plan and one layer's attention) at
sizes of the repository's model (40 query heads and 8 key/value heads of 128,
a vocabulary of 151,936) or of generic ones.  `own` picks the framework's
calls; otherwise the same operators run in elementary torch operations.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

VOCAB = 151_936
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_MASS_BITS = 44  # fraction bits of a token's weight in afx_sample


def _afx():
    from weight_streaming_canonical_gb300 import afx
    return afx


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: every request grows by one token, one in 16 needs a page
        {"name": "tables step", "op": "tables", "requests": 8, "page": 16, "cached": 700, "new": 1, "finish": 0.0},
        # a scheduler step of a large batch: some requests end, some start with a whole prompt, the rest decode
        {"name": "tables admit", "op": "tables", "requests": 4096, "page": 32, "cached": 3000, "new": 1500, "finish": 0.1},
        # the keys and values of one decode step of 64 requests, one layer
        {"name": "write step", "op": "write", "tokens": 64, "kv_heads": 8, "dim": 128, "page": 16, "type": "bf16"},
        # a prompt batch's keys and values, one layer, an odd number of tokens
        {"name": "write prompt", "op": "write", "tokens": 32_701, "kv_heads": 8, "dim": 128, "page": 64, "type": "fp16"},
        # four requests on a short system prompt: latency counts
        {"name": "attention step 4", "op": "attention", "requests": 4, "new": 1, "prefix": 1003, "own_len": 37,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 16, "type": "bf16"},
        # an ordinary decode step: 64 requests on a long system prompt, up to 1000 tokens of their own
        {"name": "attention step 64", "op": "attention", "requests": 64, "new": 1, "prefix": 8192, "own_len": 1000,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 16, "type": "bf16"},
        # two questions about one very long document: bound by reading the cache
        {"name": "attention document", "op": "attention", "requests": 2, "new": 1, "prefix": 131_000, "own_len": 300,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 64, "type": "fp16"},
        # prompts of up to 500 tokens behind a shared prefix: bound by the products
        {"name": "attention prompts", "op": "attention", "requests": 16, "new": 500, "prefix": 4100, "own_len": 500,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 32, "type": "bf16"},
        # several draft tokens a request checked at once, heads of 64
        {"name": "attention drafts", "op": "attention", "requests": 32, "new": 6, "prefix": 2000, "own_len": 6000,
         "q_heads": 32, "kv_heads": 4, "dim": 64, "page": 128, "type": "fp16"},
        # one request's next token from the fused GEMV's float32 logits: latency counts
        {"name": "sample 1", "op": "sample", "rows": 1, "vocab": VOCAB, "type": "fp32"},
        # an ordinary batch with 16-bit logits
        {"name": "sample 64", "op": "sample", "rows": 64, "vocab": VOCAB, "type": "bf16"},
        # the largest batch, float32 logits of the prefill product
        {"name": "sample 512", "op": "sample", "rows": 512, "vocab": VOCAB, "type": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "attention", "attention", "sample"])
    if op == "tables":
        return {"op": op, "requests": _log_int(rng, 1, 4096), "page": rng.choice([16, 32, 64, 128]),
                "cached": _log_int(rng, 1, 3000), "new": _log_int(rng, 1, 1500), "finish": rng.choice([0.0, 0.05, 0.2])}
    if op == "write":
        return {"op": op, "tokens": _log_int(rng, 1, 32_701), "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "fp16"])}
    if op == "sample":
        return {"op": op, "rows": _log_int(rng, 1, 512), "vocab": rng.choice([VOCAB, _log_int(rng, 500, VOCAB)]),
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    q_heads, kv_heads, dim = rng.choice([(40, 8, 128), (40, 8, 128), (32, 4, 64), (16, 16, 128), (24, 2, 128), (7, 1, 64)])
    new = rng.choice([1, 1, 1, _log_int(rng, 2, 12), _log_int(rng, 12, 400)])
    requests = _log_int(rng, 1, 128 if new <= 12 else 16)
    own_len = _log_int(rng, new, 6000 if new <= 12 else max(600, new))
    prefix = rng.choice([0, _log_int(rng, 1, 4096), _log_int(rng, 256, 131_000)])
    # no more than the largest listed cases: the scores of the prompts' case, the cache of the document's
    prefix = min(prefix, int(600_000_000 / (requests * new * q_heads)), int(1.3e8 / (kv_heads * dim)))
    own_len = max(new, min(own_len, int(600_000_000 / (requests * new * q_heads)), int(1.3e8 / (kv_heads * dim * requests))))
    return {"op": "attention", "requests": requests, "new": new, "prefix": prefix, "own_len": own_len, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "fp16"])}


def _lengths(case, seed):
    """The lengths of a case's requests: (old, new) for the tables, (new tokens, cached tokens) for attention.
    A case's lengths are the same for every seed (so its outputs' shapes are), in an order of the seed's own."""
    rng = random.Random(13)
    a, b = [], []
    for _ in range(case["requests"]):
        if case["op"] == "tables":
            old = rng.randint(0, case["cached"])
            kind = rng.random()
            if kind < case["finish"]:
                new = 0                                    # the request has ended
            elif kind < 2 * case["finish"]:
                old, new = 0, rng.randint(1, case["new"])  # a request starts with its prompt
            elif kind < 2.2 * case["finish"]:
                new = max(0, old - rng.randint(0, 8))      # draft tokens taken back
            else:
                new = old + 1
            a.append(old)
            b.append(new)
        else:
            n = rng.randint(max(1, case["new"] * 2 // 5), case["new"]) if case["new"] > 1 else 1
            a.append(n)
            b.append(max(n, rng.randint(max(1, case["own_len"] // 5), case["own_len"])))
    pairs = list(zip(a, b))
    random.Random(seed).shuffle(pairs)
    return [x for x, _ in pairs], [y for _, y in pairs]


def _pages(n, page):
    return -(-n // page)


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    _PREPARE[case["op"]](s, case, seed, g)
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_tables(s, case, seed, g):
    old, new = _lengths(case, seed)
    page, n = case["page"], case["requests"]
    held = [_pages(v, page) for v in old]
    cols = max(_pages(max(o, v), page) for o, v in zip(old, new)) + 1
    total = sum(held) + sum(_pages(v, page) for v in new) + 64
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    held_t = _ints(held)
    first = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(cols, device="cuda")
    at = (first[:, None] + col[None, :]).clamp(max=total - 1)
    s["table"] = torch.where(col[None, :] < held_t[:, None], ids[at], torch.full_like(ids[at], -1)).contiguous()
    free = ids[sum(held):]
    s["free"] = torch.cat([free, torch.full((sum(held),), -1, dtype=torch.int32, device="cuda")])
    s["count"] = _ints([free.numel()])
    s["count_out"] = torch.zeros_like(s["count"])
    s["old"], s["new"] = _ints(old), _ints(new)
    s["tokens"] = max(1, sum(max(0, v - o) for o, v in zip(old, new)) + 5)  # a few rows of padding
    s["starts"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    s["slots"] = torch.zeros(s["tokens"], dtype=torch.int32, device="cuda")
    s["positions"] = torch.zeros(s["tokens"], dtype=torch.int32, device="cuda")


def _pools(n_pages, case, g):
    shape = (n_pages, case["page"], case["kv_heads"], case["dim"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(_TYPES[case["type"]])
            if math.prod(shape) < 1 << 28 else
            torch.randn(shape, generator=g, device="cuda", dtype=_TYPES[case["type"]]) for _ in range(2)]


def _prepare_write(s, case, seed, g):
    n, page = case["tokens"], case["page"]
    pages = _pages(n, page) + 3
    s["k_pool"], s["v_pool"] = _pools(pages, case, g)
    # the rows of one fused q/k/v product: keys and values are strided views of it
    width = case["kv_heads"] * case["dim"]
    rows = torch.randn((n, 3 * width), generator=g, device="cuda").to(_TYPES[case["type"]])
    s["k"] = rows[:, width:2 * width].unflatten(1, (case["kv_heads"], case["dim"]))
    s["v"] = rows[:, 2 * width:].unflatten(1, (case["kv_heads"], case["dim"]))
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(n, device="cuda")
    s["slots"] = (order[i // page] * page + i % page).to(torch.int32)
    s["slots"][n // 2] = -1  # a row of padding
    if own:
        s["cache"] = _afx().kv_cache(s["k_pool"], s["v_pool"])


def _prepare_attention(s, case, seed, g):
    new, held = _lengths(case, seed)
    page, prefix = case["page"], case["prefix"]
    n_prefix = _pages(prefix, page)
    cols = max(_pages(v, page) for v in held)
    total = n_prefix + sum(_pages(v, page) for v in held)
    s["k_pool"], s["v_pool"] = _pools(total, case, g)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    s["prefix_table"] = ids[:n_prefix].contiguous()
    held_t = _ints([_pages(v, page) for v in held])
    first = torch.cumsum(held_t, 0) - held_t + n_prefix
    col = torch.arange(cols, device="cuda")
    at = (first[:, None] + col[None, :]).clamp(max=total - 1)
    s["table"] = torch.where(col[None, :] < held_t[:, None], ids[at], torch.full_like(ids[at], -1)).contiguous()
    s["lens"] = _ints(held)
    s["starts"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(_ints(new), 0).to(torch.int32)])
    s["tokens"], s["max_new"], s["max_len"] = sum(new), max(new), max(held)
    # the rows of one fused q/k/v product: the queries are a strided view of it
    width = case["q_heads"] * case["dim"]
    rows = torch.randn((s["tokens"], width + 64), generator=g, device="cuda").to(_TYPES[case["type"]])
    s["q"] = rows[:, :width].unflatten(1, (case["q_heads"], case["dim"]))
    s["scale"] = 1.0 / math.sqrt(case["dim"])
    s["out"] = torch.zeros((s["tokens"], case["q_heads"], case["dim"]), dtype=_TYPES[case["type"]], device="cuda")
    s["lse"] = torch.zeros((s["tokens"], case["q_heads"]), dtype=torch.float32, device="cuda")
    if own:
        afx = _afx()
        s["args"] = afx.attention_args(afx.kv_cache(s["k_pool"], s["v_pool"]), case["q_heads"], s["tokens"], s["starts"],
                                       s["lens"], s["table"], s["scale"], prefix_table=s["prefix_table"], prefix_len=prefix)
        s["workspace"] = torch.empty(afx.afx_attention_workspace(s["args"]), dtype=torch.uint8, device="cuda")


def _prepare_sample(s, case, seed, g):
    rows, vocab = case["rows"], case["vocab"]
    z = torch.randn((rows, vocab), generator=g, device="cuda") * 2.5
    spikes = torch.randint(0, vocab, (rows, 24), generator=g, device="cuda")
    z.scatter_add_(1, spikes, torch.rand((rows, 24), generator=g, device="cuda") * 12)  # the few tokens that fit
    z[:, vocab - vocab // 64:] = -math.inf  # the table's padding rows
    s["logits"] = z.to(_TYPES[case["type"]])
    rng = random.Random(seed * 104_729 + 7)
    pick = [(rng.choice([0.0, 0.6, 0.7, 1.0, 1.0, 1.3]), rng.choice([0, 0, 20, 50, 1000]), rng.choice([1.0, 0.8, 0.9, 0.95]),
             rng.choice([0.0, 0.0, 0.02, 0.1])) if r else (0.7, 50, 0.9, 0.0) for r in range(rows)]
    for k, name in enumerate(("temperature", "top_k", "top_p", "min_p")):
        s[name] = torch.tensor([p[k] for p in pick], dtype=torch.int32 if name == "top_k" else torch.float32, device="cuda")
    s["u"] = torch.rand(rows, generator=g, device="cuda")
    s["token"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.zeros(rows, dtype=torch.float32, device="cuda")


_PREPARE = {"tables": _prepare_tables, "write": _prepare_write, "attention": _prepare_attention, "sample": _prepare_sample}


# ---- one pass -----------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_tables(s):
    _afx().afx_kv_tables(s["page"], s["old"], s["new"], s["table"], s["free"], s["count"], s["count_out"], s["starts"],
                         s["slots"], s["positions"], status_dev=s["status"])
    return {k: s[k] for k in ("table", "free", "count_out", "starts", "slots", "positions")}


def _own_write(s):
    _afx().afx_kv_write(s["cache"], s["k"], s["v"], s["slots"], status_dev=s["status"])
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_attention(s):
    afx = _afx()
    afx.afx_attention_plan(s["args"], s["workspace"], status_dev=s["status"])
    afx.afx_attention(s["args"], s["q"], s["out"], s["workspace"], lse=s["lse"], status_dev=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_sample(s):
    _afx().afx_sample(s["logits"], s["u"], s["token"], logprobs=s["logprob"], temperature=s["temperature"],
                      top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"token": s["token"], "logprob": s["logprob"]}


def _exclusive(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(s):
    page, old, new, table, free = s["page"], s["old"].long(), s["new"].long(), s["table"].long(), s["free"].long()
    p_old, p_new = (old + page - 1) // page, (new + page - 1) // page
    grow, drop, add = (p_new - p_old).clamp(min=0), (p_old - p_new).clamp(min=0), (new - old).clamp(min=0)
    g0, d0, t0 = _exclusive(grow), _exclusive(drop), _exclusive(add)
    n_grow, n_drop, n_add, count = grow.sum(), drop.sum(), add.sum(), s["count"].long()[0]

    def freed(f):  # the f-th page given back, in request order
        f = f.clamp(min=0)
        r = (torch.searchsorted(d0 + drop, f, right=True)).clamp(max=old.numel() - 1)
        return table[r, (p_new[r] + f - d0[r]).clamp(min=0, max=table.shape[1] - 1)]

    def taken(j):  # the j-th page handed out, in request order: the last given back first, then the stack's top
        return torch.where(j < n_drop, freed(n_drop - 1 - j), free[(count - 1 - (j - n_drop)).clamp(min=0, max=free.numel() - 1)])

    col = torch.arange(table.shape[1], device=table.device)[None, :]
    is_new = (col >= p_old[:, None]) & (col < p_new[:, None])
    after = torch.where(is_new, taken(g0[:, None] + col - p_old[:, None]), table)
    i = torch.arange(free.numel(), device=table.device)
    stack = torch.where((i >= count) & (i < count + n_drop - n_grow), freed(i - count), free)
    t = torch.arange(s["tokens"], device=table.device)
    r = torch.searchsorted(t0 + add, t, right=True).clamp(max=old.numel() - 1)
    pos = old[r] + t - t0[r]
    slot = after[r, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    live = t < n_add
    starts = torch.cat([t0, n_add[None]])
    out = {"table": after, "free": stack, "count_out": (count + n_drop - n_grow)[None], "starts": starts,
           "slots": torch.where(live, slot, -1), "positions": torch.where(live, pos, -1)}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_write(s):
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    for pool, x in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
        pool.flatten(0, 1)[slots] = x[live]
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attention(s):
    q, starts, lens, page = s["q"].float(), s["starts"].long(), s["lens"].long(), s["page"]
    kvh, group, dim, n = s["kv_heads"], s["q_heads"] // s["kv_heads"], s["dim"], q.shape[0]
    q = q.reshape(n, kvh, group, dim) * s["scale"]
    # the prefix: every token's rows against one copy of its keys
    at = torch.arange(s["prefix"], device=q.device)
    slot = s["prefix_table"].long()[at // page] * page + at % page
    k, v = (p.flatten(0, 1)[slot].float().permute(1, 0, 2) for p in (s["k_pool"], s["v_pool"]))  # [kvh][L][dim]
    rows = q.permute(1, 0, 2, 3).reshape(kvh, n * group, dim)
    x = rows @ k.transpose(1, 2)
    m1 = x.amax(-1, keepdim=True) if s["prefix"] else torch.full((kvh, n * group, 1), -math.inf, device=q.device)
    x = torch.exp(x - m1)
    l1, o1 = x.sum(-1, keepdim=True), x @ v
    back = lambda a: a.reshape(kvh, n, group, -1).permute(1, 0, 2, 3)  # noqa: E731
    m1, l1, o1 = back(m1), back(l1), back(o1)
    # the requests' own tokens, padded to the longest
    i = torch.arange(s["max_new"], device=q.device)
    j = torch.arange(s["max_len"], device=q.device)
    new = starts[1:] - starts[:-1]
    token = (starts[:-1, None] + i[None, :]).clamp(max=n - 1)
    slot = s["table"].long()[:, j // page].clamp(min=0) * page + j % page
    k, v = (p.flatten(0, 1)[slot].float().permute(0, 2, 1, 3) for p in (s["k_pool"], s["v_pool"]))  # [r][kvh][S][dim]
    rows = q[token].permute(0, 2, 1, 3, 4).reshape(-1, kvh, s["max_new"] * group, dim)
    x = (rows @ k.transpose(2, 3)).reshape(-1, kvh, s["max_new"], group, s["max_len"])
    seen = j[None, None, :] <= (lens - new)[:, None, None] + i[None, :, None]  # [r][i][j]
    x = x.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m2 = x.amax(-1, keepdim=True)
    x = torch.exp(x - m2)
    l2 = x.sum(-1, keepdim=True)
    o2 = (x.reshape(-1, kvh, s["max_new"] * group, s["max_len"]) @ v).reshape(-1, kvh, s["max_new"], group, dim)
    t = torch.arange(n, device=q.device)
    r = torch.searchsorted(starts[1:], t, right=True)
    pick = lambda a: a.permute(0, 2, 1, 3, 4)[r, t - starts[r]]  # noqa: E731
    m2, l2, o2 = pick(m2), pick(l2), pick(o2)
    m = torch.maximum(m1, m2)
    e1, e2 = torch.exp(m1 - m), torch.exp(m2 - m)
    if not s["prefix"]:
        l1, o1 = torch.zeros_like(l2), torch.zeros_like(o2)
    total = l1 * e1 + l2 * e2
    out = (o1 * e1 + o2 * e2) / total
    return {"out": out.reshape(n, -1, dim).to(s["q"].dtype), "lse": (m + torch.log(total)).reshape(n, -1)}


def _plain_sample(s):
    z = s["logits"].float()
    z = torch.where(torch.isnan(z), -math.inf, z)
    m = z.amax(1, keepdim=True)
    greedy = ~(s["temperature"][:, None] > 0)
    y = (z - m) * (1.0 / torch.where(greedy, 1.0, s["temperature"][:, None]))
    y = torch.where(z == m, 0.0, torch.where(greedy | (z == -math.inf), -math.inf, y))
    w = torch.exp(y)
    mass = (w * 2.0 ** _MASS_BITS).to(torch.int64)
    _, order = torch.sort(z, dim=1, descending=True, stable=True)
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], z.shape[1])[:, None]
    k = torch.where(greedy, 1, k)
    by_rank = torch.where(rank < k, mass.gather(1, order), 0)
    run_sum = torch.cumsum(by_rank, 1)
    top = run_sum[:, -1:]
    p = s["top_p"][:, None]
    limit = torch.where(p < 1, torch.ceil(p.double() * top.double()).to(torch.int64).clamp(min=1), top)
    keep = (rank < k) & (run_sum - by_rank < limit)
    keep = torch.zeros_like(keep).scatter_(1, order, keep) & (w >= s["min_p"][:, None].clamp(max=1))
    run_sum = torch.cumsum(torch.where(keep, mass, 0), 1)
    total = run_sum[:, -1:]
    aim = torch.minimum((s["u"][:, None].double() * total.double()).to(torch.int64), total - 1)
    token = (run_sum <= aim).sum(1, keepdim=True)
    logprob = y.gather(1, token) - torch.log(total.float() * 2.0 ** -_MASS_BITS)
    return {"token": token[:, 0].to(torch.int32), "logprob": logprob[:, 0]}


_OWN = {"tables": _own_tables, "write": _own_write, "attention": _own_attention, "sample": _own_sample}
_PLAIN = {"tables": _plain_tables, "write": _plain_write, "attention": _plain_attention, "sample": _plain_sample}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "tables":
        old, new = _lengths(case, 1)
        page = case["page"]
        moved = sum(abs(_pages(v, page) - _pages(o, page)) for o, v in zip(old, new))
        tokens = sum(max(0, v - o) for o, v in zip(old, new))
        # lengths read; page ids read and written; starts, slots and positions written
        return {"bytes": 8 * len(old) + 8 * moved + 4 * (len(old) + 1) + 8 * tokens, "flops": 0}
    if case["op"] == "write":
        return {"bytes": case["tokens"] * (4 + 2 * 2 * 2 * case["kv_heads"] * case["dim"]), "flops": 0}
    if case["op"] == "attention":
        new, held = _lengths(case, 1)
        tokens = sum(new)
        seen = sum(n * (h - n) + n * (n + 1) // 2 for n, h in zip(new, held)) + tokens * case["prefix"]
        cache = 2 * 2 * (case["prefix"] + sum(held)) * case["kv_heads"] * case["dim"]
        return {"bytes": cache + tokens * case["q_heads"] * (2 * 2 * case["dim"] + 4),
                "flops": 4 * case["q_heads"] * case["dim"] * seen}
    size = 4 if case["type"] == "fp32" else 2
    return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": 0}


# ---- the definitions, in 64 bits ----------------------------------------------------

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "sample" and case["rows"] * case["vocab"] <= 80_000_000:
        return _exact_sample(prepare(case, seed))
    return None  # whole numbers, or copies


def _exact_attention(s):
    """Request by request: softmax over the prefix and the request's own visible tokens, laid side by side."""
    page, group = s["page"], s["q_heads"] // s["kv_heads"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for r, length in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        ids = torch.cat([s["prefix_table"][:_pages(s["prefix"], page)].repeat_interleave(page)[:s["prefix"]],
                         s["table"][r, :_pages(length, page)].repeat_interleave(page)[:length]]).long()
        off = torch.cat([torch.arange(s["prefix"], device="cuda"), torch.arange(length, device="cuda")]) % page
        hidden = torch.arange(s["prefix"] + length, device="cuda")[None, :] > \
            (s["prefix"] + length - (b - a) + torch.arange(b - a, device="cuda"))[:, None]
        for h in range(s["kv_heads"]):
            keys, values = s["k_pool"][ids, off, h].double(), s["v_pool"][ids, off, h].double()
            for c in range(h * group, (h + 1) * group):
                x = (s["q"][a:b, c].double() @ keys.T) * s["scale"]
                x[hidden] = -math.inf
                lse[a:b, c] = torch.logsumexp(x, 1)
                out[a:b, c] = torch.softmax(x, 1) @ values
    return {"out": out, "lse": lse}


def _exact_sample(s):
    z_all = s["logits"].double().cpu().numpy()
    logprob = np.empty(s["rows"])
    for r in range(s["rows"]):
        z, t = z_all[r], float(s["temperature"][r])
        if t <= 0:
            logprob[r] = 0.0
            continue
        k, p = int(s["top_k"][r]), float(s["top_p"][r])
        order = np.argsort(-z, kind="stable")[:k or None]
        w = np.exp((z[order] - z[order[0]]) / t)
        if p < 1:
            before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            order = order[before < p * w.sum()]
        w = np.exp((z[order] - z[order[0]]) / t)
        order = np.sort(order[w >= float(s["min_p"][r])])
        w = np.exp((z[order] - z.max()) / t)
        run_sum = np.cumsum(w)
        token = order[min(int(np.searchsorted(run_sum, float(s["u"][r]) * run_sum[-1], side="right")), len(order) - 1)]
        logprob[r] = (z[token] - z.max()) / t - math.log(run_sum[-1])
    return {"token": None, "logprob": logprob}
