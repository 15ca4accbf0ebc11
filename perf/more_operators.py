"""Cases for the operators around a step's products: E4M3 products with block
scales, rotary positions on the way into the cache, verification of drafts.

Each case is one call of a serving step (a product: the activations' rounding
to E4M3 and the product) at sizes of the repository's model (5120 wide, 17408
in the feed-forward layer, 40 query heads and 8 key/value heads of 128, a
vocabulary of 151,936) or of generic ones.  `own` picks the framework's calls;
otherwise the same operators run in elementary torch operations.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

VOCAB = 151_936
BLOCK = 128          # elements that share a scale
_E4M3_MAX = 448.0
_LEAST_SCALE = 2.0 ** -126
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_MASS_BITS = 44      # fraction bits of a token's weight


def _afx():
    from weight_streaming_canonical_gb300 import afx
    return afx


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one request's next token through the feed-forward layer's first matrix: bound by reading the weights
        {"name": "product token", "op": "product", "tokens": 1, "rows": 17_408, "cols": 5120, "type": "bf16", "out": "fp32"},
        # a decode step of 64 requests through its second one: long sums, few rows
        {"name": "product batch", "op": "product", "tokens": 64, "rows": 5120, "cols": 17_408, "type": "bf16", "out": "bf16"},
        # a chunk of a prompt through the queries', keys' and values' matrices laid together, an odd number of tokens
        {"name": "product chunk", "op": "product", "tokens": 501, "rows": 7168, "cols": 5120, "type": "fp16", "out": "fp16"},
        # a whole prompt: bound by the products
        {"name": "product prompt", "op": "product", "tokens": 4096, "rows": 17_408, "cols": 5120, "type": "bf16", "out": "bf16"},
        # the activations of a decode step: latency counts
        {"name": "quantize step", "op": "quantize", "tokens": 64, "cols": 5120, "type": "bf16"},
        # those of a prompt behind the feed-forward layer's float32 sums
        {"name": "quantize prompt", "op": "quantize", "tokens": 8191, "cols": 17_408, "type": "fp32"},
        # a decode step's queries, keys and values out of a product's float32 rows: latency counts
        {"name": "rotate step", "op": "rotate", "tokens": 64, "q_heads": 40, "kv_heads": 8, "dim": 128, "rotary": 128, "axes": 1,
         "order": "blocks", "pairs": "halves", "page": 16, "far": 131_000, "type": "fp32", "cache": "bf16"},
        # a batch of prompts, an odd number of tokens
        {"name": "rotate prompt", "op": "rotate", "tokens": 32_701, "q_heads": 40, "kv_heads": 8, "dim": 128, "rotary": 128, "axes": 1,
         "order": "blocks", "pairs": "halves", "page": 64, "far": 131_000, "type": "bf16", "cache": "bf16"},
        # frames of a video with positions of time, height and width
        {"name": "rotate video", "op": "rotate", "tokens": 15_953, "q_heads": 28, "kv_heads": 4, "dim": 128, "rotary": 128, "axes": 3,
         "order": "interleaved", "pairs": "halves", "page": 32, "far": 30_000, "type": "fp16", "cache": "fp16"},
        # one request's drafts: latency counts
        {"name": "verify 1", "op": "verify", "requests": 1, "drafts": 4, "vocab": VOCAB, "model": True, "cuts": True, "type": "fp32"},
        # an ordinary batch with parameters of each request's own
        {"name": "verify 64", "op": "verify", "requests": 64, "drafts": 5, "vocab": VOCAB, "model": True, "cuts": True, "type": "bf16"},
        # drafts looked up in the prompt, so without logits of their own, drawn by temperature alone
        {"name": "verify lookup", "op": "verify", "requests": 200, "drafts": 3, "vocab": VOCAB, "model": False, "cuts": False, "type": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "rotate", "verify", "verify"])
    if op == "product":
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "rows": _log_int(rng, 100, 17_408), "cols": 16 * _log_int(rng, 6, 320),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "out": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "quantize":
        return {"op": op, "tokens": _log_int(rng, 1, 8191), "cols": _log_int(rng, 100, 17_408), "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "rotate":
        dim = rng.choice([64, 128])
        axes = rng.choice([1, 1, 2, 3])
        q_heads, kv_heads = rng.choice([(40, 8), (32, 8), (28, 4), (16, 16), (7, 1)])
        return {"op": op, "tokens": _log_int(rng, 1, 32_701), "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "rotary": rng.choice([dim, dim, dim // 2]), "axes": axes, "order": rng.choice(["blocks", "interleaved"]),
                "pairs": rng.choice(["halves", "neighbours"]), "page": rng.choice([16, 32, 64, 128]), "far": _log_int(rng, 1000, 1_000_000),
                "type": rng.choice(["same", "fp32"]), "cache": rng.choice(["bf16", "fp16"])}
    model = rng.choice([True, True, False])
    drafts = rng.choice([1, 2, 3, 4, 5, 8])
    return {"op": op, "requests": _log_int(rng, 1, 384 // drafts), "drafts": drafts, "vocab": rng.choice([VOCAB, _log_int(rng, 500, VOCAB)]),
            "model": model, "cuts": rng.choice([True, True, False]), "type": rng.choice(["bf16", "fp16", "fp32"])}


def _source(case):
    return case["cache"] if case["type"] == "same" else case["type"]


def _draft_counts(case, seed):
    """Drafts a request: the same for every seed (so the outputs' shapes are), in an order of the seed's own."""
    rng = random.Random(29)
    n = [case["drafts"] if case["requests"] == 1 else rng.randint(0, case["drafts"]) for _ in range(case["requests"])]
    random.Random(seed).shuffle(n)
    return n


def _blocks(n):
    return -(-n // BLOCK)


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    _PREPARE[case["op"]](s, case, seed, g)
    return s


def _activations(tokens, cols, kind, g):
    """What a layer hands to its next product: a few columns far larger than the rest, rows of padding."""
    x = torch.randn((tokens, cols), generator=g, device="cuda")
    x *= 1 + 30 * (torch.rand(cols, generator=g, device="cuda") < 0.002)
    if tokens > 8:
        x[tokens // 3] = 0
    return x.to(_TYPES[kind])


def _prepare_quantize(s, case, seed, g):
    s["x"] = _activations(case["tokens"], case["cols"], case["type"], g)
    # rows of E4M3 start on 16 bytes
    s["width"] = -(-case["cols"] // 16) * 16
    s["x8"] = torch.zeros((case["tokens"], s["width"]), dtype=torch.uint8, device="cuda")
    s["x_scales"] = torch.zeros((_blocks(case["cols"]), case["tokens"]), dtype=torch.float32, device="cuda")


def _prepare_product(s, case, seed, g):
    _prepare_quantize(s, case, seed, g)
    rows, cols = case["rows"], case["cols"]
    # a checkpoint's weights: E4M3 with a scale for each block of 128 rows and 128 columns
    w = torch.randn((rows, cols), generator=g, device="cuda") * 0.02
    padded = torch.nn.functional.pad(w, (0, -cols % BLOCK, 0, -rows % BLOCK))
    tiles = padded.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
    s["w_scales"] = (tiles.abs().amax((1, 3)) / _E4M3_MAX).contiguous()
    tiles = (tiles / s["w_scales"][:, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    s["w8"] = tiles.flatten(2, 3).flatten(0, 1)[:rows, :cols].to(torch.float8_e4m3fn).contiguous().view(torch.uint8)
    s["y"] = torch.zeros((case["tokens"], rows), dtype=_TYPES[case["out"]], device="cuda")


def _sections(case):
    """Pairs an axis: time, height and width get about a quarter, three and three eighths."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [pairs]
    rest = 3 * pairs // 8 if axes == 3 else pairs // 2
    return [pairs - rest * (axes - 1)] + [rest] * (axes - 1)


def _axis_of_pair(case):
    """The axis whose position turns each pair: blocks of pairs, or one after another while an axis has pairs left."""
    sections = _sections(case)
    if case["order"] == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out, a = list(sections), [], 0
    while len(out) < sum(sections):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def _prepare_rotate(s, case, seed, g):
    n, dim, page = case["tokens"], case["dim"], case["page"]
    # the rows of one fused product: queries, keys and values are strided views of it
    heads = case["q_heads"] + 2 * case["kv_heads"]
    rows = torch.randn((n, heads * dim), generator=g, device="cuda").to(_TYPES[_source(case)]).unflatten(1, (heads, dim))
    s["q"], s["k"], s["v"] = rows.split([case["q_heads"], case["kv_heads"], case["kv_heads"]], 1)
    pages = -(-n // page) + 3
    shape = (pages, page, case["kv_heads"], dim)
    s["k_pool"], s["v_pool"] = (torch.randn(shape, generator=g, device="cuda").to(_TYPES[case["cache"]]) for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(n, device="cuda")
    s["slots"] = (order[i // page] * page + i % page).to(torch.int32)
    start = int(torch.randint(0, max(1, case["far"]), (1,), generator=g, device="cuda"))
    time = start + i
    if case["axes"] == 1:
        s["positions"] = time[None].to(torch.int32)
    else:  # frames of 24 rows of 40 patches
        parts = [start + i // 960, start + i // 40 % 24, start + i % 40]
        s["positions"] = torch.stack(parts[:case["axes"]]).to(torch.int32)
    s["base"] = 1_000_000.0
    s["frequencies"] = [s["base"] ** (-2.0 * j / case["rotary"]) for j in range(case["rotary"] // 2)]
    s["axis_of_pair"] = torch.tensor(_axis_of_pair(case), device="cuda")
    s["freq"] = torch.tensor(s["frequencies"], dtype=torch.float64, device="cuda")
    s["q_out"] = torch.zeros((n, case["q_heads"], dim), dtype=_TYPES[case["cache"]], device="cuda")
    if own:
        afx = _afx()
        s["description"] = afx.kv_cache(s["k_pool"], s["v_pool"])
        s["rotary_plan"] = afx.rotary(dim, rotary_dim=case["rotary"], base=s["base"], sections=_sections(case), order=case["order"],
                                      pairs=case["pairs"])


def _prepare_verify(s, case, seed, g):
    counts, vocab = _draft_counts(case, seed), case["vocab"]
    n = sum(counts) + case["requests"]  # each request's last token and its drafts
    kind = _TYPES[case["type"]]
    z = torch.randn((n, vocab), generator=g, device="cuda") * 2.5
    spikes = torch.randint(0, vocab, (n, 24), generator=g, device="cuda")
    z.scatter_add_(1, spikes, torch.rand((n, 24), generator=g, device="cuda") * 12)  # the few tokens that fit
    z[:, vocab - vocab // 64:] = -math.inf  # the table's padding rows
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c + 1)
    rng = random.Random(seed * 104_729 + 7)
    rows = case["requests"]
    if case["cuts"]:
        pick = [(rng.choice([0.0, 0.6, 0.7, 1.0, 1.0, 1.3]), rng.choice([0, 0, 20, 50, 1000]), rng.choice([1.0, 0.8, 0.9, 0.95]),
                 rng.choice([0.0, 0.0, 0.02, 0.1])) if r else (0.7, 50, 0.9, 0.0) for r in range(rows)]
    else:
        pick = [(rng.choice([0.7, 0.8, 1.0]), 0, 1.0, 0.0) for _ in range(rows)]
    for k, name in enumerate(("temperature", "top_k", "top_p", "min_p")):
        s[name] = torch.tensor([p[k] for p in pick], dtype=torch.int32 if name == "top_k" else torch.float32, device="cuda")
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    request = torch.repeat_interleave(torch.arange(rows, device="cuda"), torch.tensor(counts, device="cuda") + 1)
    # the draft model's logits: near the target's
    zd = z + 0.7 * torch.randn((n, vocab), generator=g, device="cuda")
    s["logits"] = z.to(kind)
    # drafts: the draft model's likeliest token, tempered by noise
    t = s["temperature"][request][:, None]
    top, at = zd.to(kind).float().topk(min(16, vocab - vocab // 64), dim=1)
    noise = -torch.log(-torch.log(torch.rand(top.shape, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    chosen = at.gather(1, (top + t * noise).argmax(1, keepdim=True))[:, 0]
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    first = torch.zeros(n, dtype=torch.bool, device="cuda")
    first[s["starts"][:-1].long()] = True
    s["tokens"] = torch.where(first, tokens, chosen.roll(1)).to(torch.int32)
    if case["model"]:
        s["draft_logits"] = zd.to(kind)
    s["u"] = torch.rand(n, generator=g, device="cuda")
    s["draw_u"] = torch.rand(rows, generator=g, device="cuda")
    s["out_tokens"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["counts"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["logprobs"] = torch.zeros(n, dtype=torch.float32, device="cuda")
    if own:
        s["workspace"] = torch.empty(_afx().afx_verify_workspace(n, rows), dtype=torch.uint8, device="cuda")


_PREPARE = {"product": _prepare_product, "quantize": _prepare_quantize, "rotate": _prepare_rotate, "verify": _prepare_verify}


# ---- one pass -----------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_quantize(s):
    _afx().afx_fp8_quantize(s["x"], s["x8"], s["x_scales"])
    return {"values": s["x8"][:, :s["cols"]].view(torch.float8_e4m3fn), "scales": s["x_scales"]}


def _own_product(s):
    afx = _afx()
    afx.afx_fp8_quantize(s["x"], s["x8"], s["x_scales"])
    afx.afx_fp8_product(s["w8"], s["w_scales"], s["x8"], s["x_scales"], s["y"], status_dev=s["status"])
    return {"y": s["y"]}


def _own_rotate(s):
    _afx().afx_rotate_write(s["rotary_plan"], s["positions"], s["q"], s["k"], s["v"], s["q_out"], s["description"], s["slots"],
                            status_dev=s["status"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_verify(s):
    cuts = {k: s[k] for k in ("temperature", "top_k", "top_p", "min_p")} if s["cuts"] else {"temperature": s["temperature"]}
    afx = _afx()
    afx.afx_verify(s["logits"], s["tokens"], s["starts"], s["u"], s["draw_u"], s["out_tokens"], s["counts"], s["workspace"],
                   params=cuts, draft_logits=s.get("draft_logits"), draft_params=cuts if s["model"] else None,
                   logprobs=s["logprobs"], status_dev=s["status"])
    return {"tokens": s["out_tokens"], "counts": s["counts"], "logprobs": s["logprobs"]}


def _quantize(x):
    """(values, scales): x cut into blocks of 128 columns, each divided by its scale and rounded to E4M3, as float32."""
    cols = x.shape[1]
    blocks = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).unflatten(1, (-1, BLOCK))
    scale = (blocks.abs().amax(2, keepdim=True).double() / _E4M3_MAX).float().clamp(min=_LEAST_SCALE)
    values = (blocks / scale).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn).float()
    return values.flatten(1)[:, :cols], scale[:, :, 0]


def _plain_quantize(s):
    values, scales = _quantize(s["x"])
    return {"values": values.to(torch.float8_e4m3fn), "scales": scales.T.contiguous()}


def _plain_product(s):
    values, scales = _quantize(s["x"])
    x = values * scales.repeat_interleave(BLOCK, 1)[:, :s["cols"]]
    w = s["w8"].view(torch.float8_e4m3fn).float()
    w = w * s["w_scales"].repeat_interleave(BLOCK, 0)[:s["rows"]].repeat_interleave(BLOCK, 1)[:, :s["cols"]]
    return {"y": (x @ w.T).to(s["y"].dtype)}


def _turn(x, cos, sin, pairs):
    """x [tokens][heads][dim] with its pairs turned: the two halves' elements, or neighbours."""
    half = cos.shape[1]
    a, b = (x[..., :half], x[..., half:2 * half]) if pairs == "halves" else (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    c, d = cos[:, None, :], sin[:, None, :]
    turned = [a * c - b * d, a * d + b * c]
    turned = torch.cat(turned, -1) if pairs == "halves" else torch.stack(turned, -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rotate(s):
    angle = s["positions"].double()[s["axis_of_pair"]].T * s["freq"]  # [tokens][pairs]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    slots, kind = s["slots"].long(), s["q_out"].dtype
    s["k_pool"].flatten(0, 1)[slots] = _turn(s["k"].float(), cos, sin, s["pairs"]).to(kind)
    s["v_pool"].flatten(0, 1)[slots] = s["v"].float().to(kind)
    return {"q": _turn(s["q"].float(), cos, sin, s["pairs"]).to(kind), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _shares(logits, s, request):
    """Each row's tokens as shares of what temperature, top-k, top-p and min-p leave (float32), their logarithms, and the weights."""
    z = logits.float()
    z = torch.where(torch.isnan(z), -math.inf, z)
    m = z.amax(1, keepdim=True)
    temperature = s["temperature"][request][:, None]
    greedy = ~(temperature > 0)
    y = (z - m) * (1.0 / torch.where(greedy, 1.0, temperature))
    y = torch.where(z == m, 0.0, torch.where(z == -math.inf, -math.inf, y))
    w = torch.exp(y)
    if s["cuts"]:
        mass = (w * 2.0 ** _MASS_BITS).to(torch.int64)
        _, order = torch.sort(z, dim=1, descending=True, stable=True)
        rank = torch.arange(z.shape[1], device=z.device)[None, :]
        top_k = s["top_k"][request][:, None]
        k = torch.where(greedy, 1, torch.where(top_k > 0, top_k, z.shape[1]))
        by_rank = torch.where(rank < k, mass.gather(1, order), 0)
        run_sum = torch.cumsum(by_rank, 1)
        top = run_sum[:, -1:]
        p = s["top_p"][request][:, None]
        limit = torch.where(p < 1, torch.ceil(p.double() * top.double()).to(torch.int64).clamp(min=1), top)
        keep = (rank < k) & (run_sum - by_rank < limit)
        keep = torch.zeros_like(keep).scatter_(1, order, keep) & (w >= s["min_p"][request][:, None].clamp(max=1))
        w = torch.where(keep, w, 0.0)
        y = torch.where(keep, y, -math.inf)
    total = w.double().sum(1, keepdim=True)
    return (w / total).float(), y - torch.log(total).float()


def _plain_verify(s):
    starts, tokens = s["starts"].long(), s["tokens"].long()
    n, requests = tokens.numel(), s["requests"]
    at = torch.arange(n, device=tokens.device)
    request = torch.searchsorted(starts[1:], at, right=True)
    place = at - starts[request]
    has_draft = at + 1 < starts[request + 1]
    draft = torch.where(has_draft, tokens.roll(-1), 0)
    p, log_p = _shares(s["logits"], s, request)
    p_draft = p.gather(1, draft[:, None])[:, 0]
    if s["model"]:
        q, _ = _shares(s["draft_logits"], s, request)
        q_draft = q.gather(1, draft[:, None])[:, 0]
    else:
        q_draft = torch.ones_like(p_draft)
    taken = has_draft & (s["u"].double() * q_draft.double() < p_draft.double())
    # a request's first row whose draft is not taken (its last row has none)
    length = s["drafts"] + 1
    accepted = torch.full((requests,), length, device=tokens.device).scatter_reduce_(
        0, request, torch.where(taken, length, place), "amin")
    row = starts[:-1] + accepted
    rest, refused = p[row], has_draft[row]
    if s["model"]:
        rest = torch.where(refused[:, None], (rest - q[row]).clamp(min=0), rest)
    else:
        rest = rest.scatter(1, draft[row][:, None], torch.where(refused, 0.0, rest.gather(1, draft[row][:, None])[:, 0])[:, None])
    # nothing is left where the draft was none that the draft's logits allow, as one of two equal 16-bit maxima
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[row])
    mass = (rest * 2.0 ** _MASS_BITS).to(torch.int64)
    run_sum = torch.cumsum(mass, 1)
    total = run_sum[:, -1:]
    aim = torch.minimum((s["draw_u"][:, None].double() * total.double()).to(torch.int64), total - 1)
    token = (run_sum <= aim).sum(1)
    drawn = place == accepted[request]
    kept = place < accepted[request]
    out = torch.where(kept, draft, torch.where(drawn, token[request], -1))
    logprobs = torch.where(kept | drawn, log_p.gather(1, out.clamp(min=0)[:, None])[:, 0], 0.0)
    return {"tokens": out.to(torch.int32), "counts": (accepted + 1).to(torch.int32), "logprobs": logprobs}


_OWN = {"product": _own_product, "quantize": _own_quantize, "rotate": _own_rotate, "verify": _own_verify}
_PLAIN = {"product": _plain_product, "quantize": _plain_quantize, "rotate": _plain_rotate, "verify": _plain_verify}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "quantize":
        return {"bytes": case["tokens"] * (case["cols"] * (size[case["type"]] + 1) + 4 * _blocks(case["cols"])), "flops": 0}
    if case["op"] == "product":
        t, r, c = case["tokens"], case["rows"], case["cols"]
        return {"bytes": r * c + 4 * _blocks(r) * _blocks(c) + t * c * size[case["type"]] + t * r * size[case["out"]], "flops": 2 * t * r * c}
    if case["op"] == "rotate":
        heads = case["q_heads"] + 2 * case["kv_heads"]
        return {"bytes": case["tokens"] * (heads * case["dim"] * (size[_source(case)] + 2) + 4 + 4 * case["axes"]), "flops": 0}
    counts = _draft_counts(case, 1)
    read = sum(counts) + case["requests"] + (sum(counts) if case["model"] else 0)
    return {"bytes": read * case["vocab"] * size[case["type"]] + 16 * (sum(counts) + case["requests"]), "flops": 0}


# ---- the definitions, in 64 bits ----------------------------------------------------

def exact(case, seed):
    if case["op"] == "verify" and sum(_draft_counts(case, seed)) * case["vocab"] > 30_000_000:
        return None
    return _EXACT[case["op"]](prepare(case, seed))


def _e4m3(x):
    """The nearest E4M3 value of |x| <= 448 (ties to the even one): steps of 2^-3 of a power of two, from 2^-6 on; 2^-9 below."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_quantized(s):
    x = s["x"].double()
    values, scales = torch.empty_like(x), []
    for c in range(0, s["cols"], BLOCK):
        part = x[:, c:c + BLOCK]
        scale = (part.abs().amax(1) / _E4M3_MAX).float().clamp(min=_LEAST_SCALE)  # a float32 is what is kept of it
        scales.append(scale)
        values[:, c:c + BLOCK] = _e4m3((part / scale.double()[:, None]).float().double().clamp(-_E4M3_MAX, _E4M3_MAX))
    return values, torch.stack(scales)


def _exact_quantize(s):
    values, scales = _exact_quantized(s)
    return {"values": values, "scales": scales.double()}


def _exact_product(s):
    values, scales = _exact_quantized(s)
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    w_scales = s["w_scales"].double()
    for b, c in enumerate(range(0, s["cols"], BLOCK)):
        w = s["w8"][:, c:c + BLOCK].view(torch.uint8).to(torch.int64)
        exponent, fraction = w >> 3 & 15, (w & 7).double()
        w = torch.where(exponent > 0, (1 + fraction / 8) * 2.0 ** (exponent.double() - 7), fraction * 2.0 ** -9) * (1 - 2 * (w >> 7).double())
        part = (values[:, c:c + BLOCK] * scales[b].double()[:, None]) @ w.T
        for r in range(0, s["rows"], BLOCK):
            y[:, r:r + BLOCK] += part[:, r:r + BLOCK] * w_scales[r // BLOCK, b]
    return {"y": y}


def _exact_rotate(s):
    """Pair by pair, as complex numbers."""
    half = s["rotary"] // 2
    axis = s["axis_of_pair"].tolist()

    def turned(x):
        out = x.double().clone()
        for j in range(half):
            a, b = (j, j + half) if s["pairs"] == "halves" else (2 * j, 2 * j + 1)
            angle = s["positions"][axis[j]].double() * s["frequencies"][j]
            z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.polar(torch.ones_like(angle), angle)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
        return out

    pools = {"k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    pools["k_pool"].flatten(0, 1)[s["slots"].long()] = turned(s["k"])
    pools["v_pool"].flatten(0, 1)[s["slots"].long()] = s["v"].double()
    return {"q": turned(s["q"]), **pools}


def _exact_shares(z, s, r):
    """One row's tokens as shares of what request r's parameters leave."""
    t = float(s["temperature"][r])
    z = np.where(np.isnan(z), -np.inf, z)
    p = np.zeros(len(z))
    if t <= 0:
        p[int(np.argmax(z))] = 1.0
        return p
    order = np.argsort(-z, kind="stable")
    if s["cuts"]:
        order = order[:int(s["top_k"][r]) or None]
        w = np.exp((z[order] - z[order[0]]) / t)
        if float(s["top_p"][r]) < 1:
            before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            order = order[before < float(s["top_p"][r]) * w.sum()]
        w = np.exp((z[order] - z[order[0]]) / t)
        order = order[w >= float(s["min_p"][r])]
    w = np.exp((z[order] - z[order[0]]) / t)
    p[order] = w / w.sum()
    return p


def _exact_verify(s):
    starts, tokens, u, draw_u = (s[k].tolist() for k in ("starts", "tokens", "u", "draw_u"))
    logprobs = np.zeros(len(tokens))
    for r in range(s["requests"]):
        for row in range(starts[r], starts[r + 1]):
            p = _exact_shares(s["logits"][row].double().cpu().numpy(), s, r)
            rest = p
            if row + 1 < starts[r + 1]:
                d = tokens[row + 1]
                if s["model"]:
                    q = _exact_shares(s["draft_logits"][row].double().cpu().numpy(), s, r)
                else:
                    q = np.zeros(len(p))
                    q[d] = 1.0
                if u[row] * q[d] < p[d]:
                    logprobs[row] = math.log(p[d])
                    continue
                rest = np.maximum(p - q, 0.0)
                rest = rest if rest.any() else p
            run_sum = np.cumsum(rest)
            last = int(np.nonzero(rest)[0][-1])
            token = min(int(np.searchsorted(run_sum, draw_u[r] * run_sum[-1], side="right")), last)
            logprobs[row] = math.log(p[token])
            break
    return {"tokens": None, "counts": None, "logprobs": logprobs}


_EXACT = {"product": _exact_product, "quantize": _exact_quantize, "rotate": _exact_rotate, "verify": _exact_verify}
