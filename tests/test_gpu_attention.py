"""Shared-prefix attention (afx_attention) against float64 softmax, request by
request.

Tolerances, from the arithmetic, per output element: with u the type's unit
roundoff (BF16 has 8 significant bits, u = 2^-8; FP16 has 11, u = 2^-11),
weights are rounded once before the product with V and the output once after
it, so |err| <= 2 u * sum p|v|; float32 scores add a
relative e^(2 * 128 * 2^-24 * reach) - 1 to each weight (reach = scale * sum
|q k|, at most 40 here: 6e-4), and FP16 weights below 2^-14 an absolute 2^-25
each.  lse: the scores' error and 2^-18 for the sums and the logarithm.
"""
import math
import random

import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Inputs of one call; everything a call must not use is NaN or infinite."""

    def __init__(self, new, lens, prefix, q_heads=10, kv_heads=2, dim=128, page=16, dtype="bfloat16", layout="tokens, heads",
                 seed=0, sharp=1.0, pad_tokens=0, pool_pages=None, q_shift=0):
        import torch
        self.dtype, self.page, self.prefix = getattr(torch, dtype), page, prefix
        self.u = 2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -11
        self.new, self.lens_list = new, lens
        rng = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        n_prefix = ref.pages(prefix, page)
        held = [ref.pages(n, page) for n in lens]
        total = pool_pages or (n_prefix + sum(held) + 3)
        ids = list(range(total)) if pool_pages is None else list(range(total - n_prefix - sum(held), total))
        rng.shuffle(ids)
        order = {"tokens, heads": (0, 1, 2, 3), "heads, tokens": (0, 2, 1, 3), "head pools": (2, 0, 1, 3)}[layout]
        shape = (total, page, kv_heads, dim)
        self.pools = []
        for _ in range(2):
            if pool_pages is None:
                # infinities and NaN wherever no token lies
                m = torch.full([shape[i] for i in order], math.nan, dtype=self.dtype, device="cuda")
                m.view(-1)[::3] = math.inf
            else:
                m = torch.zeros([shape[i] for i in order], dtype=self.dtype, device="cuda")
            self.pools.append(m.permute([order.index(i) for i in range(4)]))
        cols = max([1] + held) + 2
        at = n_prefix
        self.prefix_list, self.table_list = ids[:n_prefix], []
        for h in held:
            self.table_list.append(ids[at:at + h] + [-3] * (cols - h))
            at += h
        for pool in self.pools:
            for row, n in [(self.prefix_list, prefix)] + list(zip(self.table_list, lens)):
                for c in range(ref.pages(n, page)):
                    k = min(page, n - c * page)
                    pool[row[c], :k] = torch.randn((k, kv_heads, dim), generator=g, device="cuda").to(self.dtype)
        self.starts_list = [0]
        for n in new:
            self.starts_list.append(self.starts_list[-1] + n)
        self.tokens = max(1, self.starts_list[-1] + pad_tokens)
        rows = torch.randn((self.tokens, q_heads * dim + q_shift + 5 * (q_shift > 0)), generator=g, device="cuda") * sharp
        self.q = rows.to(self.dtype)[:, q_shift:q_shift + q_heads * dim].unflatten(1, (q_heads, dim))
        self.scale = 1.0 / math.sqrt(dim)
        self.prefix_table, self.table = _ints(self.prefix_list), _ints(self.table_list)
        self.starts, self.lens = _ints(self.starts_list), _ints(lens)
        self.out = torch.full((self.tokens, q_heads, dim), 7.0, dtype=self.dtype, device="cuda")
        self.lse = torch.full((self.tokens, q_heads), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, afx, **change):
        d = dict(starts=self.starts, lens=self.lens, table=self.table, scale=self.scale, prefix_table=self.prefix_table,
                 prefix_len=self.prefix)
        d.update(change)
        return afx.attention_args(afx.kv_cache(*self.pools), self.q.shape[1], self.tokens, **d)

    def run(self, afx, args=None, stream=None):
        import torch
        args = args or self.args(afx)
        ws = torch.full((afx.afx_attention_workspace(args),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        afx.afx_attention_plan(args, ws, stream=stream, status_dev=self.status)
        afx.afx_attention(args, self.q, self.out, ws, lse=self.lse, stream=stream, status_dev=self.status)
        torch.cuda.synchronize()
        return self.out, self.lse

    def check(self, afx):
        import torch
        self.run(afx)
        assert self.status.item() == 0
        out, lse, weight, reach = ref.attention(self.q, *self.pools, self.prefix_list, self.prefix, self.starts_list,
                                                self.lens_list, self.table_list, self.scale)
        n = self.starts_list[-1]
        score = torch.expm1(2 * 128 * 2.0 ** -24 * reach)[..., None]
        bound = weight * (2 * self.u + 2 * score) + (2.0 ** -25 * 4 * (self.prefix + max(self.lens_list)) if self.dtype == torch.float16 else 0)
        err = (self.out.double() - out).abs()[:n]
        assert torch.isfinite(self.out[:n]).all()
        assert (err <= bound[:n]).all(), f"largest error {(err / (bound[:n] + 1e-30)).max().item():.3g} of its bound"
        empty = torch.isinf(lse[:n])
        assert torch.equal(torch.isinf(self.lse[:n]), empty)
        assert (self.out[:n][empty] == 0).all()
        lse_err = (self.lse.double() - lse).abs()[:n][~empty]
        assert (lse_err <= (2 * 128 * 2.0 ** -24 * reach[:n] + 2.0 ** -18)[~empty]).all(), lse_err.max().item()
        assert (self.out[n:] == 7).all() and (self.lse[n:] == 7).all()  # rows past the last token


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 65, 1000])
def test_prefix_lengths(afx, dtype, prefix):
    Case([1, 1, 1], [1, 40, 129], prefix, dtype=dtype, seed=prefix).check(afx)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (10, 2), (7, 1), (16, 1), (17, 1), (40, 2), (33, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_head_layouts(afx, q_heads, kv_heads, dim):
    Case([1, 3, 1], [20, 70, 5], 200, q_heads, kv_heads, dim, seed=q_heads).check(afx)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["tokens, heads", "heads, tokens", "head pools"])
def test_pages_and_cache_layouts(afx, page, layout):
    Case([1, 2, 1], [page - 1, page, page + 1], 2 * page + 5, page=page, layout=layout, seed=page).check(afx)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_new_tokens_see_their_own_past_only(afx, dtype, dim):
    """Whole prompts: the causal edge runs through every row tile."""
    Case([64, 1, 37, 100, 2], [64, 1, 90, 333, 17], 77, dim=dim, dtype=dtype, seed=4).check(afx)


def test_prompts_without_a_prefix(afx):
    Case([130, 5, 300], [130, 5, 300], 0, seed=6).check(afx)


def test_rows_that_see_nothing(afx):
    """No prefix: a request with new tokens that are not in the cache, one whose first tokens are not, one with none."""
    Case([2, 5, 0, 1], [0, 2, 9, 3], 0, seed=7).check(afx)


def test_rows_that_see_the_prefix_only(afx):
    Case([2, 5, 0, 1], [0, 2, 0, 0], 33, seed=8).check(afx)


def test_nothing_to_do(afx):
    Case([0, 0], [5, 0], 20, pad_tokens=3, seed=9).check(afx)


def test_padding_tokens_are_left_alone(afx):
    Case([1, 2, 1], [9, 30, 2], 50, pad_tokens=6, seed=10).check(afx)


@pytest.mark.parametrize("shift", [1, 2, 3, 8])
def test_strided_queries(afx, shift):
    Case([1, 2, 1], [9, 30, 2], 50, q_shift=shift, seed=11).check(afx)


def test_strided_outputs(afx):
    import torch
    c = Case([1, 2, 1], [9, 30, 2], 50, seed=12)
    whole = torch.full((c.tokens, 3, 10 * 128 + 1), 7.0, dtype=c.dtype, device="cuda")
    c.out = whole[:, 1, 1:].unflatten(1, (10, 128))
    c.check(afx)
    assert (whole[:, 0] == 7).all() and (whole[:, 2] == 7).all() and (whole[:, 1, 0] == 7).all()


def test_sharp_scores(afx):
    """Scores in the hundreds: maxima move far between blocks of keys."""
    Case([1, 1, 20], [100, 700, 300], 900, sharp=8.0, seed=13).check(afx)


@pytest.mark.parametrize("rising", [True, False])
def test_scores_in_order(afx, rising):
    """Every key scores above (below) all before it, by a little or a lot."""
    import torch
    c = Case([1, 1], [30, 200], 500, seed=14)
    line = torch.linspace(-3, 3, 700, device="cuda").flip(0) if not rising else torch.linspace(-3, 3, 700, device="cuda")
    for row, n, first in [(c.prefix_list, 500, 0), (c.table_list[0], 30, 500), (c.table_list[1], 200, 500)]:
        for j in range(n):
            c.pools[0][row[j // 16], j % 16] = line[first + j].to(c.dtype)
    c.q.copy_(torch.ones_like(c.q) * 2)
    c.check(afx)


def test_long_prefix_and_long_requests(afx):
    Case([1, 4, 1], [3000, 5000, 1], 20_000, q_heads=8, kv_heads=2, page=64, seed=15).check(afx)


def test_many_requests(afx):
    rng = random.Random(3)
    Case([1] * 150, [rng.randint(1, 90) for _ in range(150)], 130, q_heads=5, kv_heads=1, dim=64, seed=16).check(afx)


def test_more_requests_than_plan_threads(afx):
    rng = random.Random(4)
    n = 1500
    Case([rng.choice([0, 1, 1, 2]) for _ in range(n)], [rng.randint(0, 20) for _ in range(n)], 5, q_heads=2, kv_heads=1,
         dim=64, seed=17).check(afx)


def test_a_batch_large_enough_for_row_tiles(afx):
    """Hundreds of rows a key/value head on the prefix, odd counts."""
    Case([1] * 67, [10] * 67, 700, q_heads=10, kv_heads=2, seed=18).check(afx)
    Case([1] * 131, [3] * 131, 333, q_heads=8, kv_heads=2, dim=64, dtype="float16", seed=19).check(afx)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_cases(afx, seed):
    rng = random.Random(seed)
    n = rng.choice([1, 2, 5, 20])
    kv = rng.choice([1, 2, 4])
    new = [rng.choice([0, 1, 1, 2, rng.randint(1, 90)]) for _ in range(n)]
    lens = [max(0, k + rng.choice([0, 0, -1, rng.randint(0, 400)])) for k in new]
    Case(new, lens, rng.choice([0, rng.randint(1, 50), rng.randint(100, 1500)]), kv * rng.randint(1, 12), kv,
         rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice(["bfloat16", "float16"]),
         rng.choice(["tokens, heads", "heads, tokens", "head pools"]), seed, rng.choice([0.3, 1.0, 3.0])).check(afx)


def test_pools_past_4_gib(afx):
    Case([1, 9], [100, 300], 200, q_heads=8, kv_heads=8, page=128, pool_pages=20_000, seed=20).check(afx)


def test_the_same_call_gives_the_same_bits(afx):
    c = Case([1] * 40 + [50], [300] * 40 + [60], 3000, seed=21)
    args = c.args(afx)
    first = [x.clone() for x in c.run(afx, args)]
    for _ in range(5):
        out, lse = c.run(afx, args)
        assert (out == first[0]).all() and (lse == first[1]).all()


def test_one_plan_serves_many_layers(afx):
    import torch
    c = Case([1, 3], [50, 80], 100, seed=22)
    args = c.args(afx)
    want = c.run(afx, args)[0].clone()
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    afx.afx_attention_plan(args, ws)
    others = [p.clone() for p in c.pools]
    layer = afx.attention_args(afx.kv_cache(*others), 10, c.tokens, c.starts, c.lens, c.table, c.scale, c.prefix_table, c.prefix)
    for a in (args, layer, args):
        c.out.fill_(3)
        afx.afx_attention(a, c.q, c.out, ws)
        assert torch.equal(c.out, want)


def test_another_stream_and_a_graph(afx):
    import torch
    c = Case([1, 3], [50, 80], 100, seed=23)
    args = c.args(afx)
    want = c.run(afx, args)[0].clone()
    side = torch.cuda.Stream()
    c.out.fill_(3)
    assert torch.equal(c.run(afx, args, stream=side)[0], want)
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        afx.afx_attention_plan(args, ws)
        afx.afx_attention(args, c.q, c.out, ws, lse=c.lse)
    # the lengths change on the GPU between replays
    c.lens.copy_(_ints([30, 60]))
    c.lens_list = [30, 60]
    c.out.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    again = c.out.clone()
    c.out.fill_(4)
    c.check(afx)
    assert torch.equal(again, c.out)


def test_lengths_that_make_no_sense_do_nothing(afx):
    for change in ({"starts": _ints([0, 3, 2])}, {"starts": _ints([1, 2, 3])}, {"starts": _ints([0, 1, 99])},
                   {"starts": _ints([0, -1, 2])}, {"lens": _ints([50, -1])}, {"lens": _ints([50, 16 * 200])}):
        c = Case([1, 3], [50, 80], 100, seed=24)
        c.run(afx, c.args(afx, **change))
        assert c.status.item() == afx.AFX_DEV_BAD_LENGTH
        assert (c.out == 7).all() and (c.lse == 7).all()


def test_a_page_outside_the_pool_is_flagged(afx):
    c = Case([1, 3], [50, 80], 100, seed=25)
    c.table[1, 2] = 10 ** 6
    c.run(afx)
    assert c.status.item() == afx.AFX_DEV_BAD_PAGE
    c = Case([1] * 60, [50] * 60, 1000, seed=25)
    c.prefix_table[7] = -1
    c.run(afx)
    assert c.status.item() == afx.AFX_DEV_BAD_PAGE


def test_a_workspace_without_the_plan_is_flagged(afx):
    import torch
    c = Case([1, 3], [50, 80], 100, seed=26)
    args = c.args(afx)
    ws = torch.full((afx.afx_attention_workspace(args),), 255, dtype=torch.uint8, device="cuda")
    afx.afx_attention(args, c.q, c.out, ws, status_dev=c.status)
    assert c.status.item() == afx.AFX_DEV_BAD_PLAN and (c.out == 7).all()
    c.status.zero_()
    afx.afx_attention_plan(args, ws)
    afx.afx_attention(c.args(afx, prefix_len=99), c.q, c.out, ws, status_dev=c.status)
    assert c.status.item() == afx.AFX_DEV_BAD_PLAN and (c.out == 7).all()


def test_attention_refuses_bad_arguments(afx):
    import torch
    c = Case([1, 3], [50, 80], 100, seed=27)
    args = c.args(afx)
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    with pytest.raises(afx.AfxError) as err:
        afx.afx_attention_plan(args, ws[:-256])
    assert err.value.status == afx.AFX_E_NOSPACE
    for change in ({"scale": math.inf}, {"scale": math.nan}):
        with pytest.raises(afx.AfxError) as err:
            afx.afx_attention_workspace(c.args(afx, **change))
        assert err.value.status == afx.AFX_E_ARG
    with pytest.raises(afx.AfxError):
        afx.afx_attention_workspace(afx.attention_args(afx.kv_cache(*c.pools), 9, c.tokens, c.starts, c.lens, c.table, c.scale))
    for bad in (dict(q=c.q[:2], out=c.out), dict(q=c.q, out=c.out.float()), dict(q=c.q[:, :8], out=c.out), dict(q=c.q.cpu(), out=c.out)):
        with pytest.raises(ValueError):
            afx.afx_attention(args, bad["q"], bad["out"], ws)
    with pytest.raises(ValueError):
        c.args(afx, prefix_table=None)
    with pytest.raises(ValueError):
        c.args(afx, prefix_len=1000)
