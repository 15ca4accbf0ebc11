"""Shared-prefix attention where its kernels change over: row counts around
those that choose a kernel, caches that no tensor map describes, queries and
outputs off their usual alignment in tiles, units that outnumber the warps.
Inputs and tolerances: test_gpu_attention.
"""
import random

import pytest

from test_gpu_attention import Case, _ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 1000])
@pytest.mark.parametrize("tokens", [15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 513])
def test_one_request_of_rows_around_the_borders(afx, tokens, prefix):
    Case([tokens], [tokens + 300], prefix, q_heads=2, kv_heads=2, seed=tokens).check(afx)


@pytest.mark.parametrize("requests", [2, 3, 25, 26, 51, 52])
def test_shared_rows_around_the_borders(afx, requests):
    """Five rows a request: 10 to 260 rows on the prefix."""
    Case([1] * requests, [20 + r for r in range(requests)], 2500, dtype="float16", seed=requests).check(afx)


def test_single_tokens_beside_prompts(afx):
    rng = random.Random(30)
    new = [rng.choice([1, 1, 4, 26, 150]) for _ in range(40)]
    Case(new, [n + rng.randint(0, 700) for n in new], 1500, seed=30).check(afx)


def test_more_units_than_warps(afx):
    rng = random.Random(31)
    Case([1] * 200, [rng.randint(200, 1000) for _ in range(200)], 300, q_heads=8, kv_heads=4, dim=64, seed=31).check(afx)


def test_more_requests_of_several_tokens_than_the_plan_lists(afx):
    Case([9 + r % 3 for r in range(700)], [12 + r % 5 for r in range(700)], 33, q_heads=2, kv_heads=1, dim=64, seed=32).check(afx)


def test_a_plan_of_both_kernels_serves_many_layers(afx):
    import torch
    c = Case([1] * 90 + [200], [400] * 90 + [250], 700, seed=33)
    args = c.args(afx)
    want = c.run(afx, args)[0].clone()
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    afx.afx_attention_plan(args, ws)
    for _ in range(4):
        c.out.fill_(3)
        afx.afx_attention(args, c.q, c.out, ws)
        assert torch.equal(c.out, want)


@pytest.mark.parametrize("shift", [1, 2, 8])
@pytest.mark.parametrize("new", [[60, 3], [1] * 70])
def test_strided_queries_in_tiles(afx, shift, new):
    Case(new, [n + 40 for n in new], 300, q_shift=shift, seed=34).check(afx)


@pytest.mark.parametrize("shift", [1, 8])
def test_strided_outputs_in_tiles(afx, shift):
    import torch
    c = Case([150, 1, 30], [150, 9, 400], 300, seed=35)
    whole = torch.full((c.tokens, 10 * 128 + 8), 7.0, dtype=c.dtype, device="cuda")
    c.out = whole[:, shift:shift + 1280].unflatten(1, (10, 128))
    c.check(afx)
    assert (whole[:, :shift] == 7).all() and (whole[:, shift + 1280:] == 7).all()


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("new", [[1, 1], [1] * 40, [130, 1]])
def test_scales_that_are_not_positive(afx, scale, new):
    c = Case(new, [n + 50 for n in new], 400, dtype="float16", seed=36)
    c.scale = scale
    c.check(afx)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_sharp_scores_in_tiles(afx, dtype):
    """Maxima that move by more than 2^14 between blocks of keys, in shared and in own tiles."""
    Case([1] * 30 + [300], [50] * 30 + [700], 900, dtype=dtype, sharp=8.0, seed=37).check(afx)


@pytest.mark.parametrize("new", [[1, 2], [1] * 40, [200, 1]])
def test_caches_that_no_tensor_map_describes(afx, new):
    """Tokens eight elements further apart than their heads fill: the stride is no multiple of a head's."""
    import torch
    c = Case(new, [n + 90 for n in new], 500, seed=38)
    views = []
    for pool in c.pools:
        pages, page, heads, dim = pool.shape
        padded = torch.full((pages, page, heads * dim + 8), float("nan"), dtype=pool.dtype, device="cuda")
        view = padded[..., :heads * dim].unflatten(2, (heads, dim))
        view.copy_(pool)
        views.append(view)
    c.pools = views
    c.check(afx)


def test_a_request_longer_than_its_table_row_does_nothing(afx):
    c = Case([60, 60], [70, 80], 100, seed=39)
    c.run(afx, c.args(afx, lens=_ints([70, 16 * c.table.shape[1] + 1])))
    assert c.status.item() == afx.AFX_DEV_BAD_LENGTH
    assert (c.out == 7).all() and (c.lse == 7).all()
