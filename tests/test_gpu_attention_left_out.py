"""Attention where a table names a page outside the pool: its keys and values
are left out, in either kernel, and the status says so.

The reference takes the remaining keys of every row.  Page 0 holds NaN, so a
key read from another page in place of the missing one shows.  Inputs and
tolerances: test_gpu_attention.
"""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def _reference(c):
    """serving_ref.attention over the pages inside the pool."""
    n_pages, page, kvh, dim = c.pools[0].shape
    group = c.q.shape[1] // kvh
    out = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(c.q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weight, reach = torch.zeros_like(out), torch.zeros_like(lse)
    for r, length in enumerate(c.lens_list):
        a, b = c.starts_list[r], c.starts_list[r + 1]
        # page, place, and the row of the request from which on the key is seen
        where = [(c.prefix_list[j // page], j % page, 0) for j in range(c.prefix)]
        where += [(c.table_list[r][j // page], j % page, max(0, j - (length - (b - a)))) for j in range(length)]
        at = torch.tensor([w for w in where if 0 <= w[0] < n_pages], device="cuda").reshape(-1, 3)
        for t in range(a, b):
            seen = at[at[:, 2] <= t - a]
            if len(seen) == 0:
                continue
            k = c.pools[0][seen[:, 0], seen[:, 1]].double().repeat_interleave(group, 1)
            v = c.pools[1][seen[:, 0], seen[:, 1]].double().repeat_interleave(group, 1)
            x = torch.einsum("hd,khd->hk", c.q[t].double(), k) * c.scale
            lse[t] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            out[t] = torch.einsum("hk,khd->hd", p, v)
            weight[t] = torch.einsum("hk,khd->hd", p, v.abs())
            reach[t] = (torch.einsum("hd,khd->hk", c.q[t].double().abs(), k.abs()) * abs(c.scale)).amax(1)
    return out, lse, weight, reach


def _check(afx, c, prefix_columns=(), own_columns=(), bad=-1):
    """own_columns: (request, column)."""
    for pool in c.pools:
        pool[0] = math.nan
    for col in prefix_columns:
        c.prefix_list[col] = bad
        c.prefix_table[col] = bad
    for r, col in own_columns:
        c.table_list[r][col] = bad
        c.table[r, col] = bad
    c.run(afx)
    assert c.status.item() == afx.AFX_DEV_BAD_PAGE
    out, lse, weight, reach = _reference(c)
    score = torch.expm1(2 * 128 * 2.0 ** -24 * reach)[..., None]
    bound = weight * (2 * c.u + 2 * score) + (2.0 ** -25 * 4 * (c.prefix + max(c.lens_list)) if c.dtype == torch.float16 else 0)
    assert torch.isfinite(c.out).all()
    assert ((c.out.double() - out).abs() <= bound).all()
    empty = torch.isinf(lse)
    assert torch.equal(c.lse == -math.inf, empty)
    assert (c.out[empty] == 0).all()
    lse_err = (c.lse.double() - lse).abs()[~empty]
    assert (lse_err <= (2 * 128 * 2.0 ** -24 * reach + 2.0 ** -18)[~empty]).all()


def _case(new, lens, prefix, page=16, **kw):
    held = ref.pages(prefix, page) + sum(ref.pages(n, page) for n in lens)
    return Case(new, lens, prefix, page=page, pool_pages=held + 1, **kw)  # no token lies in page 0


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, 10 ** 6])
def test_any_id_outside_the_pool(afx, bad):
    _check(afx, _case([1, 3], [50, 80], 100, seed=1), [2], [(1, 2)], bad)


def test_the_first_id_past_the_pool(afx):
    c = _case([1, 3], [50, 80], 100, seed=2)
    _check(afx, c, [0], [(0, 3), (1, 0)], c.pools[0].shape[0])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_single_tokens(afx, dtype, dim, page):
    """Pages within a step of 16 keys' range, at its start and its end, in the prefix and in own pages."""
    c = _case([1, 1, 2], [3 * page + 5, page, 2 * page + 1], 6 * page + 3, page=page, dim=dim, dtype=dtype, seed=page)
    _check(afx, c, [0, 3, 6], [(0, 1), (0, 3), (2, 2)])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests", [20, 60])
def test_tiles_on_the_prefix(afx, requests, dim, page):
    """100 and 300 rows on the prefix: the two tiles take steps in turn, or both work on each."""
    n = max(700, 5 * page) + 7
    c = _case([1] * requests, [9] * requests, n, page=page, dim=dim, seed=page + requests)
    last = (n - 1) // page
    _check(afx, c, sorted({0, 3, last - 1, last}))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("new", [[20, 200], [25, 300, 1]])
def test_prompts(afx, new, page, dtype):
    """A request's own tiles run over the prefix and its own pages."""
    c = _case(new, [n + 90 for n in new], 3 * page + 20, page=page, dtype=dtype, seed=page)
    _check(afx, c, [1, 3], [(0, 0), (1, 1), (1, (new[1] + 89) // page)])


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new", [[1, 1], [70, 200]])
def test_no_page_left(afx, new, page):
    """All pages of the prefix and of one request are missing: its rows see nothing."""
    c = _case(new, [n + 30 for n in new], 200, page=page, seed=page)
    _check(afx, c, range(ref.pages(200, page)), [(0, i) for i in range(ref.pages(new[0] + 30, page))])


def test_many_steps_with_missing_pages(afx):
    """Every fifth page of a long prefix, over many steps of the tile kernel's ring, beside others' own tiles."""
    c = _case([1] * 40 + [150], [30] * 40 + [400], 5000, page=32, dim=64, q_heads=8, kv_heads=2, dtype="float16", seed=8)
    _check(afx, c, range(0, 157, 5), [(40, 1), (40, 12), (7, 0)])
