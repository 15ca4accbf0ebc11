"""Attention with NaN among what a row sees: queries, keys or values.  The
row's result is NaN, as the formula's is; every other row's is the one
without NaN.  Inputs and tolerances: test_gpu_attention.
"""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def _check(afx, c, spoiled):
    """spoiled: bool [token][q head], the rows whose outputs are NaN."""
    c.run(afx)
    assert c.status.item() == 0
    out, lse, weight, reach = ref.attention(c.q, *c.pools, c.prefix_list, c.prefix, c.starts_list, c.lens_list, c.table_list, c.scale)
    assert torch.isnan(lse[spoiled]).all() and torch.isfinite(out[~spoiled]).all()
    assert torch.isnan(c.out[spoiled]).all() and torch.isnan(c.lse[spoiled]).all()
    score = torch.expm1(2 * 128 * 2.0 ** -24 * reach)[..., None]
    bound = weight * (2 * c.u + 2 * score) + (2.0 ** -25 * 4 * (c.prefix + max(c.lens_list)) if c.dtype == torch.float16 else 0)
    assert ((c.out.double() - out).abs() <= bound)[~spoiled].all()
    assert ((c.lse.double() - lse).abs() <= 2 * 128 * 2.0 ** -24 * reach + 2.0 ** -18)[~spoiled].all()


SHAPES = {
    "single tokens": ([1, 1, 2], [5, 40, 90], 100),
    "without a prefix": ([1, 3], [1, 60], 0),
    "many pieces": ([1, 1], [3, 700], 9000),
    "shared tiles, in turn": ([1] * 20, [7] * 20, 600),
    "shared tiles": ([1] * 60, [7] * 60, 900),
    "prompts": ([20, 150, 60], [25, 200, 60], 300),
    "prompts without a prefix": ([30, 300], [30, 300], 0),
    "many rows": ([1] * 300, [9] * 300, 50),
}


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", list(SHAPES))
def test_a_query_of_nan_spoils_its_row_alone(afx, name, dim, dtype):
    c = Case(*SHAPES[name], dim=dim, dtype=dtype, seed=len(name))
    spoiled = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (c.tokens - 1, 9), (c.tokens // 2, 4)):
        c.q[t, h, 5] = math.nan
        spoiled[t, h] = True
    _check(afx, c, spoiled)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_keys_of_nan_spoil_the_rows_that_see_them(afx, name, dtype):
    """All keys of one request's head, so that whole pieces of its rows' keys are NaN, beside a healthy prefix."""
    c = Case(*SHAPES[name], dtype=dtype, seed=len(name))
    r = len(c.lens_list) - 1
    for j in range(c.lens_list[r]):
        c.pools[0][c.table_list[r][j // 16], j % 16, 1, 3] = math.nan
    spoiled = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    spoiled[c.starts_list[r]:c.starts_list[r + 1], 5:] = True  # heads 5 to 9 read the second key/value head
    _check(afx, c, spoiled)


@pytest.mark.parametrize("name", ["many pieces", "shared tiles, in turn", "shared tiles", "prompts"])
def test_keys_of_nan_in_the_prefix(afx, name):
    """The prefix's last key of one head: every row that reads the head, however the prefix is cut."""
    c = Case(*SHAPES[name], seed=len(name))
    j = c.prefix - 1
    c.pools[0][c.prefix_list[j // 16], j % 16, 0] = math.nan
    spoiled = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    spoiled[:, :5] = True
    _check(afx, c, spoiled)
