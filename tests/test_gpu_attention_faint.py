"""FP16 attention where one key outweighs very many faint ones: their shares,
each below 2^-25 of the largest, add up and must reach the output, not the
sum alone.

One key scores 18 above all others (weights e^-18, about 2^-26), its value is
0 and all others' are 1, so with n of them the output is n e^-18 / (1 + n
e^-18).  Weights are held with 2^7 of headroom below the largest: those below
2^-21 of it have an absolute error of 2^-32 each, so |err| <= n 2^-32 + 2 u
out, and a few u of the scores (2^-24 * 18, relative).  The sum itself is a
running one in float32: a thread adds n / 4 weights or fewer to it, each
rounded by 2^-24 of the sum at most, so lse has an error of n 2^-26 besides.
"""
import math

import pytest
import torch

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

DIM, PAGE = 64, 256


def _run(afx, starts, lens, prefix_table, prefix, table, pools, q_heads):
    tokens = starts[-1]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = torch.zeros((tokens, q_heads, DIM), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 12.0
    out, lse = torch.empty_like(q), torch.empty((tokens, q_heads), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = afx.attention_args(afx.kv_cache(*pools), q_heads, tokens, ints(starts), ints(lens), ints(table), 1 / math.sqrt(DIM),
                              ints(prefix_table) if prefix else None, prefix)
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    afx.afx_attention_plan(args, ws, status_dev=status)
    afx.afx_attention(args, q, out, ws, lse=lse, status_dev=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out.double(), lse.double()


def _pools(pages, heads):
    """All keys zero and all values one, but token 0 of page 0."""
    k = torch.zeros((pages, PAGE, heads, DIM), dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, :, 0] = 12.0  # 12 * 12 / 8 = 18
    v[0, 0] = 0.0
    return k, v


def _check(out, lse, n):
    """n: faint keys a token."""
    n = torch.tensor(n, dtype=torch.float64, device="cuda")[:, None]
    want = n * math.exp(-18.0) / (1 + n * math.exp(-18.0))
    err = (out - want[..., None]).abs()
    assert (err <= (n * 2.0 ** -32 + want * (2 * 2.0 ** -11 + 2.0 ** -18))[..., None]).all(), (err.max().item(), want.max().item())
    assert ((lse - 18.0 - torch.log1p(n * math.exp(-18.0))).abs() <= 2.0 ** -17 + n * 2.0 ** -26).all()


def test_single_tokens(afx):
    """64 requests on the same 20,480 keys, 32 heads: pieces of thousands of keys."""
    n = 80 * PAGE
    out, lse = _run(afx, list(range(65)), [n] * 64, [], 0, [list(range(80))] * 64, _pools(80, 32), 32)
    _check(out, lse, [n - 1] * 64)


@pytest.mark.parametrize("tokens", [100, 250])
def test_prompts(afx, tokens):
    """A tile group a head and a head an SM, so that none is cut; 100 rows: the two tiles take the steps in turn."""
    heads = torch.cuda.get_device_properties(0).multi_processor_count
    pages, prefix = 65, 64 * PAGE
    out, lse = _run(afx, [0, tokens], [tokens], list(range(64)), prefix, [[64]], _pools(pages, heads), heads)
    _check(out, lse, [prefix + i for i in range(tokens)])


def test_the_largest_key_comes_last(afx):
    """The reference rises late: the weights so far are scaled in float32."""
    n = 80 * PAGE
    k, v = _pools(80, 32)
    out, lse = _run(afx, list(range(65)), [n] * 64, [], 0, [list(range(1, 80)) + [0]] * 64, (k, v), 32)
    _check(out, lse, [n - 1] * 64)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 20], [1] * 20, [1] * 60, [40, 200]])
def test_scores_far_apart(afx, new, dim):
    """Scores in the hundreds: maxima rise past what the weights' headroom takes, within a step and between steps."""
    Case(new, [n + 60 for n in new], 900, dim=dim, dtype="float16", sharp=8.0, seed=dim).check(afx)


@pytest.mark.parametrize("most", [0.2, 1.0, 3.0])
@pytest.mark.parametrize("requests", [2, 20, 60])
def test_scores_that_rise(afx, requests, most):
    """Every key scores above all before it, by a little or a lot."""
    c = Case([1] * requests, [9] * requests, 1100, dtype="float16", seed=14)
    line = torch.linspace(-most, most, 1100, device="cuda").to(c.dtype)
    for j in range(1100):
        c.pools[0][c.prefix_list[j // 16], j % 16] = line[j]
    c.q.copy_(torch.ones_like(c.q) * 2)
    c.check(afx)
