"""Plain 64-bit definitions of the serving operators, for the tests.

Written from the definitions in include/afx.h: Python lists and a stack for
the page tables, one request at a time for attention, one row at a time for
sampling.  They share no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch


def pages(n: int, page: int) -> int:
    return -(-n // page)


def kv_tables(page, old, new, table, stack, count, max_tokens):
    """(table, stack, count, starts, slots, positions) after the call; table and stack are nested lists."""
    table = [list(r) for r in table]
    free = list(stack[:count])
    for r in range(len(old)):
        for c in range(pages(new[r], page), pages(old[r], page)):
            free.append(table[r][c])
    starts, slots, positions = [], [], []
    for r in range(len(old)):
        starts.append(len(slots))
        for c in range(pages(old[r], page), pages(new[r], page)):
            table[r][c] = free.pop()
        for pos in range(old[r], new[r]):
            slots.append(table[r][pos // page] * page + pos % page)
            positions.append(pos)
    starts.append(len(slots))
    pad = [-1] * (max_tokens - len(slots))
    # the stack's entries up to the lower of the two counts keep their values
    stack = free + list(stack[len(free):])
    return table, stack, len(free), starts, slots + pad, positions + pad


def attention(q, k_pool, v_pool, prefix_table, prefix_len, starts, lens, table, scale):
    """(out, lse, weight, reach) in float64: weight = sum_j p_j |v_j|, the scale of the output's rounding
    errors; reach = max_j scale * sum |q_i k_ji|, that of the scores' (q [t][hq][d], pools [page][token][hkv][d])."""
    page, kvh = k_pool.shape[1], k_pool.shape[2]
    group = q.shape[1] // kvh
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    weight, reach = torch.zeros_like(out), torch.zeros_like(lse)
    for r, length in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        where = [(prefix_table[j // page], j % page) for j in range(prefix_len)]
        where += [(table[r][j // page], j % page) for j in range(length)]
        if a == b or not where:
            continue
        at = torch.tensor(where, device=q.device)
        k = k_pool[at[:, 0], at[:, 1]].double().repeat_interleave(group, 1)  # [keys][hq][d]
        v = v_pool[at[:, 0], at[:, 1]].double().repeat_interleave(group, 1)
        for t in range(a, b):
            n = max(0, min(len(where), prefix_len + length - (b - a) + (t - a) + 1))
            n = max(n, prefix_len)
            if n == 0:
                continue
            x = torch.einsum("hd,khd->hk", q[t].double(), k[:n]) * scale
            lse[t] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            out[t] = torch.einsum("hk,khd->hd", p, v[:n])
            weight[t] = torch.einsum("hk,khd->hd", p, v[:n].abs())
            reach[t] = (torch.einsum("hd,khd->hk", q[t].double().abs(), k[:n].abs()) * abs(scale)).amax(1)
    return out, lse, weight, reach


def sample(z, u, t=1.0, k=0, p=1.0, min_p=0.0, near=0.0):
    """(token, logprob, sure, allows): the token drawn and its log probability; sure: no decision (a top-p or min-p
    boundary, the draw) came within `near`, as a share of the mass, of the other side; allows(token) -> (low, high) or
    None: whether a token can come of decisions each off by at most `near`, and between what its logprob then lies."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    top = z.max()
    if top == -np.inf:
        return -1, -math.inf, True, None
    if not t > 0:
        return int(np.argmax(z)), 0.0, True, None
    with np.errstate(invalid="ignore"):
        y = np.where(z == top, 0.0, np.where(z == -np.inf, -np.inf, (z - top) / t))
    w = np.exp(y)
    order = np.lexsort((np.arange(len(z)), -z))
    if k > 0:
        order = order[:k]
    before, total = np.cumsum(w[order]) - w[order], w[order].sum()

    def kept(p_, min_p_):
        keep = np.ones(len(order), bool)
        if p < 1:
            keep &= before < p_ * total
        if min_p > 0:
            keep &= w[order] >= min(min_p_, 1.0)
        keep[0] = True
        mass = np.zeros(len(z))
        mass[order[keep]] = w[order[keep]]
        return mass

    mass, low, high = kept(p, min_p), kept(p - near, min_p + near), kept(p + near, min_p - near)
    run = np.cumsum(mass)
    token = min(int(np.searchsorted(run, u * run[-1], side="right")), int(np.nonzero(mass)[0][-1]))
    run_low, run_high = np.cumsum(low), np.cumsum(high)

    def allows(i):
        if not (0 <= i < len(z)) or high[i] == 0:
            return None
        if (run_low[i] - low[i]) / run_high[-1] > u + near or run_high[i] / run_low[-1] < u - near:
            return None
        return y[i] - math.log(run_high[-1]), y[i] - math.log(run_low[-1])

    edge = np.abs(run / run[-1] - u)[np.nonzero(mass)[0][:-1]]
    sure = np.array_equal(low, high) and (len(edge) == 0 or edge.min() > near)
    return token, float(y[token] - math.log(run[-1])), bool(sure), allows
