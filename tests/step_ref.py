"""Plain 64-bit definitions of the operators around a step's products, for the
tests: rounding to E4M3 in blocks of 128, products of such matrices, rotary
positions, verification of drafts.  Written from the definitions in
include/afx.h; they share no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128


def round_error(y: torch.Tensor, kind) -> torch.Tensor:
    """The most that one rounding to a type is off by: half a step, relative, and half the smallest number."""
    least = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
    return y.abs() * (torch.finfo(kind).eps / 2) + least[kind]


def e4m3_values() -> np.ndarray:
    """The value of each byte."""
    out = np.empty(256)
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        v = math.nan if (b & 127) == 127 else (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
        out[b] = -v if b & 128 else v
    return out


def quantize(x: np.ndarray):
    """(bytes' values, scales [blocks][tokens]) of float32 x [tokens][cols], each value the nearest of E4M3's."""
    table = e4m3_values()
    positive = table[:127]  # 0 .. 448, rising
    n, cols = x.shape
    values = np.empty((n, cols))
    scales = np.empty((-(-cols // BLOCK), n), np.float32)
    with np.errstate(all="ignore"):
        for b in range(scales.shape[0]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float32)
            a = np.abs(part).max(1)
            s = np.maximum((a.astype(np.float64) / 448).astype(np.float32), np.float32(2.0 ** -126))
            s = np.where(np.isfinite(part).all(1), s, np.float32(math.nan))
            scales[b] = s
            q = (part.astype(np.float64) / s.astype(np.float64)[:, None]).astype(np.float32).astype(np.float64)
            m = np.minimum(np.abs(q), 448.0)
            at = np.searchsorted(positive, m)          # positive[at - 1] < m <= positive[at]
            at = np.minimum(at, 126)
            low, high = positive[np.maximum(at - 1, 0)], positive[at]
            even = np.where(at % 2 == 0, high, low)    # bytes count up: an even byte is an even fraction
            near = np.where(m - low < high - m, low, np.where(m - low > high - m, high, even))
            near = np.where(m == high, high, near)
            values[:, b * BLOCK:(b + 1) * BLOCK] = np.where(np.isnan(q), math.nan, np.copysign(near, q))
    return values, scales


def product(w, w_scales, x, x_scales):
    """(y, reach) in float64: values w [rows][cols], x [tokens][cols]; reach = the sum of the magnitudes."""
    rows, cols = w.shape
    n = x.shape[0]
    y, reach = (torch.zeros((n, rows), dtype=torch.float64, device=w.device) for _ in range(2))
    by_row = w_scales.double().repeat_interleave(BLOCK, 0)[:rows]
    for b in range(-(-cols // BLOCK)):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        xs, ws = x[:, part].double(), w[:, part].double()
        f = x_scales[b].double()[:, None] * by_row[:, b][None, :]
        y += f * (xs @ ws.T)
        reach += f.abs() * (xs.abs() @ ws.abs().T)
    return y, reach


def rotate(x, positions, frequencies, axis_of_pair, rotary_dim, pairs, amplitude=1.0):
    """(y, reach) of x [tokens][heads][dim], positions [axes][tokens]: pair by pair, turns left out in integers of 2^-200."""
    y, reach = x.double().cpu().clone(), x.double().cpu().abs()
    one = 1 << 200
    # pi to 60 digits, for whole turns of far positions
    two_pi = 2 * 314159265358979323846264338327950288419716939937510582097494 * one // 10 ** 59
    half = rotary_dim // 2
    src = x.double().cpu()
    for i in range(half):
        num, den = float(frequencies[i]).as_integer_ratio()
        angles = []
        for p in positions[axis_of_pair[i]].tolist():
            angles.append((p * num * one // den) % two_pi / one)
        angle = torch.tensor(angles, dtype=torch.float64)[:, None]
        a, b = (i, i + half) if pairs == "halves" else (2 * i, 2 * i + 1)
        c, s = amplitude * angle.cos(), amplitude * angle.sin()
        y[..., a] = src[..., a] * c - src[..., b] * s
        y[..., b] = src[..., a] * s + src[..., b] * c
        both = abs(amplitude) * (src[..., a].abs() + src[..., b].abs())
        reach[..., a] = reach[..., b] = both
    return y, reach


def shares(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, near=0.0):
    """(p, sure, doubtful, amount): every token's share of what the parameters keep of logits z, in 64 bits; sure: no min-p boundary
    came within `near`, relative, of the other side; doubtful: the tokens around the top-p boundary that float32 weights may
    keep or not, amount their share together.  A
    weight e^y is off by 3 |y| 2^-24 (the difference, the reciprocal of T and their product are rounded) and 2^-22
    (the exponential), relative, so a running sum's share of the whole by at most twice the weights' mean of that, and
    2^-44 a token; half as much again is allowed for."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    p = np.zeros(len(z))
    m = z.max()
    if m == -np.inf:
        return p, True, set(), 0.0
    if not temperature > 0:
        p[int(np.argmax(z))] = 1.0
        return p, True, set(), 0.0
    with np.errstate(invalid="ignore"):
        y = np.where(z == m, 0.0, np.where(z == -np.inf, -np.inf, (z - m) / temperature))
    w = np.exp(y)
    order = np.lexsort((np.arange(len(z)), -z))
    if top_k > 0:
        order = order[:top_k]
    sure, doubtful, amount = True, set(), 0.0
    keep = np.ones(len(order), bool)
    if top_p < 1:
        before = (np.cumsum(w[order]) - w[order]) / w[order].sum()
        keep &= before < top_p
        share = w[order] / w[order].sum()
        off = 2 * (share * (3 * np.where(share > 0, np.abs(y[order]), 0.0) * 2.0 ** -24 + 2.0 ** -22)).sum() + len(order) * 2.0 ** -44
        close = np.abs(before - top_p) <= 1.5 * off
        doubtful, amount = set(order[close].tolist()), float(share[close].sum()) / top_p
    if min_p > 0:
        keep &= w[order] >= min(min_p, 1.0)
        sure &= np.abs(w[order] / min(min_p, 1.0) - 1).min() > near
    keep[0] = True
    p[order[keep]] = w[order[keep]] / w[order[keep]].sum()
    return p, bool(sure), doubtful, amount


def verify(p_rows, q_rows, drafts, u, draw_u, nears, doubtful):
    """(drafts that stand, the tokens that may be drawn behind them, sure) of one request: p_rows and q_rows the target's
    and the drafts' shares row by row (q_rows None: drafts that were not drawn); sure: no draft's test came within the
    row's `near` of the other result or was about one of a row's doubtful tokens.  A token may be drawn if draw_u is within `near` of
    its part of the running sum, of what is left over where that is a part.  -1: nothing to draw from."""
    sure, out = True, []
    rest, near = p_rows[len(drafts)], nears[len(drafts)]
    for i, d in enumerate(drafts):
        p, near = p_rows[i], nears[i]
        if d < 0 or d >= len(p):
            rest = p
            break
        sure &= d not in doubtful[i]
        q = q_rows[i] if q_rows is not None else (np.arange(len(p)) == d) * 1.0
        sure &= abs(u[i] * q[d] - p[d]) > near * max(p[d], u[i] * q[d]) or p[d] == q[d] == 0
        if u[i] * q[d] < p[d]:
            out.append(d)
            near = nears[len(drafts)]
            continue
        rest = np.maximum(p - q, 0.0)
        left = rest.sum()
        if left == 0:
            rest = p
        else:  # the differences' errors against their sum
            near = near / min(left, 1.0)
        break
    if rest.sum() == 0:
        return out, {-1}, sure
    run = np.cumsum(rest) / rest.sum()
    before = np.concatenate([[0.0], run[:-1]])
    may = (before <= draw_u + near) & (draw_u < run + near) & (rest > 0)
    may[np.nonzero(rest)[0][-1]] |= draw_u >= 1 - near
    return out, set(np.nonzero(may)[0].tolist()) | doubtful[len(out)], bool(sure)
