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
