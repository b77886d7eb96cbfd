"""Plain float64 forms of the calls on a paged cache, with the error that their
float32 arithmetic and roundings may have (numpy, CPU)."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}   # half a subnormal step


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy()


def turns(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=1, fast=32.0, slow=1.0):
    """(radians per position [rotary_dim/2], magnitude)."""
    i = np.arange(rotary_dim // 2)
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = np.exp(-2.0 * i / rotary_dim * math.log(base))
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((original_len * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return g * f + (1 - g) * f / factor, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def norm_rope(x, pos, weight=None, eps=1e-6, freq=None, mag=1.0, interleaved=False):
    """x float64 [T][h][d] -> (y, scale of its float32 error: the length of each rotated pair)."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    size = np.abs(y)
    if freq is not None:
        half = len(freq)
        lo = np.arange(half) * 2 if interleaved else np.arange(half)
        hi = lo + 1 if interleaved else lo + half
        z = (y[..., lo] + 1j * y[..., hi]) * mag * np.exp(1j * pos[:, None, None] * freq)
        y[..., lo], y[..., hi] = z.real, z.imag
        size[..., lo] = size[..., hi] = np.abs(z)
    return y, size


def norm_rope_tolerance(y, size, dtype):
    """Half a step of the output type, and 2^-19 of the pair's length for the float32 arithmetic: a
    sum of d squares by 16 products per lane and four shuffles (20 roundings, halved by the root),
    rsqrt (2 of them), three products, sincospi (2) and the rounding of the fraction of a turn
    (2^-25 turns = 2^-22 radians, 4): 23 * 2^-24, doubled for the second order and the division."""
    return HALF_STEP[dtype] * np.abs(y) * 1.01 + TINY[dtype] + 2.0 ** -18.5 * size


def attend(q, keys, values, dist, scale, cap=0.0, slope=0.0, p_step=0.0, p_tiny=0.0):
    """One query over rows: q [d], keys, values [n][d], dist [n] -> (out [d], error bound [d]).

    p_step, p_tiny: half a step of the type that probabilities are rounded to, and its smallest.
    A score is off by 2^-17 of scale * sum |q_c k_c| (d/16 products of 16 terms, each good to some
    2^-22 of the running sum), 2^-21 of the cap and of every term that is added or subtracted (the
    score, the maximum, the bias), a probability by that factor and 2^-20 (powers, sums of n terms
    in many short chains); probabilities are relative to a maximum, so the sum is at least 2^-8 of
    the scale that the smallest step belongs to."""
    if len(keys) == 0:
        return np.zeros(q.shape[0]), np.zeros(q.shape[0])
    dots = keys @ q
    s = dots * scale
    if cap:
        s = cap * np.tanh(s / cap)
    s = s - slope * dist
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    out = p @ values / total
    delta = 2.0 ** -17 * scale * (np.abs(keys) @ np.abs(q)) + 2.0 ** -20 + \
        2.0 ** -21 * (cap + np.abs(s) + abs(top) + slope * dist)
    weigh = p * (delta + p_step) + p_tiny
    err = weigh @ np.abs(values) / total + np.abs(out) * (p * delta).sum() / total
    return out, err


def gather(pool, table_row, j, head, page):
    """Rows j of one sequence's head from pool [n_pages][H][page][d]."""
    j = np.asarray(j, np.int64)
    return pool[table_row[j // page], head, j % page]
