"""Plain 64-bit form of the attention of a chunk over bf16 pages, and the bound of the
kernel's error (not collected by pytest)."""
from __future__ import annotations

import math

import torch


def seen(position, n, window, sinks):
    """Truth values [n]: the keys that the query at `position` sees."""
    t = torch.arange(n)
    see = t <= position
    if window:
        see &= (t > position - window) | (t < sinks)
    return see


def attention(q, keys, values, first, window, sinks, scale):
    """(out, bound) [k][Hq][D] doubles for one request whose queries sit at first + j.

    bound: a weight is rounded to bf16 (2^-8 of it) before its product and the sum; its
    score, D products accumulated in fp32 and scaled, is off by (D + 64) 2^-24 of
    scale sum |q k| (64: the scale's product, the exponential's 2 ulp, the running
    maximum's factors).  Numerator and denominator both carry that, so 2 delta of
    sum_t p_t |v_t|; partial sums in fp32 add less than 2^-16 of it; the result is
    rounded to bf16 once (2^-8 of it)."""
    k, hq, d = q.shape
    g = hq // keys.shape[1]
    n = keys.shape[0]
    out = torch.zeros((k, hq, d), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for j in range(k):
        see = seen(first + j, n, window, sinks)
        for c in range(keys.shape[1]):
            kk, vv = keys[see, c], values[see, c]
            qq = q[j, c * g:(c + 1) * g]
            p = torch.softmax(qq @ kk.T * scale, -1)
            o = p @ vv
            out[j, c * g:(c + 1) * g] = o
            size = float((qq.abs() @ kk.abs().T).max()) * abs(scale)
            delta = 2.0 ** -8 + size * (d + 64) * 2.0 ** -24 + 2.0 ** -17
            bound[j, c * g:(c + 1) * g] = (2 * delta * (p @ vv.abs()) * (1 + 2.0 ** -8)
                                           + 2.0 ** -8 * o.abs() + math.ulp(0.0))
    return out, bound
