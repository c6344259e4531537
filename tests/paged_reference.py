"""Plain 64-bit forms of the rotary paged appends and of the attention over
block-scaled e4m3 pages, position by position (not collected by pytest)."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn
EXP_MIN, EXP_MAX = -100, 100


def decode(byte_tensor: torch.Tensor) -> torch.Tensor:
    """e4m3 bytes (uint8) as doubles."""
    return byte_tensor.cpu().view(E4M3).to(torch.float32).double()


def rotate(x, table, pos, interleaved):
    """x [heads][D] doubles, rotated by row `pos` of the table."""
    r = table.shape[1]
    c, s = table[pos, :r // 2].double(), table[pos, r // 2:].double()
    y = x.clone()
    ia = torch.arange(r // 2) * 2 if interleaved else torch.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    y[:, ia] = x[:, ia] * c - x[:, ib] * s
    y[:, ib] = x[:, ib] * c + x[:, ia] * s
    return y


def pair_magnitude(x, table, interleaved):
    """|x| + |partner| for every element: the rotation's absolute terms (each
    cosine and sine is at most 1)."""
    r = table.shape[1]
    m = x.abs().clone()
    ia = torch.arange(r // 2) * 2 if interleaved else torch.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    both = m[:, ia] + m[:, ib]
    m[:, ia], m[:, ib] = both, both
    return m


def scale_exponent(amax: float) -> int:
    """Least e in [EXP_MIN, EXP_MAX] with amax <= 448 * 2^e."""
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def attention(q, keys, values, positions, window, scale, value_scales=None):
    """out [k][Hq][D] doubles and W = sum_t p_t |v_t| for one request.

    q [k][Hq][D]; keys, values [n][Hkv][D] (positions 0..n-1); positions[j] of
    query j; value_scales [n][Hkv]: the scales within the values (their bytes stand
    for value / scale).  With them W also holds the floor of the weights'
    rounding (see attention_tolerance)."""
    k, hq, d = q.shape
    hkv = keys.shape[1]
    g = hq // hkv
    out = torch.zeros((k, hq, d), dtype=torch.float64)
    weight = torch.zeros_like(out)
    for j in range(k):
        p = int(positions[j])
        lo = max(0, p - window + 1) if window else 0
        for c in range(hkv):
            s = q[j, c * g:(c + 1) * g] @ keys[lo:p + 1, c].T * scale
            w = torch.softmax(s, -1)
            out[j, c * g:(c + 1) * g] = w @ values[lo:p + 1, c]
            weight[j, c * g:(c + 1) * g] = w @ values[lo:p + 1, c].abs()
            if value_scales is not None:
                vs = value_scales[lo:p + 1, c]
                top = (w * vs).amax(-1, keepdim=True)
                bytes_ = (values[lo:p + 1, c].abs() / vs[:, None]).sum(0)
                weight[j, c * g:(c + 1) * g] += 2.0 ** -18 * top * bytes_
    return out, weight


def score_magnitude(q, keys, scale):
    """Largest scale * sum_d |q_d k_d| over queries and keys."""
    k, hq, d = q.shape
    g = hq // keys.shape[1]
    return max(float((q[:, c * g:(c + 1) * g].abs().reshape(-1, d) @ keys[:, c].abs().T).max())
               for c in range(keys.shape[1])) * abs(scale)


def attention_tolerance(out, weight, q, keys, scale):
    """Elementwise bound of the bf16 output's error.

    Every weight p_t is off by at most a relative delta: its rounding to f16
    (2^-11), and its score, a sum of D products accumulated in fp32, by
    (D + 64) 2^-24 of sum |q k| (64: the scales' products, the exponential's 2
    ulp and the conversion to log2 units).  The numerator carries both; the
    denominator, a sum of the weights before that rounding, the second.  The
    result is rounded to bf16 once (2^-8).

    Floor: the weights p_t vs_t that meet the bytes are formed times 64 / (a weight
    of the row), so the row's largest is at least 64 then, as f16 (off by at most
    2^-25) and as three e5m2 pieces, the last in steps of 2^-16 / 64 (off by at most
    2^-23): less than 2^-28 of the largest weight, times the byte's value.
    attention() adds 2^-18 of that product to W, which delta >= 2^-10 makes 2^-28."""
    d = q.shape[2]
    delta = 2 * (2.0 ** -11 + score_magnitude(q, keys, scale) * (d + 64) * 2.0 ** -24)
    return 2.0 ** -8 * out.abs() + delta * weight * (1 + 2.0 ** -8) + math.ulp(0.0)
