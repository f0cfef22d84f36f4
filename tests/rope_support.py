"""Rotary positions restated in float64 for the tests.  Shares no code with the CUDA
path or with the binding's frequencies."""
from __future__ import annotations

import math

import numpy as np

P = 16


def rotate(x, pos, freq, rot, interleaved, m=1.0, weight=None, eps=0.0):
    """(y, e) of x float64 [rows, heads, d] at positions pos [rows]: the rotated rows and the sizes m (|a| + |b|) of
    each value's pair, which the error bounds are relative to (|value| where it is not rotated)."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, size = x.copy(), np.abs(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = np.array([_angle(int(p), float(freq[i])) for p in pos])[:, None]
        c, s = np.cos(t), np.sin(t)
        y[..., a] = m * (x[..., a] * c - x[..., b] * s)
        y[..., b] = m * (x[..., b] * c + x[..., a] * s)
        size[..., a] = size[..., b] = m * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


_PI = 3141592653589793238462643383279502884197169399375105820974944  # 10^60 pi


def _angle(p, f):
    """p * f modulo 2 pi, in [-pi, pi), by whole numbers."""
    n, d = f.as_integer_ratio()
    scale = 10 ** 60
    x = p * n * scale // d  # 10^60 p f
    return ((x + _PI) % (2 * _PI) - _PI) / scale


def check(got, want, norm):
    """Values of bf16 rows against (y, size) of ``rotate``, by the roundings on the way:
    angle   p 2^-65 turns of the frequency's rounding and 2^-40 turns cut off: below 2^-31 rad
    sines   to fp32 by one rounding, 2^-24, from values that are good to 2^-35
    turn    a product, a fused product: 2^-24 of each of the two terms and of the result
    together below m (|a| + |b|) (2^-31 + 2^-24 + 2^-35 + 2^-23) < size 2^-21
    norm    the sum of squares: 19 additions, halved by the root, 9.5 2^-24; mean and eps 2 2^-24; the root 2^-22; two
            products 2 2^-24: below 18 2^-24 < 2^-19.8 of each value, 2^-19.2 with the above
    out     half a step of bf16, 2^-8 of the value"""
    y, size = want
    e = size * 2.0 ** (-19.2 if norm else -21)
    tol = e + 2.0 ** -8 * (np.abs(y) + e) + 1e-37
    err = np.abs(got - y)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))


def frequencies(n, base=10000.0, kind=None, s=1.0, original=0, fast=32.0, slow=1.0, low=1.0, high=4.0):
    """Radians a token of the n / 2 pairs: each scaling from its definition, a pair at a time."""
    out = []
    for i in range(n // 2):
        f = math.exp(-math.log(base) * 2 * i / n)
        turns = original * f / (2 * math.pi)
        if kind == "linear":
            f = f / s
        elif kind == "ntk":  # geometric from 1 to the last pair's frequency over s
            f = f / s ** (i / (n / 2 - 1))
        elif kind == "yarn":
            # pairs are numbered by how often they turn; between the two bounds, mixed by number
            first = max(0, math.floor(n * math.log(original / (fast * 2 * math.pi)) / (2 * math.log(base))))
            last = min(n - 1, math.ceil(n * math.log(original / (slow * 2 * math.pi)) / (2 * math.log(base))))
            mix = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
            f = mix * f / s + (1 - mix) * f
        elif kind == "wavelength":
            if turns <= low:
                f = f / s
            elif turns < high:
                mix = (turns - low) / (high - low)
                f = (1 - mix) * f / s + mix * f
        out.append(f)
    return np.array(out)


def places(t):
    """(row, page, slot, position) of every new row of a page table (numpy arrays)."""
    out = []
    for r in range(len(t["last_page_len"])):
        a0, a1 = int(t["qo_indptr"][r]), int(t["qo_indptr"][r + 1])
        p0, np_ = int(t["kv_indptr"][r]), int(t["kv_indptr"][r + 1] - t["kv_indptr"][r])
        kv = (np_ - 1) * P + int(t["last_page_len"][r]) if np_ else 0
        for row in range(a0, a1):
            pos = kv - (a1 - a0) + row - a0
            out.append((row, int(t["page_indices"][p0 + pos // P]), pos % P, pos))
    return np.array(out, np.int64).reshape(-1, 4)
