"""The frequencies of rotary positions: how far each pair of a head's dims turns a
token, with the scalings that models use for contexts longer than they were trained
on.  Host arithmetic in float64; the calls that rotate are in the package itself."""
from __future__ import annotations

import math

import numpy as np

# keys of a scaling beside "type" and "factor"
_SCALINGS = {"linear": (), "ntk": (), "yarn": ("original", "beta_fast", "beta_slow", "magnitude"),
             "wavelength": ("original", "low", "high")}


def rope_frequencies(rotary_dim, base=10000.0, scaling=None):
    """(radians a token of the rotary_dim / 2 pairs, float64; magnitude) of
    f_i = base^(-2 i / rotary_dim) under ``scaling``: None, or a dict with "type",
    "factor" s >= 1 and what its type takes besides:

    * ``linear``: f_i / s (positions interpolated);
    * ``ntk``: base * s^(rotary_dim / (rotary_dim - 2)) in base's place: the fastest
      pair as it was, the slowest slower by s;
    * ``yarn``: with n_i = ``original`` f_i / 2 pi turns in the trained context, pairs
      of more than ``beta_fast`` (32) turns as they were, of fewer than ``beta_slow``
      (1) f_i / s, a linear mixture over the pairs' indices between (the first bound
      rounded down to a pair, the second up); the magnitude is 0.1 ln s + 1 unless
      "magnitude" gives another;
    * ``wavelength``: pairs of ``high`` (4) turns or more in the ``original`` context
      as they were, of ``low`` (1) or fewer f_i / s, mixed in between by their turns.
    """
    f, m = frequencies_of(rotary_dim, base, scaling)
    return np.array(f), m


def frequencies_of(rotary_dim, base, scaling):
    """``rope_frequencies`` with the frequencies in a list."""
    n, base = int(rotary_dim), float(base)
    if n < 2 or n % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (math.isfinite(base) and base > 0):
        raise ValueError("base must be finite and > 0")
    f = [base ** (-2 * i / n) for i in range(n // 2)]
    if scaling is None:
        return f, 1.0
    kind = scaling.get("type")
    if kind not in _SCALINGS:
        raise ValueError(f"scaling type must be one of {', '.join(sorted(_SCALINGS))}")
    takes = _SCALINGS[kind]
    unknown = set(scaling) - {"type", "factor"} - set(takes)
    if unknown:
        raise ValueError(f"{kind} scaling takes no {', '.join(sorted(map(str, unknown)))}")
    s = float(scaling.get("factor", math.nan))
    if not (math.isfinite(s) and s >= 1):
        raise ValueError("scaling needs a factor >= 1")
    if "original" in takes:
        original = scaling.get("original")
        if original is None or not (math.isfinite(original) and original > 0):
            raise ValueError(f"{kind} scaling needs the original context, > 0")
        turns = float(original) / (2 * math.pi)
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "ntk":
        if n < 4:
            raise ValueError("ntk scaling needs a rotary_dim of 4 or more")
        base *= s ** (n / (n - 2))
        return [base ** (-2 * i / n) for i in range(n // 2)], 1.0
    if kind == "wavelength":
        low, high = float(scaling.get("low", 1.0)), float(scaling.get("high", 4.0))
        if not 0 <= low < high < math.inf:
            raise ValueError("wavelength scaling needs 0 <= low < high")
        keep = [min(max((turns * x - low) / (high - low), 0.0), 1.0) for x in f]
        return [k * x + (1 - k) * x / s for k, x in zip(keep, f)], 1.0
    fast, slow = float(scaling.get("beta_fast", 32.0)), float(scaling.get("beta_slow", 1.0))
    if not 0 < slow <= fast < math.inf or base <= 1:
        raise ValueError("yarn scaling needs 0 < beta_slow <= beta_fast and a base > 1")
    # the (fractional) pair that makes b turns: base^(2 i / n) = turns / b
    pair_of = lambda b: n / 2 * math.log(turns / b) / math.log(base)  # noqa: E731
    lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), n - 1)
    mix = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(n // 2)]
    return [x * (1 - k) + x / s * k for k, x in zip(mix, f)], float(scaling.get("magnitude", 0.1 * math.log(s) + 1))
