"""Frequencies of rotary positions, as the rotating calls take them.

``frequencies`` gives the radians a position of each pair of values, for the plain
form and for the usual scalings of a trained model to longer contexts; ``Rotary``
holds them on the device in the library's form, 64-bit fractions of a turn. The product
of a position and such a fraction is exact modulo a turn; what the angle is off by is the
frequency's own rounding: position * 2^-65 turns from the fraction (2^-25 of a turn at
position 2^40), and position times the rounding of the double that it is made from (a
relative 2^-50 at most: 2^-10 radians at one radian a position and position 2^40).
"""
from __future__ import annotations

import math
from fractions import Fraction

import torch

_TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


def frequencies(rotary_dim, base=10000.0, scaling=None):
    """(frequencies in radians a position, a float for each of the rotary_dim / 2 pairs;
    the factor on cosines and sines). Without scaling they are base ** (-2 i / rotary_dim).

    ``scaling`` is a dict with a "type" and a "factor" f > 0 (how much longer contexts
    get), and
      "linear"    every position counts as position / f;
      "ntk"       the base grows, by f ** (rotary_dim / (rotary_dim - 2)), so that the
                  slowest pair is slowed by f and the fastest not at all;
      "by_parts"  pairs whose wavelength is above trained / low_turns are slowed by f, those
                  below trained / high_turns not at all, the others in between, linear in
                  the turns they make within the trained length (keys
                  "original_max_position", "low_turns" = 1, "high_turns" = 4);
      "yarn"      the same with a ramp over the pairs' numbers, between the ones that make
                  "fast_turns" = 32 and "slow_turns" = 1 turns in "original_max_position",
                  and a factor 0.1 ln f + 1 on cosines and sines unless
                  "attention_factor" is given.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not base > 0 or not math.isfinite(base):
        raise ValueError(f"base must be positive, got {base}")
    half = rotary_dim // 2
    plain = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    if scaling is None:
        return plain, 1.0
    how, f = scaling.get("type"), float(scaling.get("factor", 1.0))
    if not f > 0 or not math.isfinite(f):
        raise ValueError(f"scaling: factor must be positive, got {f}")
    known = {"linear": (), "ntk": (),
             "by_parts": ("original_max_position", "low_turns", "high_turns"),
             "yarn": ("original_max_position", "fast_turns", "slow_turns", "attention_factor")}
    if how not in known:
        raise ValueError(f"scaling: type must be one of {sorted(known)}, got {how!r}")
    extra = set(scaling) - {"type", "factor", *known[how]}
    if extra:
        raise ValueError(f"scaling: {how} has no {sorted(extra)}")
    if how == "linear":
        return [w / f for w in plain], 1.0
    if how == "ntk":
        if rotary_dim < 4:
            raise ValueError("scaling: ntk needs two pairs at least")
        return frequencies(rotary_dim, base * f ** (rotary_dim / (rotary_dim - 2.0)))
    trained = float(scaling["original_max_position"])
    if not trained > 0:
        raise ValueError("scaling: original_max_position must be positive")
    if how == "by_parts":
        lo, hi = (float(scaling.get(k, v)) for k, v in (("low_turns", 1.0), ("high_turns", 4.0)))
        if not 0 < lo < hi:
            raise ValueError("scaling: 0 < low_turns < high_turns")
        out = []
        for w in plain:
            kept = min(1.0, max(0.0, (trained * w / (2.0 * math.pi) - lo) / (hi - lo)))
            out.append(w * kept + w / f * (1.0 - kept))
        return out, 1.0
    fast, slow = (float(scaling.get(k, v)) for k, v in (("fast_turns", 32.0), ("slow_turns", 1.0)))
    if not 0 < slow < fast or not base > 1:
        raise ValueError("scaling: 0 < slow_turns < fast_turns, and a base above 1")

    def pair_of(turns):  # the (fractional) pair that makes so many in the trained length
        return rotary_dim * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    lo = max(math.floor(pair_of(fast)), 0)
    hi = min(math.ceil(pair_of(slow)), rotary_dim - 1)
    out = []
    for i, w in enumerate(plain):
        slowed = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
        out.append(w / f * slowed + w * (1.0 - slowed))
    m = scaling.get("attention_factor")
    return out, (0.1 * math.log(f) + 1.0 if f > 1 else 1.0) if m is None else float(m)


def turns_of(radians) -> list[int]:
    """Each frequency (radians a position) in units of 2^-64 turns, modulo a whole turn."""
    out = []
    for w in radians:
        if not math.isfinite(w):
            raise ValueError(f"frequencies must be finite, got {w}")
        out.append(round(Fraction(float(w)) * 2 ** 64 / _TWO_PI) % 2 ** 64)
    return out


class Rotary:
    """Rotary positions of the first ``rotary_dim`` values (a multiple of 16) of each head:
    ``turns`` and ``factor`` for qk_rope and qk_rope_append, from a base and a scaling (see
    ``frequencies``) or from frequencies (radians a position) given as they are.
    ``interleaved`` pairs neighbouring values, otherwise the two halves."""

    def __init__(self, rotary_dim, base=10000.0, scaling=None, interleaved=False, radians=None,
                 factor=None, device="cuda"):
        if rotary_dim < 16 or rotary_dim % 16:
            raise ValueError(f"rotary_dim must be a multiple of 16, got {rotary_dim}")
        made, m = frequencies(rotary_dim, base, scaling) if radians is None else (radians, 1.0)
        self.radians = [float(w) for w in made]
        if len(self.radians) != rotary_dim // 2:
            raise ValueError(f"{rotary_dim // 2} frequencies are wanted, got {len(self.radians)}")
        self.rotary_dim, self.interleaved = rotary_dim, bool(interleaved)
        self.factor = float(m if factor is None else factor)
        signed = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns_of(self.radians)]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)

    def args(self):
        """The keyword arguments of the rotating calls."""
        return {"turns": self.turns, "factor": self.factor, "interleaved": self.interleaved}
