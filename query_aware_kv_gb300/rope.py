"""Rotary positions on the host: frequencies (unscaled, or stretched for contexts longer than a
model was trained on) and the descriptor that the library's calls take."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

from . import _lib

SCALINGS = (None, "linear", "ntk", "bands", "yarn")


def rope_frequencies(rotary_dim: int = _lib.HEAD_DIM, base: float = 10000.0,
                     scaling: Optional[str] = None, factor: float = 1.0,
                     original_length: Optional[float] = None, low_turns: float = 1.0,
                     high_turns: float = 4.0, beta_fast: float = 32.0, beta_slow: float = 1.0
                     ) -> Tuple[list, float]:
    """The rotary_dim / 2 frequencies (radians per position) and the magnitude that cosines and
    sines are multiplied by.  Pair i has base^(-2 i / rotary_dim), and with a scaling:

    ``linear``  every frequency divided by factor (positions interpolated);
    ``ntk``     the base times factor^(d / (d - 2)): the slowest pair divided by factor, the
                fastest as it is;
    ``bands``   pairs that turn less than low_turns times over original_length positions are
                divided by factor, those that turn more than high_turns times are not, those
                between in proportion to their turns;
    ``yarn``    in proportion to the pair's index between those that turn beta_fast times (not
                divided) and beta_slow times (divided by factor), with a magnitude of
                0.1 ln(factor) + 1.
    """
    d = int(rotary_dim)
    if d < 8 or d > _lib.HEAD_DIM or d % 8:
        raise ValueError("rotary_dim must be 8, 16, ..., 128")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError("base must be finite and above 1")
    if not factor > 0.0 or not math.isfinite(factor):
        raise ValueError("factor must be finite and positive")
    if scaling in ("bands", "yarn") and not (original_length or 0) > 0:
        raise ValueError(f"{scaling} needs original_length")
    if scaling == "ntk":
        base = base * factor ** (d / (d - 2))
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    magnitude = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "bands":
        if not 0 <= low_turns < high_turns:
            raise ValueError("low_turns must be at least 0 and below high_turns")
        for i, x in enumerate(f):
            turns = original_length * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            f[i] = keep * x + (1 - keep) * x / factor
    elif scaling == "yarn":
        if not 0 < beta_slow < beta_fast:
            raise ValueError("beta_slow must be positive and below beta_fast")

        def pair(turns):  # the index of the pair that turns this often
            return d * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), d - 1)
        for i, x in enumerate(f):
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f[i] = ramp * x / factor + (1 - ramp) * x
        magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return f, magnitude


class Rope:
    """A rotation of heads by their positions, for ``rotate``, ``prefill_rotary`` and the other
    rotary calls.  The pairs are dims (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with
    ``interleaved``; the dims past rotary_dim pass through.  The arguments are those of
    ``rope_frequencies``; ``magnitude`` replaces the scaling's own."""

    def __init__(self, rotary_dim: int = _lib.HEAD_DIM, base: float = 10000.0,
                 interleaved: bool = False, scaling: Optional[str] = None, factor: float = 1.0,
                 original_length: Optional[float] = None, magnitude: Optional[float] = None, **kw):
        f, m = rope_frequencies(rotary_dim, base, scaling, factor, original_length, **kw)
        self._fill(f, interleaved, m if magnitude is None else magnitude)

    @classmethod
    def from_frequencies(cls, inv_freq: Sequence[float], interleaved: bool = False,
                         magnitude: float = 1.0) -> "Rope":
        """A rotation of 2 len(inv_freq) dims by these frequencies (radians per position)."""
        self = cls.__new__(cls)
        self._fill([float(x) for x in inv_freq], interleaved, magnitude)
        return self

    def _fill(self, inv_freq, interleaved, magnitude):
        if len(inv_freq) > 64:  # the descriptor's room
            raise ValueError("at most 64 frequencies")
        self.inv_freq, self.interleaved = tuple(inv_freq), bool(interleaved)
        self.magnitude, self.rotary_dim = float(magnitude), 2 * len(inv_freq)
        self.desc = _lib.QuestRope()
        arr = (ctypes.c_double * max(1, len(inv_freq)))(*inv_freq)
        _lib._check(_lib.load().quest_rope_init(ctypes.byref(self.desc), self.rotary_dim,
                                                int(self.interleaved), arr, self.magnitude))
        self.ref = ctypes.byref(self.desc)
