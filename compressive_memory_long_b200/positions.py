"""Frequencies of the rotary positions (host side): the table ``binding.rotary`` and
``binding.paged_decode_step`` take.

``rotary_frequencies(rot)`` gives base^(-2i/rot), i < rot/2, in 64 bits.  Three published ways
of running a model past its trained length change the table:

* ``"linear"``: positions divided by ``factor`` (position interpolation), that is every
  frequency divided by it;
* ``"ntk"``: the base raised to base * factor^(rot / (rot - 2)), which leaves the fastest pair
  as it is and divides the slowest by ``factor``;
* ``"yarn"``: pairs that turn more than ``fast`` times over the trained length keep their
  frequency, those that turn less than ``slow`` times are divided by ``factor``, with a linear
  ramp over the pair's index between, and q and k are each scaled by 0.1 ln(factor) + 1.
"""
from __future__ import annotations

import math

import torch


def rotary_frequencies(rot: int, *, base: float = 10000.0, scaling=None, factor: float = 1.0,
                       trained_length=None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(freq [rot/2] fp64 on ``device``, scale): the table and the factor of ``rotary``."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot must be even and not negative, got {rot}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling is not None and factor < 1:
        raise ValueError(f"factor must be at least 1, got {factor}")
    scale = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / max(rot, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if trained_length is None:
            raise ValueError("yarn needs trained_length")
        scale = 0.1 * math.log(factor) + 1.0

        def index(turns):   # the pair that turns this often over the trained length
            return rot * math.log(trained_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
    return freq.to(device), scale
