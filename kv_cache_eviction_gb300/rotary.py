"""Frequencies of rotary positions, for ``kv_rotary``: plain ones, and the ways to stretch those of
a model trained on shorter contexts."""
from __future__ import annotations

import math


def kv_rotary_inv_freq(rot: int, base: float = 10000.0, scaling: str = "none",
                       factor: float = 1.0, trained: int = 8192, slow: float = 1.0,
                       fast: float = 32.0):
    """The ``rot / 2`` frequencies (float64, host) and the magnitude for ``KvRotaryShape``.

    f_i = base^(-2 i / rot), and with ``scaling``

    * ``"none"``: f_i;
    * ``"linear"``: f_i / factor (positions interpolated);
    * ``"base"``: base times factor^(rot / (rot - 2)), so that the slowest pair is the linear one's
      and the fastest stays;
    * ``"bands"``: by the turns n_i = trained f_i / 2 pi that a pair makes over the trained
      length: f_i / factor up to ``slow`` of them, f_i from ``fast`` on, and between the mix
      with the weight (n_i - slow) / (fast - slow) on f_i;
    * ``"yarn"``: the same two ends, mixed by a ramp over the pairs' numbers, from the pair of
      ``fast`` turns (rounded down, pair 0 at least) to that of ``slow`` turns (rounded up), which
      lies behind the last pair where all of them make more turns; the magnitude is
      0.1 ln(factor) + 1.
    """
    import torch
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be positive and even")
    if not (base > 1.0 and factor >= 1.0 and trained > 0 and 0.0 < slow < fast):
        raise ValueError("base > 1, factor >= 1, trained > 0 and 0 < slow < fast are needed")
    if scaling == "base":
        if rot <= 2:
            raise ValueError("scaling 'base' needs more than one pair")
        base *= factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if scaling in ("none", "base"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(fast)), 0)
        hi = math.ceil(pair(slow))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    raise ValueError("scaling must be none, linear, base, bands or yarn")
