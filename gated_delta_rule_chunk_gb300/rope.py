"""The rotary table of the attention front end: cos and sin of position times frequency,
evaluated in 64 bits and rounded once, so that long positions lose nothing (in 32 bits the
angle of position 10^5 alone is off by about 4e-3). Made once per model and kept."""
from __future__ import annotations

import math
from typing import Optional

import torch


def rope_frequencies(rot: int, base: float = 10000.0, linear: float = 1.0, ntk: float = 1.0,
                     by_parts: Optional[tuple] = None) -> torch.Tensor:
    """The rot / 2 angles per position, base^(-2i/rot) (fp64), scaled for long contexts.

    linear    positions are divided by this factor
    ntk       the base is raised to base * ntk^(rot / (rot - 2)): the slowest pair is
              stretched by the factor, the fastest kept
    by_parts  (factor, trained_length, few, many): a pair that turns fewer than `few` times
              within trained_length is stretched by the factor, one that turns more than
              `many` times is kept, linear in the number of turns between (the "by parts"
              interpolation of Peng et al., "YaRN: Efficient Context Window Extension of
              Large Language Models", 2023, section 3.2)
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if ntk != 1.0 and rot > 2:
        base = base * ntk ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / linear
    if by_parts is not None:
        factor, trained, few, many = by_parts
        if not many > few:
            raise ValueError("by_parts needs many > few")
        keep = ((f * trained / (2 * math.pi) - few) / (many - few)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f


def rope_table(max_pos: int, rot: int, base: float = 10000.0, linear: float = 1.0,
               ntk: float = 1.0, by_parts: Optional[tuple] = None, magnitude: float = 1.0,
               device="cuda") -> torch.Tensor:
    """fp32 [max_pos, rot]: magnitude * cos(p f_i), then magnitude * sin(p f_i), for the
    frequencies of rope_frequencies. `magnitude` is the factor on q and k that some
    long-context rules add (0.1 ln(factor) + 1 in the paper named there)."""
    f = rope_frequencies(rot, base, linear, ntk, by_parts)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return (magnitude * torch.cat([angle.cos(), angle.sin()], 1)).to(torch.float32).to(device)
