"""Frequencies of rotary positions: the table that ``dsa_rope`` reads."""
from __future__ import annotations

import math
from dataclasses import dataclass
from fractions import Fraction

import torch

_SCALINGS = ("none", "linear", "ntk", "yarn")


@dataclass
class RopeTable:
    """Rotation frequencies on a device, built once per model.

    turns holds, per pair, the turns per position in units of 2^-64 (the bits
    of an unsigned 64-bit integer), so that a position times an entry, mod
    2^64, is the phase: exact for any position."""
    turns: torch.Tensor         # int64 [rot_dim / 2] (bits of uint64)
    rot_dim: int
    interleaved: bool
    amplitude: float            # factor of the rotated dims (YaRN's attention factor)

    @staticmethod
    def frequencies(rot_dim: int, theta: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                    original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0) -> list:
        """Radians per position of every pair j (64 bits).

        none    f_j = theta^(-2j / rot_dim)
        linear  f_j / factor (position interpolation)
        ntk     f_j with theta * factor^(rot_dim / (rot_dim - 2)): the lowest frequency is divided by
                factor, the highest is kept
        yarn    f_j r_j / factor + f_j (1 - r_j), r_j = clamp((j - low) / (high - low), 0, 1): pairs that turn
                more than beta_fast times over original_max positions keep their frequency, those
                that turn less than beta_slow times are interpolated
        """
        if not isinstance(rot_dim, int) or rot_dim < 2 or rot_dim % 2:
            raise ValueError(f"rot_dim={rot_dim}: expected an even number of at least 2")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling={scaling!r}: expected one of {_SCALINGS}")
        theta, factor = float(theta), float(factor)
        if not (math.isfinite(theta) and theta > 1.0 and math.isfinite(factor) and factor >= 1.0):
            raise ValueError(f"theta={theta}, factor={factor}: expected theta > 1 and factor >= 1")
        if scaling == "none" and factor != 1.0:
            raise ValueError("a factor needs a scaling")
        if scaling == "ntk":
            if rot_dim < 4:
                raise ValueError("ntk scaling needs rot_dim of at least 4")
            theta *= factor ** (rot_dim / (rot_dim - 2))
        f = [theta ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)]
        if scaling == "linear":
            f = [x / factor for x in f]
        if scaling == "yarn":
            if not (original_max >= 1 and beta_fast >= beta_slow > 0):
                raise ValueError("yarn scaling needs original_max >= 1 and beta_fast >= beta_slow > 0")

            def pair_of(turns):     # the (fractional) pair that turns this often over original_max positions
                return rot_dim * math.log(original_max / (turns * 2 * math.pi)) / (2 * math.log(theta))

            low = max(math.floor(pair_of(beta_fast)), 0)
            high = min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
            width = max(high - low, 0.001)
            ramp = [min(max((j - low) / width, 0.0), 1.0) for j in range(rot_dim // 2)]
            f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
        return f

    @staticmethod
    def build(rot_dim: int, theta: float = 10000.0, *, interleaved: bool = True, scaling: str = "none",
              factor: float = 1.0, original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
              amplitude: float | None = None, device="cuda") -> "RopeTable":
        """The table for `rot_dim` rotated dims (``frequencies`` says what each
        scaling means).  amplitude None: 0.1 ln(factor) + 1 for yarn, else 1."""
        f = RopeTable.frequencies(rot_dim, theta, scaling=scaling, factor=factor, original_max=original_max,
                                  beta_fast=beta_fast, beta_slow=beta_slow)
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
        if not math.isfinite(amplitude):
            raise ValueError(f"amplitude={amplitude}: expected a finite number")
        # a double's turns per position (off by 2^-52 of the angle), then rounded to units of 2^-64
        units = [round(Fraction(x / (2 * math.pi)) * 2 ** 64) % 2 ** 64 for x in f]
        signed = [u - 2 ** 64 if u >= 2 ** 63 else u for u in units]
        return RopeTable(torch.tensor(signed, dtype=torch.int64).to(device), rot_dim, bool(interleaved),
                         float(amplitude))
