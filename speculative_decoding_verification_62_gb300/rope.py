"""Rotary frequencies for the cache append (host logic, float64, no GPU work).

Pair j of a head turns by position * f_j radians.  ``frequencies`` gives f_j, for
contexts longer than the model was trained on with one of three scalings:

* ``linear``: positions divided by the factor (f_j / factor);
* ``ntk``: the base raised so that the lowest frequency is divided by the factor and
  the highest stays, base * factor ** (rot_dim / (rot_dim - 2));
* ``by_parts``: pairs that turn at least ``beta_fast`` times within the trained context
  stay, pairs that turn at most ``beta_slow`` times are divided by the factor, and a linear ramp
  over the pairs between (by their index) joins the two.  ``by_parts_scale`` gives the
  factor on cos and sin that goes with it.

``fixed_point`` turns them into what the kernel takes: turns a position as whole
multiples of 2^-64, so that position * f_j modulo one turn is exact integer arithmetic.
"""
from __future__ import annotations

import math

import torch


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                trained_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> torch.Tensor:
    """float64 [rot_dim / 2]: radians a position of each pair."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must exceed 1 and factor be at least 1")
    n = rot_dim // 2
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs two pairs")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = torch.tensor(base, dtype=torch.float64) ** (-torch.arange(n, dtype=torch.float64) / n)
    if scaling in ("none", "ntk"):
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        if trained_len < 1 or not beta_fast > beta_slow > 0.0:
            raise ValueError("by_parts needs trained_len and beta_fast > beta_slow > 0")

        def pair_of(turns):  # index of the pair that turns so often within trained_len
            return n * math.log(trained_len / (2.0 * math.pi * turns)) / math.log(base)

        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = math.ceil(pair_of(beta_slow))  # behind the last pair where that one turns more often
        ramp = ((torch.arange(n, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / factor * ramp
    raise ValueError(f"unknown scaling {scaling!r}")


def by_parts_scale(factor: float) -> float:
    """The factor on cos and sin that goes with by_parts: 0.1 ln(factor) + 1."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def _pi(bits: int) -> int:
    """floor(pi 2^bits) up to the last few bits, by Machin's formula."""
    def atan_inverse(x):
        term, total, k = (1 << (bits + 16)) // x, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= x * x
            k += 2
        return total
    return (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 16


def fixed_point(freq) -> torch.Tensor:
    """int64 [n]: freq (radians a position) in turns, as whole multiples of 2^-64 modulo
    one turn, rounded once from the exact quotient by 2 pi."""
    f = torch.as_tensor(freq, dtype=torch.float64).cpu()
    if f.dim() != 1 or not bool(torch.isfinite(f).all()):
        raise ValueError("freq must be one dimension of finite numbers")
    two_pi = 2 * _pi(192)
    out = []
    for x in f.tolist():
        n, d = x.as_integer_ratio()
        turns = ((n << (64 + 192 + 1)) // (d * two_pi) + 1) >> 1
        turns &= (1 << 64) - 1
        out.append(turns - (1 << 64) if turns >> 63 else turns)
    return torch.tensor(out, dtype=torch.int64)


__all__ = ["frequencies", "by_parts_scale", "fixed_point"]
