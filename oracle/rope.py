"""CPU fp64 oracle for rotary positions — test infrastructure only, like the rest of ``oracle/``.

A token at position p multiplies pair i of every head's row, read as the
complex number a_i + i b_i, by mag * e^{i p f_i}; the pair is columns
(i, r + i) (half layout) or (2i, 2i + 1) (interleaved) of the first 2r, and the
columns from 2r on pass unchanged.  The map is linear; its transpose, the
gradient, is the same with -f_i.
"""
from __future__ import annotations

import math

import torch

from .attention import F64, as_f64


def inv_freq(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, fast_turns=32.0, slow_turns=1.0):
    """(inverse frequencies [rot_dim / 2], magnitude) by the formulas of ``fa_rope_scaling`` in fa.h."""
    n = rot_dim // 2
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = [1.0 / base ** (2 * i / rot_dim) for i in range(n)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "parts":
        return torch.tensor(f, dtype=F64), 1.0
    # index at which a pair makes `turns` turns in original_len positions
    at = lambda turns: rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(fast_turns)), 0), min(math.ceil(at(slow_turns)), rot_dim - 1)
    if at(slow_turns) < 0:  # every pair turns less than slow_turns times
        lo = hi - 1
    elif lo >= hi:  # a ramp of no width, or one past the last pair
        hi = lo + 0.001
    keep = [1 - min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(n)]
    return (torch.tensor([x * k + x / factor * (1 - k) for x, k in zip(f, keep)], dtype=F64),
            0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


def rotate(x, positions, freqs, interleaved=False, magnitude=1.0, back=False):
    """x [T, heads, D] rotated by its tokens' positions (by minus them with ``back``)."""
    x = as_f64(x)
    r = len(freqs)
    ang = torch.outer(torch.as_tensor(positions).to(F64), as_f64(freqs))
    w = torch.polar(torch.full_like(ang, magnitude), -ang if back else ang)[:, None, :]
    y = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * r:2], x[..., 1:2 * r:2]) * w
        y[..., 0:2 * r:2], y[..., 1:2 * r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r], x[..., r:2 * r]) * w
        y[..., :r], y[..., r:2 * r] = z.real, z.imag
    return y
