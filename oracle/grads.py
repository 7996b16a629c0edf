"""The gradient-list operators, written out as plain numpy (TEST INFRASTRUCTURE ONLY).

* the global norm of a list of tensors (root of the sum of squares, or the
  largest magnitude), the clip scale and the overflow flag;
* the gradients times the scale, rounded to a type;
* micro-batches' gradients summed in fp32.

[codex] 6.3 and [llmnex] pitfall 1 (one norm and one coefficient for every
partition) as in ``zero3``; [codex] 6.2 (the gradient of a step is what its
reductions leave).  The pages have no list and no accumulation: their
definition is the header's, restated here with exact sums (``math.fsum``) and
extended precision.

Pinned by: ``math.hypot`` and torch's norms (the norm), ``zero3``'s finalize
step at loss scale 1, exact fractions (the accumulation) and torch's casts
(the clip).
"""

from __future__ import annotations

import math
from typing import Sequence, Tuple

import numpy as np

from .zero3 import from_f32, to_f32


def widened(bits: np.ndarray, dtype: str) -> np.ndarray:
    """A tensor's elements in fp32 (16-bit types as their bits)."""
    return np.asarray(bits, np.float32) if dtype == "fp32" else to_f32(bits, dtype)


def part(x: np.ndarray, kind: str) -> float:
    """What a tensor adds: the sum of its squares, or its largest magnitude."""
    x = np.abs(np.asarray(x, np.float32)).astype(np.float64)
    if np.isnan(x).any():
        return math.nan
    if np.isinf(x).any():
        return math.inf
    if kind == "inf":
        return float(x.max()) if x.size else 0.0
    return math.fsum((x * x).tolist())


def join(parts: Sequence[float], kind: str) -> float:
    parts = list(parts)
    if any(math.isnan(p) for p in parts):
        return math.nan
    if any(math.isinf(p) for p in parts):
        return math.inf
    return math.fsum(parts) if kind == "2" else max(parts, default=0.0)


def sums(tensors: Sequence[Tuple[np.ndarray, bool]], kind: str, peers: Sequence[float], rank: int) -> list:
    """``tensors``: (fp32 values, shared).  ``peers``: world + 1 entries, of which
    the own one and the last are replaced."""
    out = list(peers)
    each = [(part(x, kind), shared) for x, shared in tensors]
    out[rank] = join([p for p, shared in each if not shared], kind)
    out[-1] = join([p for p, shared in each if shared], kind)
    return out


def finalize(s: Sequence[float], kind: str, max_norm: float, loss_scale: float) -> Tuple[float, float, bool]:
    """(norm, scale before its rounding to fp32, not finite)."""
    total = join(s, kind)
    norm = (math.sqrt(total) if kind == "2" and not math.isnan(total) else total) / loss_scale
    if not math.isfinite(total):
        return norm, math.nan, True
    return norm, min(1.0, max_norm / (norm + 1e-6)) / loss_scale, False


def clip(x: np.ndarray, scale: float, dtype: str) -> np.ndarray:
    """fp32 values times the scale, as bits of a 16-bit type or as fp32."""
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        y = (np.asarray(x, np.float32) * np.float32(scale)).astype(np.float32)
    return y if dtype == "fp32" else from_f32(y, dtype)


def accumulate(acc: np.ndarray, x: np.ndarray, factor: float, first: bool) -> np.ndarray:
    """One fp32 rounding of factor * x (+ acc).  The product of two fp32 values has
    48 bits, so it is exact in the 64 of extended precision."""
    f = np.longdouble(np.float32(factor))
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        y = f * np.asarray(x, np.float32).astype(np.longdouble)
        if not first:
            y = y + np.asarray(acc, np.float32).astype(np.longdouble)
        return y.astype(np.float32)
