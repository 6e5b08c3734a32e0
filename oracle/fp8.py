"""CPU oracle for the 8-bit products and quantisers -- TEST INFRASTRUCTURE ONLY.

Works on numpy arrays of the codes' values (float64) and of the scales; nothing
here imports the product package.  Products are plain sums in binary64.  The
quantiser's codes and scales are defined by fp32 operations (two divisions and
one product, round to nearest) and are reproduced exactly with numpy float32.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MAXIMA = {"e4m3": 448.0, "e5m2": 57344.0}
# (mantissa bits, exponent of the smallest normal number)
FORMATS = {"e4m3": (3, -6), "e5m2": (2, -14)}


def spread(s, rows: int, cols: int, by: str) -> np.ndarray:
    """One scale for each element from the scales of blocks (by "row") or tiles."""
    s = np.repeat(np.asarray(s, dtype=np.float64), BLOCK, axis=-1)[..., :cols]
    return np.repeat(s, BLOCK, axis=-2)[..., :rows, :] if by == "tile" else s


def values(q, s, by: str) -> np.ndarray:
    q = np.asarray(q, dtype=np.float64)
    return q * spread(s, q.shape[-2], q.shape[-1], by)


def product(qa, sa, qb, sb, by: str) -> tuple[np.ndarray, np.ndarray]:
    """(a b^T, |a| |b|^T) of the values."""
    a, b = values(qa, sa, "row"), values(qb, sb, by)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def by_experts(qa, sa, qb, sb, offsets) -> tuple[np.ndarray, np.ndarray]:
    """Rows offsets[e] .. offsets[e+1] - 1 against expert e's matrix; NaN where no expert is."""
    out = np.full((len(qa), qb.shape[1]), np.nan)
    size = np.zeros_like(out)
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        out[r], size[r] = product(qa[r], np.asarray(sa)[r], qb[e], sb[e], "tile")
    return out, size


def first_blocks(offsets) -> list[int]:
    """The first block of 128 of each expert's rows, and one past the last."""
    at = [0]
    for e in range(len(offsets) - 1):
        at.append(at[-1] + -(-(offsets[e + 1] - offsets[e]) // BLOCK))
    return at


def by_depth(qa, sa, qb, sb, offsets) -> tuple[np.ndarray, np.ndarray]:
    a, b = values(qa, sa, "row"), values(qb, sb, "row")
    at = first_blocks(offsets)
    parts = [slice(at[e] * BLOCK, at[e + 1] * BLOCK) for e in range(len(at) - 1)]
    return (np.stack([a[:, p] @ b[:, p].T for p in parts]),
            np.stack([np.abs(a[:, p]) @ np.abs(b[:, p]).T for p in parts]))


def round8(v: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest values of the format, ties to even, saturating; exact for float32 v."""
    mantissa, low = FORMATS[fmt]
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    with np.errstate(invalid="ignore"):
        step = np.ldexp(1.0, np.maximum(e - 1, low) - mantissa)
        return np.clip(np.rint(v / step) * step, -MAXIMA[fmt], MAXIMA[fmt])


def block_codes(x: np.ndarray, fmt: str) -> tuple[np.ndarray, np.float32]:
    """(codes' values, scale) of one block of numbers (float32)."""
    top = np.float32(MAXIMA[fmt])
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.maximum(np.max(np.abs(x)), top * np.float32(2.0 ** -126)) if x.size else \
            top * np.float32(2.0 ** -126)
        scale, factor = np.float32(amax / top), np.float32(top / amax)
        return round8((x * factor).astype(np.float32), fmt), scale


def quantise_rows(x: np.ndarray, fmt: str) -> tuple[np.ndarray, np.ndarray]:
    r, k = x.shape
    q, s = np.zeros((r, k)), np.zeros((r, -(-k // BLOCK)), dtype=np.float32)
    for i in range(r):
        for b in range(s.shape[1]):
            c = slice(b * BLOCK, (b + 1) * BLOCK)
            q[i, c], s[i, b] = block_codes(x[i, c], fmt)
    return q, s


def quantise_tiles(x: np.ndarray, fmt: str) -> tuple[np.ndarray, np.ndarray]:
    n, k = x.shape
    q, s = np.zeros((n, k)), np.zeros((-(-n // BLOCK), -(-k // BLOCK)), dtype=np.float32)
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            t = (slice(i * BLOCK, (i + 1) * BLOCK), slice(b * BLOCK, (b + 1) * BLOCK))
            q[t], s[i, b] = block_codes(x[t], fmt)
    return q, s


def quantise_columns(x: np.ndarray, offsets, fmt: str) -> tuple[np.ndarray, np.ndarray]:
    """Transposed, blocks along the rows; every expert's rows start a new block."""
    r, c = x.shape
    blocks = r // BLOCK + max(len(offsets) - 1, 1)
    q = np.zeros((c, blocks * BLOCK))
    s = np.full((c, blocks), block_codes(np.zeros(1), fmt)[1], dtype=np.float32)
    at = 0
    for e in range(len(offsets) - 1):
        for i in range(offsets[e], offsets[e + 1], BLOCK):
            rows = x[i:min(i + BLOCK, offsets[e + 1])]
            for j in range(c):
                q[j, at * BLOCK:at * BLOCK + len(rows)], s[j, at] = block_codes(rows[:, j], fmt)
            at += 1
    return q, s
