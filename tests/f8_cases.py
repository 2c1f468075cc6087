"""Inputs and plain 64-bit forms of the 8-bit operators, shared by their GPU
tests (numpy, float64, written from the formulas)."""
from __future__ import annotations

import numpy as np
import torch

FORMAT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
IN_TYPE = {"e4m3": 3, "e5m2": 4}             # tcg_input
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def table(fmt: str) -> np.ndarray:
    """The values of all 256 codes."""
    man_bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    c = np.arange(256)
    sign = np.where(c & 128, -1.0, 1.0)
    e, m = (c & 127) >> man_bits, (c & ((1 << man_bits) - 1)) / 2.0 ** man_bits
    v = sign * np.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * 2.0 ** (e - bias))
    if fmt == "e4m3":
        v[(c & 127) == 127] = np.nan
    else:
        v[(c & 127) == 124] = np.inf * sign[(c & 127) == 124]
        v[(c & 127) > 124] = np.nan
    return v


def values(codes: torch.Tensor, fmt: str) -> np.ndarray:
    return table(fmt)[codes.cpu().view(torch.uint8).numpy()]


def nearest(v: np.ndarray, fmt: str) -> np.ndarray:
    """v rounded to the format's grid, ties to even."""
    man_bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = np.frexp(np.abs(v))
    step = 2.0 ** (np.maximum(e - 1, low) - man_bits)
    return np.round(v / step) * step


def codes(shape, fmt: str, seed: int, pad: int = 0):
    """Random codes in rows padded to 16 bytes and `pad` further octets of 16
    with NaN codes, on the device; and their values."""
    rng = np.random.default_rng(seed)
    v = np.clip(rng.standard_normal(shape) * LARGEST[fmt] / 3, -LARGEST[fmt], LARGEST[fmt])
    t = torch.from_numpy(v).float().to(FORMAT[fmt])
    ld = -(-shape[-1] // 16) * 16 + 16 * pad
    full = torch.full(tuple(shape[:-1]) + (ld,), 0x7f, dtype=torch.uint8)
    full[..., :shape[-1]] = t.view(torch.uint8)
    return full.cuda(), values(t, fmt)


def scales(shape, fmt: str, seed: int, size: float = 1.0, pad: int = 0):
    """Random positive scales (rows padded with NaN) on the device, and their values."""
    rng = np.random.default_rng(seed)
    s = ((0.5 + rng.random(shape)) * size * 3 / LARGEST[fmt]).astype(np.float32)
    full = np.full(tuple(shape[:-1]) + (shape[-1] + pad,), np.nan, np.float32)
    full[..., :shape[-1]] = s
    return torch.from_numpy(full).cuda(), s.astype(np.float64)


def spread(s: np.ndarray, rows: int, columns: int) -> np.ndarray:
    """Square scales to one for each element."""
    return np.repeat(np.repeat(s, BLOCK, -2)[..., :rows, :], BLOCK, -1)[..., :columns]


def along(s: np.ndarray, n: int) -> np.ndarray:
    """Scales [blocks][m] to one for each of n along the first dimension."""
    return np.repeat(s, BLOCK, 0)[:n]


def row_blocks(offsets: np.ndarray, R: int):
    """The scale row of each grouped row (-1: of no group)."""
    at = np.full(R, -1)
    for g in range(len(offsets) - 1):
        n = offsets[g + 1] - offsets[g]
        at[offsets[g]:offsets[g + 1]] = offsets[g] // BLOCK + g + np.arange(n) // BLOCK
    return at
