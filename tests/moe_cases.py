"""Inputs and plain 64-bit forms of the mixture-of-experts operators, shared by
their GPU tests (numpy, float64, written from the formulas)."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DTYPE = {"f32": 0, "f16": 1, "bf16": 2}        # tcg_dtype
IN_TYPE = {"f16": 0, "bf16": 1}                # tcg_input
U_OUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # unit roundoff of the stored type
#: half the smallest subnormal: absolute rounding of values near zero
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def order(expert: np.ndarray, E: int):
    """offsets, position, source of [T][topk] expert ids (numpy int32)."""
    flat = expert.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    source = np.argsort(key, kind="stable")
    rank = np.empty_like(source)
    rank[source] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1))])[:E + 1]
    position = np.where(key < E, rank, -1 - rank).reshape(expert.shape)
    return offsets.astype(np.int32), position.astype(np.int32), source.astype(np.int32)


def rows(shape, dtype: str, seed: int, pad: int = 0, scale: float = 1.0):
    """A device tensor of `shape` inside rows padded by `pad` NaN elements, and
    its values as float64."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.float32).to(TORCH[dtype])
    full = torch.full(tuple(shape[:-1]) + (shape[-1] + pad,), float("nan"), dtype=TORCH[dtype])
    full[..., :shape[-1]] = x
    return full.cuda(), x.double().numpy()


def close(got: np.ndarray, ref: np.ndarray, S: np.ndarray, tau: float, out: str, what=""):
    """|got - ref| <= tau S (accumulation) + one rounding to the stored type."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bound = tau * S + U_OUT[out] * (np.abs(ref) + tau * S) + TINY[out]
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), got.size, np.argwhere(bad)[:4].tolist(),
                           got[bad][:4], ref[bad][:4], bound[bad][:4])


def group_offsets(sizes, first: int = 0):
    return (first + np.concatenate([[0], np.cumsum(sizes)])).astype(np.int32)


def to_host(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()
