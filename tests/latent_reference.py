"""The latent cache's operators in float64, plainly, on the CPU (numpy), and the
inputs of their tests."""
from __future__ import annotations

import numpy as np
import torch

PAGE = 64
LATENT = 512


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def e4m3_values() -> np.ndarray:
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v = np.where(code & 127 == 127, np.nan, v)
    return np.where(code >= 128, -v, v)


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, norm=True, leading=False, halves=False):
    """(y, size): the normed and rotated vectors of x [..., D] (first dim:
    tokens), and |a| + |b| of the pair that each value was turned from (its own
    magnitude outside the rotated part), the scale of its rounding errors."""
    y = f64(x).copy()
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * f64(weight)
    size = np.abs(y)
    if inv_freq is not None and len(inv_freq):
        pairs = len(inv_freq)
        first = 0 if leading else y.shape[-1] - 2 * pairs
        j = np.arange(pairs)
        ia = first + (j if halves else 2 * j)
        ib = ia + (pairs if halves else 1)
        theta = f64(positions)[:, None] * f64(inv_freq)
        theta = theta.reshape((theta.shape[0],) + (1,) * (y.ndim - 2) + (pairs,))
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia] = a * np.cos(theta) - b * np.sin(theta)
        y[..., ib] = a * np.sin(theta) + b * np.cos(theta)
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


# Rounding errors of the float32 part, relative to `size` above: the sum of
# squares (8 fmas a lane, then at most 6 additions: 14 half steps, of which the
# root passes on half), mean, eps, root and reciprocal (4), the two products
# with r and the weight (2), sin and cos (the fraction of a turn, rounded at
# 2^-25 and so off by up to 2 pi 2^-26 = 1.6 half steps of 1 -- with their own
# error of up to 2 steps, 6 in all), the rotation's products and sum (3): under
# 24 half steps of 2^-24.
F32 = 24 * 2.0 ** -24


def assert_near_bf16(got: torch.Tensor, y: np.ndarray, size: np.ndarray) -> None:
    """Off by at most bf16's half step (2^-8 of the value, 2^-134 below its
    normal range) and the float32 part's."""
    err = F32 * size
    d = np.abs(f64(got) - y)
    bad = d > (np.abs(y) + err) * 2.0 ** -8 + err + 2.0 ** -134
    assert not bad.any(), f"{bad.sum()} values off, worst {d.max():.3e} at {np.argwhere(bad)[:3].tolist()}"


def assert_near_fp8(codes: np.ndarray, scales: np.ndarray, y: np.ndarray, size: np.ndarray) -> None:
    """codes uint8 [n, D], scales [n]: the scale is amax/448 up to the float32
    part's error, every value off by at most e4m3's half step (2^-4 of the
    value, 2^-10 scales below its normal range) and that error."""
    amax = np.abs(y).max(-1)
    err = F32 * size
    want = np.where(amax > 0, amax / 448, 1.0)
    assert (np.abs(scales - want) <= want * 2.0 ** -23 + err.max(-1) / 448).all()
    v = e4m3_values()[codes]
    assert np.isfinite(v).all()
    d = np.abs(v * scales[:, None].astype(np.float64) - y)
    slack = err + (np.abs(y) + err) * 2.0 ** -22  # the quotient's own rounding, and the scale's
    bad = d > np.maximum((np.abs(y) + slack) * 2.0 ** -4, scales[:, None] * 2.0 ** -10) * (1 + 2.0 ** -20) + slack
    assert not bad.any(), f"{bad.sum()} values off, worst {d.max():.3e}"


def inv_freq(pairs: int, base: float = 10000.0) -> torch.Tensor:
    return torch.tensor(base ** (-np.arange(pairs) / max(pairs, 1)), dtype=torch.float32)


def vectors(rng: np.random.Generator, shape, spread: float = 1.0) -> torch.Tensor:
    """bf16 vectors of several magnitudes, the first of them zero."""
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    if len(x) > 2:
        x[2] = 0.0
    return torch.from_numpy(x).to(torch.bfloat16)
