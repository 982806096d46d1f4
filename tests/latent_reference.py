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


def latent_values(kv: torch.Tensor, scales, fp8: bool) -> np.ndarray:
    """The latents [pages, 64, 512] that a pool (uint8 codes and float32 scales,
    or bf16) stands for."""
    if not fp8:
        return f64(kv).reshape(-1, PAGE, LATENT)
    return e4m3_values()[kv.cpu().numpy().reshape(-1, PAGE, LATENT)] * f64(scales).reshape(-1, PAGE, 1)


def attention(q, latents, tables, lengths, scale, selected=None, sinks=None):
    """(out, lse, tolerances): row b of q [rows, heads, 512] over the positions
    selected[b] (None: all) below lengths[b], whose pages tables[b] (None: the
    row has no valid table) names.

    The tolerances follow the library's roundings.  Scores: products of bf16
    values summed in float32, 512 of them and the scales: |error| <= 516 2^-24
    sum_d |q_d c_d| scale = E.  Probabilities: exp passes E on, and is itself,
    with its argument's rounding, within 2^-20; rounded to bf16 (2^-8 of the
    value at most) for the products, which are summed in float32 over n
    positions.  With A = sum_p p |c_p| / z
      |out error| <= A (2^-8 + 2 E + 2^-19 + n 2^-24) + 2^-8 |out|
      |lse error| <= E + 2^-20 + n 2^-24 + |lse| 2^-22
    The probabilities' roundings are independent from position to position, so
    the error's norm over the 512 values is also far below that sum: at most
    2^-8 sqrt(sum_p p^2 |c_p|^2) / z were all of them at their largest and
    orthogonal; twice that (and the rest as above, over the norms) is `norm`.
    """
    q = f64(q)
    rows, heads, _ = q.shape
    out, lse = np.zeros((rows, heads, LATENT)), np.full((rows, heads), -np.inf)
    tol, tol_lse, norm = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(lse)
    pages = latents.shape[0]
    for b in range(rows):
        L = int(lengths[b])
        at = np.arange(L) if selected is None else np.asarray(selected[b][: min(len(selected[b]), max(L, 0))], dtype=np.int64)
        at = at[(at >= 0) & (at < L)]
        page = np.full(len(at), -1) if tables[b] is None else np.asarray(tables[b])[at // PAGE]
        if ((page < 0) | (page >= pages)).any():
            out[b], lse[b] = np.nan, np.nan
            continue
        c = latents[page, at % PAGE]
        x = scale * (q[b] @ c.T)
        E = 516 * 2.0 ** -24 * abs(scale) * (np.abs(q[b]) @ np.abs(c).T).max(-1, initial=0.0)
        s = x if sinks is None else np.concatenate([x, f64(sinks)[:, None]], 1)
        if s.shape[1] == 0:
            continue
        top = s.max(-1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        e = np.exp(s - top)
        z = e.sum(-1, keepdims=True)
        p = np.divide(e, z, where=z > 0, out=np.zeros_like(e))[:, : len(at)]
        with np.errstate(divide="ignore"):
            lse[b] = (top + np.log(z))[:, 0]
        out[b] = p @ c
        n, A = len(at), p @ np.abs(c)
        other = (2 * E + 2.0 ** -19 + n * 2.0 ** -24)[:, None]
        tol[b] = A * (2.0 ** -8 + other) + 2.0 ** -8 * np.abs(out[b]) + 2.0 ** -126
        tol_lse[b] = E + 2.0 ** -20 + n * 2.0 ** -24 + np.where(np.isinf(lse[b]), 0, np.abs(lse[b])) * 2.0 ** -22
        spread = np.sqrt((p * p) @ (c * c).sum(-1))
        norm[b] = (2 * 2.0 ** -8 * spread + other[:, 0] * np.linalg.norm(A, axis=-1)
                   + 2.0 ** -8 * np.linalg.norm(out[b], axis=-1) + 2.0 ** -120)
    return out, lse, (tol, tol_lse, norm)


def assert_attention(got, got_lse, want) -> None:
    out, lse, (tol, tol_lse, norm) = want
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(out)), "NaN rows differ"
    live = ~np.isnan(out)
    d = np.abs(got - out)
    bad = live & (d > tol)
    assert not bad.any(), f"{bad.sum()} values off, worst {d[bad].max():.3e} at {np.argwhere(bad)[:3].tolist()}"
    rows = live[..., 0]
    far = np.linalg.norm(np.where(live, got - out, 0.0), axis=-1)
    assert (far <= norm)[rows].all(), f"norm of the error {far[rows].max():.3e}, ratio {(far / norm)[rows].max():.2f}"
    if got_lse is None:
        return
    got_lse = f64(got_lse)
    assert np.array_equal(np.isnan(got_lse), np.isnan(lse)) and np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
    fin = np.isfinite(lse)
    d = np.abs(np.where(fin, got_lse, 0) - np.where(fin, lse, 0))
    assert (d <= tol_lse).all(), f"lse off by {d.max():.3e}"
