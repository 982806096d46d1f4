"""The operators of the cache of keys and values by head in float64, plainly, on
the CPU (numpy), and the inputs of their tests."""
from __future__ import annotations

import numpy as np
import torch

from latent_reference import e4m3_values, f64

PAGE = 64
BF16_MAX = 3.3895313892515355e38


def plan(cached, added, free, table, n):
    """(table, slots, positions, row_table, seqlens, starts, taken), request by request and token by token."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    taken, starts, rows = 0, [0], []
    for r, (c, a) in enumerate(zip(cached, added)):
        c, a = max(int(c), 0), max(int(a), 0)
        for j in range(-(-c // PAGE), min(-(-(c + a) // PAGE), width)):
            table[r, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + a):
            if len(rows) == n:
                break
            page = table[r, p // PAGE] if p // PAGE < width else -1
            rows.append((page * PAGE + p % PAGE if page >= 0 else -1, p, r, min(p + 1, 2 ** 31 - 1)))
        starts.append(starts[-1] + a)
    rows += [(-1, 0, 0, 0)] * (n - len(rows))
    return (table, *np.array(rows, dtype=np.int64).reshape(n, 4).T, np.array(starts), taken)


def values_of(pages, scales=None):
    """Stored blocks [..., 64, D] in float64: code times scale, or bf16 values."""
    if pages.dtype == torch.bfloat16:
        return f64(pages)
    codes = pages.contiguous().view(torch.uint8).cpu().numpy()
    return e4m3_values()[codes] * f64(scales)[..., None]


def table_of(table, row_table, b):
    """Row b's page table, or None where its index is out of range."""
    if row_table is None:
        return table[b if len(table) > 1 else 0]
    t = int(row_table[b])
    return table[t] if 0 <= t < len(table) else None


def bounds(keys, table, first, lengths, old, num_pages, row_table=None):
    """Bounds [pages, heads, 2, D] of float64 keys [pages, heads, 64, D], unrounded;
    pages that no row names as they are in `old`."""
    out = np.array(old, dtype=np.float64)
    for b, length in enumerate(lengths):
        tab = table_of(table, row_table, b)
        if tab is None:
            continue
        length = min(max(int(length), 0), len(tab) * PAGE)
        for j in range(max(int(first[b]), 0) // PAGE, -(-length // PAGE)):
            page = int(tab[j])
            if not 0 <= page < num_pages:
                continue
            k = keys[page, :, : min(length - j * PAGE, PAGE)]
            none = np.isnan(k).all(1)
            lo = np.where(none, 0.0, np.fmin.reduce(k, 1))
            hi = np.where(none, 0.0, np.fmax.reduce(k, 1))
            out[page, :, 0], out[page, :, 1] = lo, hi
    return np.clip(out, -BF16_MAX, BF16_MAX)


def scores(q, near, table, lengths, first_pages, last_pages, num_pages, row_table=None):
    """(scores [rows, heads, width], size: the sums of the products' amounts, counts)."""
    rows, heads = len(q), near.shape[1]
    width = table.shape[1]
    group = q.shape[1] // heads
    out = np.full((rows, heads, width), -np.inf)
    size = np.zeros_like(out)
    counts = np.zeros((rows, heads), dtype=np.int64)
    for b, length in enumerate(lengths):
        tab = table_of(table, row_table, b)
        count = min(-(-max(int(length), 0) // PAGE), width)
        counts[b] = count
        for j in range(count):
            page = -1 if tab is None else int(tab[j])
            if j < first_pages or j >= count - last_pages:
                out[b, :, j] = np.inf
            elif not 0 <= page < num_pages:
                out[b, :, j] = np.nan
            else:
                x = q[b].reshape(heads, group, -1)
                lo, hi = near[page, :, None, 0], near[page, :, None, 1]
                best = np.maximum(x * lo, x * hi)
                out[b, :, j] = best.sum(-1).max(-1)
                size[b, :, j] = np.abs(best).sum(-1).max(-1)
    return out, size, counts


def attention(q, keys, values, table, selected, lengths, scale, num_pages, sinks=None, row_table=None):
    """(out, lse, size, far) for float64 q [rows, heads, D] and pools [pages, kv heads,
    64, D]: size is sum_p P_p |v_p|, far the largest sum of |scale q_d k_d| of a
    head's positions, the scales of their rounding errors."""
    rows, heads, dim = q.shape
    kv_heads = keys.shape[1]
    group = heads // kv_heads
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, far = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    for b in range(rows):
        tab = table_of(table, row_table, b)
        width = table.shape[1]
        length = min(max(int(lengths[b]), 0), width * PAGE)
        count = -(-length // PAGE)
        for h in range(kv_heads):
            listed = list(range(count)) if selected is None else [int(j) for j in selected[b, h][: min(selected.shape[2], count)]]
            listed = [j for j in listed if 0 <= j < count]
            i = slice(h * group, (h + 1) * group)
            if any(tab is None or not 0 <= int(tab[j]) < num_pages for j in listed):
                out[b, i] = lse[b, i] = np.nan
                continue
            at = [(int(tab[j]), min(length - j * PAGE, PAGE)) for j in listed]
            k = np.concatenate([keys[p, h, :n] for p, n in at] + [np.zeros((0, dim))])
            v = np.concatenate([values[p, h, :n] for p, n in at] + [np.zeros((0, dim))])
            x = scale * q[b, i] @ k.T
            every = x if sinks is None else np.concatenate((x, sinks[i, None]), 1)
            if every.shape[1] == 0:
                continue
            top = every.max(1)
            lse[b, i] = top + np.log(np.exp(every - top[:, None]).sum(1))
            p = np.exp(x - lse[b, i, None])
            out[b, i], size[b, i] = p @ v, p @ np.abs(v)
            if len(k):
                far[b, i] = abs(scale) * (np.abs(q[b, i]) @ np.abs(k).T).max(1)
    return out, lse, size, far


def assert_near_attention(out, lse, want, dim, positions):
    """Off by at most: bf16's half step (2^-8) for each probability and for the
    result; of a score, the float32 sums of `dim` products (dim + 4 half steps of
    2^-24 of the products' amounts, which bound the score too, its product with
    scale * log2(e) and the difference to the reference among them), the
    exponential's step of 2^-23 and one more of a rescaling; of the denominator,
    a rounding each for what a lane adds up of the positions and 64 of pieces and
    waves."""
    y, log, size, far = want
    got, got_log = f64(out), f64(lse)
    bad = np.isnan(log)
    assert np.isnan(got[bad]).all() and np.isnan(got_log[bad]).all()
    empty = np.isneginf(log)
    assert (got[empty] == 0).all() and np.isneginf(got_log[empty]).all()
    fine = ~bad & ~empty
    one = far * (dim + 8) * 2.0 ** -24 + 2.0 ** -22
    total = (positions / 4 + 64) * 2.0 ** -24
    err = size * (2.0 ** -8 + 2 * one + total)[..., None] * (1 + 2.0 ** -7) + np.abs(y) * 2.0 ** -8 + 2.0 ** -133
    d = np.abs(got - y)[fine]
    assert (d <= err[fine]).all(), f"{(d > err[fine]).sum()} of {d.size} off, worst {d.max():.3e}, {np.argwhere(np.abs(got - y) > err)[:4].tolist()}"
    far_log = one + total + np.abs(log) * 2.0 ** -22
    dl = np.abs(got_log - log)[fine]
    assert (dl <= far_log[fine]).all(), f"lse off by {dl.max():.3e}"


def make_pools(gen, pages, kv_heads, dim, fp8, layout="fused", device="cuda"):
    """(k_pages, v_pages, scales): views of the pool's layout: "fused": each block with
    its scales behind it, keys and values of a page side by side; "heads": head
    major, all keys before all values; "apart": four tensors."""
    shape = (pages, kv_heads, PAGE, dim)

    def block():
        x = torch.randn(shape, generator=gen)
        return (x * 110).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)

    def scale():
        return (torch.rand(shape[:3], generator=gen) + 0.6) / 110

    k, v = block(), block()
    ks, vs = (scale(), scale()) if fp8 else (None, None)
    if layout == "apart":
        place = lambda x: None if x is None else x.to(device)  # noqa: E731
        return place(k), place(v), () if not fp8 else (place(ks), place(vs))
    if layout == "heads":
        whole = torch.stack((k.view(torch.uint8 if fp8 else torch.bfloat16), v.view(torch.uint8 if fp8 else torch.bfloat16)))
        whole = whole.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        kk, vv = whole[0], whole[1]
        if not fp8:
            return kk, vv, ()
        both = torch.stack((ks, vs)).transpose(1, 2).contiguous().to(device).transpose(1, 2)
        return kk.view(torch.float8_e4m3fn), vv.view(torch.float8_e4m3fn), (both[0], both[1])
    if not fp8:
        whole = torch.stack((k, v), 1).to(device)
        return whole[:, 0], whole[:, 1], ()
    pool = torch.empty((pages, 2, kv_heads, PAGE * (dim + 4)), dtype=torch.uint8)
    for i, (x, s) in enumerate(((k, ks), (v, vs))):
        pool[:, i, :, : PAGE * dim] = x.view(torch.uint8).flatten(2)
        pool[:, i, :, PAGE * dim :] = s.view(torch.uint8).flatten(2)
    pool = pool.to(device)
    codes = pool[..., : PAGE * dim].unflatten(-1, (PAGE, dim))
    scales = pool[..., PAGE * dim :].view(torch.float32)
    return codes[:, 0], codes[:, 1], (scales[:, 0], scales[:, 1])
