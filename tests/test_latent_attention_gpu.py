"""Attention over paged latents on the GPU against float64."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from latent_reference import LATENT, PAGE, assert_attention, attention, f64, inv_freq, latent_values

pytestmark = pytest.mark.gpu

SCALE = LATENT ** -0.5
PAGE8 = PAGE * (LATENT + 4)


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


class Cache:
    """A pool of latents: codes (uint8 [pages, 64, 512]) and scales, or bf16, as
    tensors on the CPU, and the device copy in one of the layouts."""

    def __init__(self, rng, pages, fp8, layout="fused"):
        self.fp8, self.pages = fp8, pages
        if fp8:
            codes = rng.integers(0, 256, (pages, PAGE, LATENT), dtype=np.uint8)
            codes[(codes & 127) == 127] = 0x30
            # magnitudes that a normed vector has: most codes of a uniform draw are tiny
            x = torch.from_numpy(rng.standard_normal((pages, PAGE, LATENT)).astype(np.float32) * 110)
            mixed = torch.from_numpy(rng.random((pages, PAGE, 1)) < 0.1)
            self.kv = torch.where(mixed, torch.from_numpy(codes), x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            self.scales = torch.from_numpy(((rng.random((pages, PAGE)) + 0.5) / 110).astype(np.float32))
            self.scales = torch.where(mixed[..., 0], self.scales * 0.3, self.scales)
        else:
            self.kv = torch.from_numpy(rng.standard_normal((pages, PAGE, LATENT)).astype(np.float32)).to(torch.bfloat16)
            self.scales = None
        self.layout = layout

    def poison(self, keep):
        """Every slot but those of the set `keep` holds NaN."""
        other = np.ones(self.pages * PAGE, bool)
        other[list(keep)] = False
        other = torch.from_numpy(other.reshape(self.pages, PAGE))
        if self.fp8:
            self.kv[other] = 0x7F
            self.scales[other] = float("nan")
        else:
            self.kv[other] = float("nan")

    def device(self):
        kv = self.kv.cuda()
        if not self.fp8:
            if self.layout == "padded":
                wide = torch.full((self.pages, PAGE * LATENT + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
                wide[:, : PAGE * LATENT] = kv.reshape(self.pages, -1)
                return (wide,), dict(kv_page_stride=2 * (PAGE * LATENT + 40))
            return (kv,), {}
        if self.layout == "fused":
            fused = torch.empty((self.pages, PAGE8), dtype=torch.uint8, device="cuda")
            fused[:, : PAGE * LATENT] = kv.reshape(self.pages, -1)
            fused[:, PAGE * LATENT:] = self.scales.cuda().view(torch.uint8)
            return (fused, fused.data_ptr() + PAGE * LATENT), {}
        scales = torch.full((self.pages, 70), float("nan"), device="cuda")
        scales[:, :PAGE] = self.scales.cuda()
        return (kv, scales), dict(kv_page_stride=PAGE * LATENT, kscale_page_stride=280)

    def values(self):
        return latent_values(self.kv, self.scales, self.fp8)


def queries(rng, rows, heads, spread=1.5):
    return torch.from_numpy(rng.standard_normal((rows, heads, LATENT)) * spread).to(torch.bfloat16)


def call(lib, cache, q, table, selected, lengths, *, sinks=None, row_table=None, lse=True, workspace=None, stream=None,
         scale=SCALE, num_pages=None, **kw):
    pool, strides = cache.device() if isinstance(cache, Cache) else cache
    fn = lib.idx_latent_attention_fp8 if len(pool) == 2 else lib.idx_latent_attention_bf16
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    logs = torch.full(q.shape[:2], 9.0, device="cuda") if lse else None
    to = lambda t: None if t is None else t.cuda()  # noqa: E731
    fn(q.cuda(), *pool, to(table), to(selected), to(lengths), out, logs, scale=scale,
       num_pages=cache.pages if num_pages is None else num_pages, sinks=to(sinks), row_table=to(row_table), workspace=workspace,
       stream=stream, **strides, **kw)
    torch.cuda.synchronize()
    return out, logs


def some(rng, length, k, total):
    """A top-k list of `total` entries: min(k, length) positions in ascending
    order, -1 behind them."""
    picked = np.sort(rng.permutation(max(length, 1))[: min(k, max(length, 0))])
    return np.concatenate([picked, np.full(total - len(picked), -1)]).astype(np.int32)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows,heads,width,k,layout", [
    (1, 1, 1, 1, "fused"),
    (1, 64, 3, 64, "fused"),
    (2, 16, 2, 65, "split"),
    (3, 17, 5, 127, "padded"),
    (5, 33, 9, 300, "fused"),
    (4, 128, 12, 513, "split"),
    (40, 64, 20, 700, "fused"),
    (1, 100, 64, 2048, "padded"),
    (300, 40, 6, 129, "fused"),
    (1100, 8, 2, 70, "split"),
    (7, 64, 4, 1000, "fused"),      # lists longer than any row
])
def test_selected(lib, fp8, rows, heads, width, k, layout):
    """Lists of every length, each row its own pages; nothing that no list names
    is read (all else holds NaN)."""
    rng = np.random.default_rng(rows * 7 + heads + k)
    announce(f"selected fp8={fp8} rows={rows} heads={heads} width={width} k={k} {layout}")
    pages = min(rows * width, 400)
    table = np.stack([rng.permutation(pages)[:width] for _ in range(rows)]).astype(np.int32)
    lengths = rng.integers(1, width * PAGE + 1, rows)
    for b, v in enumerate([width * PAGE, 0, 1, -5, width * PAGE + 99, 63]):
        if b + 1 < rows:
            lengths[b] = v
    clamped = np.clip(lengths, 0, width * PAGE)
    selected = np.stack([some(rng, int(L), k, k) for L in clamped])
    for b in range(0, rows, 3):  # entries to skip inside a list: padding, past the row, past the table
        if clamped[b] > 8 and k > 8:
            selected[b, [1, 4]] = [-1, width * PAGE + 7]
            selected[b, 6] = min(clamped[b], 2 ** 31 - 1)
    sinks = torch.from_numpy(rng.standard_normal(heads).astype(np.float32) * 2) if rows % 2 else None
    cache = Cache(rng, pages, fp8, layout)
    used = set()
    for b in range(rows):
        at = selected[b][: min(k, clamped[b])].astype(np.int64)
        at = at[(at >= 0) & (at < clamped[b])]
        used |= set((table[b][at // PAGE] * PAGE + at % PAGE).tolist())
    cache.poison(used)
    table_dead = table.copy()
    for b in range(rows):  # table entries past a row's length are never read
        table_dead[b, (clamped[b] + PAGE - 1) // PAGE:] = -7
    q = queries(rng, rows, heads)
    want = attention(q, np.nan_to_num(cache.values()), table, clamped, SCALE, selected, sinks)
    out, lse = call(lib, cache, q, torch.from_numpy(table_dead), torch.from_numpy(selected),
                    torch.from_numpy(lengths.astype(np.int32)), sinks=sinks)
    assert_attention(out, lse, want)
    again, _ = call(lib, cache, q, torch.from_numpy(table_dead), torch.from_numpy(selected),
                    torch.from_numpy(lengths.astype(np.int32)), sinks=sinks, lse=False)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows,heads,width,lengths", [
    (1, 64, 1, [1]),
    (1, 5, 1, [64]),
    (3, 32, 2, [65, 0, 128]),
    (6, 48, 7, [447, 448, 1, 63, 64, 65]),
    (2, 128, 130, [8320, 4097]),
    (1, 16, 600, [38400]),
    (520, 3, 3, None),
])
def test_every_position(lib, fp8, rows, heads, width, lengths):
    rng = np.random.default_rng(width)
    announce(f"every position fp8={fp8} rows={rows} heads={heads} width={width}")
    pages = min(rows * width, 700)
    table = np.stack([rng.permutation(pages)[:width] for _ in range(rows)]).astype(np.int32)
    lengths = np.array(lengths) if lengths else rng.integers(0, width * PAGE + 1, rows)
    cache = Cache(rng, pages, fp8)
    used = {int(table[b][p // PAGE]) * PAGE + p % PAGE for b in range(rows) for p in range(lengths[b])}
    cache.poison(used)
    q = queries(rng, rows, heads)
    want = attention(q, np.nan_to_num(cache.values()), table, lengths, SCALE)
    out, lse = call(lib, cache, q, torch.from_numpy(table), None, torch.from_numpy(lengths.astype(np.int32)))
    assert_attention(out, lse, want)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("width", [3, 70])
def test_one_position_takes_all(lib, fp8, width):
    """A query along one latent picks it: every place of a tile, split and page,
    and every value of the output."""
    rng = np.random.default_rng(1)
    total = width * PAGE
    picks = np.unique(np.concatenate([np.arange(0, 130), total - 1 - np.arange(70), rng.integers(0, total, 60)]))
    cache = Cache(rng, width, fp8)
    values = cache.values().reshape(-1, LATENT)
    order = rng.permutation(width).astype(np.int32)
    rows = len(picks)
    q = torch.from_numpy(values[order[picks // PAGE] * PAGE + picks % PAGE][:, None].repeat(3, 1)).to(torch.bfloat16)
    lengths = torch.full((rows,), total, dtype=torch.int32)
    out, lse = call(lib, cache, q, torch.from_numpy(order[None]), None, lengths, scale=1.0)
    assert_attention(out, lse, attention(q, cache.values(), [order] * rows, lengths.numpy(), 1.0))


def test_shared_tables_and_row_tables(lib):
    """A prefill of one request (one table for all rows), and of three with a
    row table; a table index outside the tables makes its row NaN."""
    rng = np.random.default_rng(2)
    rows, heads, width, k = 70, 24, 6, 100
    cache = Cache(rng, 20, True)
    tables = np.stack([rng.permutation(20)[:width] for _ in range(3)]).astype(np.int32)
    wide = torch.full((3, width + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, :width] = torch.from_numpy(tables)
    lengths = -(-width * PAGE * (np.arange(rows) + 1) // rows)
    selected = torch.from_numpy(np.stack([some(rng, int(n), k, k) for n in lengths]))
    q = queries(rng, rows, heads)
    sl = torch.from_numpy(lengths.astype(np.int32))
    out, lse = call(lib, cache, q, torch.from_numpy(tables[:1]), selected, sl)
    assert_attention(out, lse, attention(q, cache.values(), [tables[0]] * rows, lengths, SCALE, selected.numpy()))
    which = rng.integers(0, 3, rows).astype(np.int32)
    which[5], which[40] = 3, -1
    picked = [tables[t] if 0 <= t < 3 else None for t in which]
    want = attention(q, cache.values(), picked, lengths, SCALE, selected.numpy())
    assert np.isnan(want[0][5]).all() and np.isnan(want[0][40]).all()
    out, lse = call(lib, cache, q, wide[:, :width], selected, sl, row_table=torch.from_numpy(which))
    assert_attention(out, lse, want)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows", [3, 600])
def test_bad_pages(lib, fp8, rows):
    """A selected position whose page id lies outside the pool makes its row NaN,
    and no other; the page is not read."""
    rng = np.random.default_rng(4)
    width, k, heads = 5, 90, 20
    cache = Cache(rng, 30, fp8)
    table = np.stack([rng.permutation(30)[:width] for _ in range(rows)]).astype(np.int32)
    lengths = np.full(rows, width * PAGE)
    selected = np.stack([some(rng, width * PAGE, k, k) for _ in range(rows)])
    table[1, 2] = 30          # the first id past the pool
    table[2, 0] = -2 ** 31
    selected[0] = np.where(selected[0] // PAGE == 3, -1, selected[0])
    table[0, 3] = 2 ** 31 - 1  # not selected: no harm
    want = attention(queries(np.random.default_rng(9), rows, heads), cache.values(), table, lengths, SCALE, selected)
    assert np.isnan(want[0][1]).all() and np.isnan(want[0][2]).all() and not np.isnan(want[0][0]).any()
    q = queries(np.random.default_rng(9), rows, heads)
    out, lse = call(lib, cache, q, torch.from_numpy(table), torch.from_numpy(selected), torch.from_numpy(lengths.astype(np.int32)))
    assert_attention(out, lse, want)


@pytest.mark.parametrize("rows", [2, 530])
def test_sinks(lib, rows):
    """Sinks far below and far above the scores, none (-inf), and rows with
    nothing but a sink."""
    rng = np.random.default_rng(5)
    heads, width = 6, 4
    cache = Cache(rng, 8, True)
    table = np.stack([rng.permutation(8)[:width] for _ in range(rows)]).astype(np.int32)
    lengths = rng.integers(0, width * PAGE + 1, rows)
    lengths[1] = 0
    sinks = torch.tensor([-200.0, 200.0, -np.inf, 0.0, 3.5, 90.0])
    q = queries(rng, rows, heads)
    out, lse = call(lib, cache, q, torch.from_numpy(table), None, torch.from_numpy(lengths.astype(np.int32)), sinks=sinks)
    assert_attention(out, lse, attention(q, cache.values(), table, lengths, SCALE, None, sinks))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_of_the_scores(lib, scale):
    """No scores, negative ones, and a range of hundreds: the running maximum
    moves from tile to tile."""
    rng = np.random.default_rng(6)
    rows, heads, width = 4, 40, 30
    cache = Cache(rng, 40, False)
    grow = torch.linspace(0.05, 3.0, 40)[:, None, None]
    cache.kv = (cache.kv.float() * grow).to(torch.bfloat16)
    table = np.stack([np.sort(rng.permutation(40)[:width]) for _ in range(rows)]).astype(np.int32)
    lengths = np.array([1920, 1919, 700, 64])
    q = queries(rng, rows, heads, 1.0)
    out, lse = call(lib, cache, q, torch.from_numpy(table), None, torch.from_numpy(lengths.astype(np.int32)), scale=scale)
    assert_attention(out, lse, attention(q, cache.values(), table, lengths, scale))


def test_a_position_twice_counts_twice(lib):
    rng = np.random.default_rng(7)
    cache = Cache(rng, 2, True)
    selected = torch.tensor([[5, 5, 5, 70, 2, -1, 70]], dtype=torch.int32)
    q = queries(rng, 1, 4)
    table = np.array([[1, 0]], dtype=np.int32)
    out, lse = call(lib, cache, q, torch.from_numpy(table), selected, torch.tensor([100], dtype=torch.int32))
    assert_attention(out, lse, attention(q, cache.values(), table, [100], SCALE, selected.numpy()))


@pytest.mark.parametrize("fp8", [True, False])
def test_far_pages(lib, fp8):
    """Pages whose bytes lie past 4 GiB of the pool."""
    rng = np.random.default_rng(8)
    stride = PAGE8 if fp8 else 2 * PAGE * LATENT
    pages = (5 << 30) // stride
    small = Cache(rng, 6, fp8)
    pool = torch.empty((pages, stride), dtype=torch.uint8, device="cuda")
    (src, *_), _ = small.device()
    pool[pages - 6:] = src.reshape(6, -1).view(torch.uint8)
    args = (pool, pool.data_ptr() + PAGE * LATENT) if fp8 else (pool,)
    table = np.stack([rng.permutation(6)[:4] for _ in range(3)]).astype(np.int32)
    lengths = np.array([256, 200, 1])
    q = queries(rng, 3, 64)
    out, lse = call(lib, (args, {}), q, torch.from_numpy(table + pages - 6), None, torch.from_numpy(lengths.astype(np.int32)),
                    num_pages=pages)
    assert_attention(out, lse, attention(q, small.values(), table, lengths, SCALE))


def test_long_context(lib):
    """262,208 positions (4,097 pages), all of them and 2,048 of them."""
    rng = np.random.default_rng(9)
    pages = 4097
    kv = torch.randint(0, 120, (pages, PAGE8), dtype=torch.uint8, device="cuda")  # codes of positive values, no NaN
    kv[:, PAGE * LATENT:] = (torch.rand((pages, PAGE), device="cuda") * 0.01).view(torch.uint8)
    pool = ((kv, kv.data_ptr() + PAGE * LATENT), {})
    values = latent_values(kv[:, : PAGE * LATENT].contiguous(), kv[:, PAGE * LATENT:].contiguous().view(torch.float32), True)
    table = rng.permutation(pages)[None].astype(np.int32)
    lengths = np.array([pages * PAGE - 3])
    q = queries(rng, 1, 8, 0.02)
    out, lse = call(lib, pool, q, torch.from_numpy(table), None, torch.from_numpy(lengths.astype(np.int32)), num_pages=pages)
    assert_attention(out, lse, attention(q, values, table, lengths, SCALE))
    selected = some(rng, int(lengths[0]), 2048, 2048)[None]
    out, lse = call(lib, pool, q, torch.from_numpy(table), torch.from_numpy(selected), torch.from_numpy(lengths.astype(np.int32)),
                    num_pages=pages)
    assert_attention(out, lse, attention(q, values, table, lengths, SCALE, selected))


def test_nothing_to_do(lib):
    """No rows, no heads, no table columns, an empty list: the outputs of rows
    with nothing selected are 0 and -inf, and nothing else is written."""
    rng = np.random.default_rng(10)
    cache = Cache(rng, 2, True)
    for rows, heads, width, k in [(0, 4, 2, 3), (3, 0, 2, 3), (3, 4, 0, 3), (3, 4, 2, 0), (3, 4, 0, None)]:
        q = queries(rng, rows, heads)
        table = torch.zeros((max(rows, 1), width), dtype=torch.int32)
        selected = None if k is None else torch.zeros((rows, k), dtype=torch.int32)
        out, lse = call(lib, cache, q, table, selected, torch.full((rows,), 70, dtype=torch.int32))
        assert (out == 0).all() and torch.isneginf(lse).all()


def test_split_join(lib):
    """Two disjoint sets of positions, joined by their lse, give the whole: out is
    off by the parts' tolerances."""
    rng = np.random.default_rng(11)
    cache = Cache(rng, 10, True)
    table = rng.permutation(10)[None].astype(np.int32)
    q = queries(rng, 1, 64)
    length = torch.tensor([640], dtype=torch.int32)
    order = rng.permutation(640).astype(np.int32)
    parts = [torch.from_numpy(np.sort(order[:300])[None]), torch.from_numpy(np.sort(order[300:])[None])]
    got = [call(lib, cache, q, torch.from_numpy(table), p, length) for p in parts]
    w = [torch.exp(l.double()) for _, l in got]
    joined = sum(o.double() * x[..., None] for (o, _), x in zip(got, w)) / sum(w)[..., None]
    out, lse, tols = attention(q, cache.values(), table, [640], SCALE)
    # each part carries its own tolerance, of the same form; joined they weigh as
    # their sums do, and the lse's errors shift that weight
    assert (np.abs(f64(joined) - out) <= 2 * tols[0] + 4 * tols[1][..., None] * np.abs(cache.values()).max()).all()


def test_streams_workspaces_and_graphs(lib):
    """Two calls at once on two streams with a workspace each; captured calls
    replayed on new queries, lists and lengths."""
    rng = np.random.default_rng(12)
    rows, heads, width, k = 3, 64, 16, 512
    cache = Cache(rng, 48, True)
    table = torch.from_numpy(rng.permutation(48).reshape(3, 16).astype(np.int32))
    pool, strides = cache.device()
    need = lib.idx_latent_attention_workspace(rows, heads, width, k)
    assert need > 0
    sets = []
    for _ in range(2):
        q = queries(rng, rows, heads).cuda()
        lengths = torch.from_numpy(rng.integers(200, 1024, rows).astype(np.int32)).cuda()
        selected = torch.from_numpy(np.stack([some(rng, int(n), k, k) for n in lengths.cpu()])).cuda()
        sets.append((q, selected, lengths, torch.empty_like(q), torch.empty((rows, heads), device="cuda"),
                     torch.empty(need, dtype=torch.uint8, device="cuda")))
    td = table.cuda()

    def go(s, stream=None):
        q, selected, lengths, out, lse, ws = s
        lib.idx_latent_attention_fp8(q, *pool, td, selected, lengths, out, lse, scale=SCALE, num_pages=48, workspace=ws, stream=stream)

    def check(s):
        q, selected, lengths, out, lse, _ = s
        assert_attention(out, lse, attention(q, cache.values(), table.numpy(), lengths.cpu().numpy(), SCALE, selected.cpu().numpy()))

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(sets, streams):
            go(s, st)
    torch.cuda.synchronize()
    for s in sets:
        check(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(sets[0])
        go(sets[1])
    for i in range(3):
        for s in sets:
            s[0].copy_(queries(rng, rows, heads))
            s[2].copy_(torch.from_numpy(rng.integers(0, 1025, rows).astype(np.int32)))
            s[1].copy_(torch.from_numpy(np.stack([some(rng, int(n), k, k) for n in s[2].cpu()])))
            s[3].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for s in sets:
            check(s)
        go(sets[0])  # eager work between the replays
        torch.cuda.synchronize()


def test_workspace_refusals(lib):
    q = torch.zeros((1, 64, LATENT), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((64, PAGE8), dtype=torch.uint8, device="cuda")
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    args = (q, kv, kv.data_ptr() + PAGE * LATENT, table, None, torch.tensor([4096], dtype=torch.int32, device="cuda"), torch.empty_like(q))
    need = lib.idx_latent_attention_workspace(1, 64, 64)
    small = torch.empty(need - 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.IdxError):
        lib.idx_latent_attention_fp8(*args, scale=1.0, num_pages=64, workspace=small)
    with pytest.raises(ValueError, match="raw stream"):
        lib.idx_latent_attention_fp8(*args, scale=1.0, num_pages=64, stream=torch.cuda.current_stream().cuda_stream)
    with pytest.raises(lib.IdxError):
        lib.idx_latent_attention_fp8(*args, scale=float("inf"), num_pages=64)
    lib.idx_latent_attention_fp8(*args, scale=1.0, num_pages=64, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fp8", [True, False])
def test_indexer_step(lib, fp8):
    """A decode step as it is used: new index keys and latents are normed,
    rotated and stored, index queries rotated, positions scored and selected,
    and the selected latents attended to."""
    rng = np.random.default_rng(13)
    rows, width, k, n = 6, 20, 256, 6 * 1280
    pages = rows * width
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    slots = torch.from_numpy(rng.permutation(n)).cuda()
    token = torch.from_numpy(rng.integers(0, 100000, n)).cuda()
    freq = inv_freq(32).cuda()
    keys, latents = new(n, 128), new(n, LATENT)
    kv = torch.zeros((pages, 8448), dtype=torch.uint8, device="cuda")
    lib.idx_norm_rope_store_fp8(keys, token, freq, slots, kv, kv.data_ptr() + 8192, num_pages=pages, halves=True)
    if fp8:
        pool = torch.zeros((pages, PAGE8), dtype=torch.uint8, device="cuda")
        lib.idx_norm_rope_store_fp8(latents, token, freq, slots, pool, pool.data_ptr() + PAGE * LATENT, num_pages=pages)
    else:
        pool = torch.zeros((pages, PAGE, LATENT), dtype=torch.bfloat16, device="cuda")
        lib.idx_norm_rope_store_bf16(latents, token, freq, slots, pool, num_pages=pages)
    stored = torch.empty((n, LATENT), dtype=torch.bfloat16, device="cuda")
    if fp8:
        lib.idx_load_slots_fp8(pool, pool.data_ptr() + PAGE * LATENT, slots, stored, num_pages=pages)
    else:
        lib.idx_load_slots_bf16(pool, slots, stored, num_pages=pages)
    at = torch.from_numpy(rng.integers(100000, 100010, rows)).cuda()
    iq, aq = new(rows, 64, 128), new(rows, 64, LATENT)
    lib.idx_norm_rope(iq, at, freq, iq, halves=True)
    lib.idx_norm_rope(aq, at, freq, aq)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").reshape(rows, width)
    lengths = torch.tensor([1280, 1279, 700, 256, 100, 0], dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.standard_normal((rows, 64)).astype(np.float32)).cuda()
    logits = torch.empty((rows, width * PAGE), device="cuda")
    selected = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    lib.idx_paged_mqa_topk_fp8(iq, kv, kv.data_ptr() + 8192, table, lengths, w, logits, selected, num_pages=pages)
    out, lse = torch.empty_like(aq), torch.empty((rows, 64), device="cuda")
    if fp8:
        lib.idx_latent_attention_fp8(aq, pool, pool.data_ptr() + PAGE * LATENT, table, selected, lengths, out, lse, scale=SCALE, num_pages=pages)
        values = latent_values(pool[:, : PAGE * LATENT].contiguous(), pool[:, PAGE * LATENT:].contiguous().view(torch.float32), True)
    else:
        lib.idx_latent_attention_bf16(aq, pool, table, selected, lengths, out, lse, scale=SCALE, num_pages=pages)
        values = f64(pool)
    flat = values.reshape(-1, LATENT)[slots.cpu().numpy()]
    assert (np.abs(f64(stored) - flat) <= np.abs(flat) * (2.0 ** -8 + 2.0 ** -23)).all()
    chosen = selected.cpu().numpy()
    assert [(c >= 0).sum() for c in chosen] == [256, 256, 256, 256, 100, 0]
    assert_attention(out, lse, attention(aq, values, table.cpu().numpy(), lengths.cpu().numpy(), SCALE, chosen))


def repeated(rows, distinct, *tensors):
    """Rows 0 .. distinct-1 of each tensor, over and over."""
    at = torch.arange(rows) % distinct
    return [t[at].contiguous() for t in tensors]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads", [8, 70])
def test_long_lists_in_one_unit(lib, fp8, heads):
    """Rows enough that none is split, so that one workgroup goes through all
    tiles of a list: lists of 8, 9, 12, 13, 16, 17 and 32 tiles, whole and with a
    part of a tile behind them, with entries to skip and a bad page in the tiles
    whose places are resolved while the first are used."""
    rng = np.random.default_rng(21 + heads)
    rows, width, k, scale = 264, 48, 2048, SCALE
    counts = [512, 513, 576, 577, 768, 769, 832, 900, 1024, 1030, 1100, 2047, 2048, 2048, 2048, 2048]
    distinct = len(counts)
    pages = 60
    table = np.stack([rng.permutation(pages)[:width] for _ in range(distinct)]).astype(np.int32)
    lengths = np.array([c if c < k else width * PAGE - 5 for c in counts])
    selected = np.stack([some(rng, int(L), k, k) for L in lengths])
    announce(f"long lists fp8={fp8} rows={rows} heads={heads}")
    for b, c in enumerate(counts):  # skipped: padding, past the row, past the table, before it
        for tile in (0, 7, 8, 9, 11, 12, (c - 1) // 64):
            if 64 * tile < c:
                at = 64 * tile + rng.permutation(min(64, c - 64 * tile))[:4]
                selected[b, at] = np.array([-1, lengths[b], width * PAGE + 3, -2 ** 31])[: len(at)]
    selected[12, 8 * 64: 9 * 64] = -1             # a tile with nothing in it
    selected[13, : 9 * 64] = -1                   # nothing before tile 9
    selected[14, 31 * 64:] = -1                   # nothing in the last tile
    bad = {10: 8, 11: 12, 15: 31}                 # one bad page in that tile
    for b, tile in bad.items():
        live = [p for p in selected[b, 64 * tile: 64 * tile + 64] if 0 <= p < lengths[b]]
        page = live[len(live) // 2] // PAGE
        inside = (selected[b] >= page * PAGE) & (selected[b] < (page + 1) * PAGE)
        inside[64 * tile: 64 * tile + 64] = False
        selected[b, inside] = -1                  # only that tile names it
        table[b, page] = pages + b
    cache = Cache(rng, pages, fp8)
    used = set()
    for b in range(distinct):
        at = selected[b][: min(k, lengths[b])].astype(np.int64)
        at = at[(at >= 0) & (at < lengths[b])]
        page = table[b][at // PAGE]
        used |= set((page * PAGE + at % PAGE)[page < pages].tolist())
    cache.poison(used)
    q = queries(rng, distinct, heads)
    sinks = torch.from_numpy(rng.standard_normal(heads).astype(np.float32))
    want = attention(q, np.nan_to_num(cache.values()), table, lengths, scale, selected, sinks)
    assert [b for b in range(distinct) if np.isnan(want[0][b]).any()] == sorted(bad)
    assert lib.idx_latent_attention_workspace(rows, heads, width, k) == 0  # unsplit
    args = repeated(rows, distinct, q, torch.from_numpy(table), torch.from_numpy(selected), torch.from_numpy(lengths.astype(np.int32)))
    out, lse = call(lib, cache, *args, sinks=sinks)
    assert_attention(out[:distinct], lse[:distinct], want)
    # the same rows elsewhere in the batch: the same bits
    first = torch.arange(rows, device="cuda") % distinct
    assert torch.equal(out.view(torch.int16), out[first].view(torch.int16))
    again, logs = call(lib, cache, *args, sinks=sinks)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(logs.view(torch.int32), lse.view(torch.int32))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("scale", [0.3, -0.3, 4.0])
def test_scores_that_grow_in_one_unit(lib, fp8, scale):
    """The running maximum moves from tile to tile of one workgroup's, by a few
    and by hundreds, up and (negative scales) down."""
    rng = np.random.default_rng(30)
    rows, heads, width, distinct = 260, 40, 30, 4
    cache = Cache(rng, 40, fp8)
    grow = torch.linspace(0.05, 3.0, 40)[:, None]
    if fp8:
        cache.scales = cache.scales * grow
    else:
        cache.kv = (cache.kv.float() * grow[..., None]).to(torch.bfloat16)
    table = np.stack([np.sort(rng.permutation(40)[:width]) for _ in range(distinct)]).astype(np.int32)
    lengths = np.array([1920, 1919, 700, 64])
    q = queries(rng, distinct, heads, 1.0)
    assert lib.idx_latent_attention_workspace(rows, heads, width) == 0
    args = repeated(rows, distinct, q, torch.from_numpy(table), torch.from_numpy(lengths.astype(np.int32)))
    out, lse = call(lib, cache, args[0], args[1], None, args[2], scale=scale)
    assert_attention(out[:distinct], lse[:distinct], attention(q, cache.values(), table, lengths, scale))
    first = torch.arange(rows, device="cuda") % distinct
    assert torch.equal(out.view(torch.int16), out[first].view(torch.int16))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows", [4, 270])
def test_no_numbers_stay_where_they_are(lib, fp8, rows):
    """A query that holds a NaN or infinities of both signs makes its own head
    NaN, a latent that holds a NaN the rows that select it, a sink that is NaN its
    head; the other heads and rows have the bits that they have without."""
    rng = np.random.default_rng(31)
    heads, width, distinct, k = 40, 12, 4, 400
    cache = Cache(rng, 30, fp8)
    table = np.stack([rng.permutation(28)[:width] for _ in range(distinct)]).astype(np.int32)
    table[2, 5] = 28  # a page of row 2's alone
    lengths = np.array([768, 700, 768, 65])
    selected = np.stack([some(rng, int(n), k, k) for n in lengths])
    inside = np.flatnonzero(selected[2] // PAGE == 5)[0]
    q = queries(rng, distinct, heads)
    sinks = torch.from_numpy(rng.standard_normal(heads).astype(np.float32))
    args = lambda q: repeated(rows, distinct, q, torch.from_numpy(table), torch.from_numpy(selected), torch.from_numpy(lengths.astype(np.int32)))  # noqa: E731
    plain, plain_lse = call(lib, cache, *args(q), sinks=sinks)
    bad = q.clone()
    bad[0, 3, 100] = float("nan")
    bad[1, 35] = torch.where(torch.arange(LATENT) % 2 == 0, float("inf"), -float("inf")).to(torch.bfloat16)
    slot = int(selected[2][inside]) % PAGE
    if fp8:
        cache.kv[28, slot, 77] = 0xFF
    else:
        cache.kv[28, slot, 77] = float("nan")
    odd = sinks.clone()
    odd[7] = float("nan")
    out, lse = call(lib, cache, *args(bad), sinks=odd)
    none = torch.zeros((distinct, heads), dtype=torch.bool)
    none[0, 3] = none[1, 35] = True
    none[2] = True
    none[:, 7] = True
    none = none[torch.arange(rows) % distinct].cuda()
    assert out[none].isnan().all() and lse[none].isnan().all()
    assert torch.equal(out[~none].view(torch.int16), plain[~none].view(torch.int16))
    assert torch.equal(lse[~none].view(torch.int32), plain_lse[~none].view(torch.int32))
