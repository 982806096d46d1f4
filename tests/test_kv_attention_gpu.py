"""Attention of one new token per row over paged keys and values by head, on the GPU
against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
from kv_reference import PAGE, assert_near_attention, make_pools, values_of
from latent_reference import f64

pytestmark = pytest.mark.gpu

I32, BF16 = torch.int32, torch.bfloat16


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32).cuda()


class Case:
    """Inputs of a call, its guarded outputs, and the float64 result."""

    def __init__(self, seed, lengths, heads, kv_heads, dim, width, fp8, k=None, sinks=False, row_table=None, layout="fused", tables=None,
                 bad=(), selected=None, scale=None, size=1.0, spare=1, num_pages=None, spoil=None):
        gen = torch.Generator().manual_seed(seed)
        rows = len(lengths)
        tables = tables or (rows if row_table is None else 3)
        pages = tables * width + spare
        self.k, self.v, self.scales = make_pools(gen, pages, kv_heads, dim, fp8, layout)
        if spoil:
            spoil(self)
        self.fp8, self.dim, self.scale = fp8, dim, dim ** -0.5 if scale is None else scale
        self.q = (size * torch.randn((rows, heads, dim), generator=gen)).to(BF16).cuda()
        table = torch.randperm(pages, generator=gen)[: tables * width].reshape(tables, width).to(I32)
        for t, j, page in bad:
            table[t, j] = page
        self.table = table.cuda()
        self.lengths = i32(lengths)
        self.sinks = (2 * torch.randn((heads,), generator=gen)).cuda() if sinks else None
        self.row_table = None if row_table is None else i32(row_table)
        self.num_pages = num_pages
        self.selected = None
        if selected is not None:
            self.selected = i32(selected)
        elif k is not None:  # as a top-k leaves it: ascending, -1 behind
            picks = torch.full((rows, kv_heads, k), -1, dtype=I32)
            for b, n in enumerate(lengths):
                count = min(-(-max(n, 0) // PAGE), width)
                for h in range(kv_heads):
                    some = torch.randperm(count, generator=gen)[:k].sort().values.to(I32)
                    picks[b, h, : len(some)] = some
            self.selected = picks.cuda()
        self.guard = torch.full((rows + 2, heads, dim), 7.0, dtype=BF16, device="cuda")
        self.guard_lse = torch.full((rows + 2, heads), 7.0, device="cuda")
        self.out, self.lse = self.guard[1:-1], self.guard_lse[1:-1]

    def run(self, lib, **kw):
        kw = dict(scale=self.scale, sinks=self.sinks, row_table=self.row_table, num_pages=self.num_pages, **kw)
        call = lib.idx_kv_attention_fp8 if self.fp8 else lib.idx_kv_attention_bf16
        call(self.q, self.k, self.v, *self.scales, self.table, self.selected, self.lengths, self.out, self.lse, **kw)

    def want(self):
        scales = self.scales or (None, None)
        return ref.attention(f64(self.q), values_of(self.k, scales[0]), values_of(self.v, scales[1]), self.table.cpu().numpy(),
                             None if self.selected is None else self.selected.cpu().numpy(), self.lengths.cpu().numpy(), self.scale,
                             self.k.shape[0] if self.num_pages is None else self.num_pages, None if self.sinks is None else f64(self.sinks),
                             None if self.row_table is None else self.row_table.cpu().numpy())

    def check(self, lib, **kw):
        self.run(lib, **kw)
        torch.cuda.synchronize()
        positions = int(self.lengths.clamp(min=0).max()) if self.selected is None else PAGE * self.selected.shape[-1]
        assert_near_attention(self.out, self.lse, self.want(), self.dim, positions)
        for g in (self.guard, self.guard_lse):
            assert (g[0] == 7).all() and (g[-1] == 7).all()


LENGTHS = [1, 64, 0, 65, 300, 63, 640, 129]


@pytest.mark.parametrize("heads,kv_heads,dim", [
    (1, 1, 64), (8, 8, 64), (40, 8, 64), (34, 2, 64), (64, 1, 64), (130, 2, 64),
    (1, 1, 128), (8, 2, 128), (64, 8, 128), (17, 1, 128), (64, 2, 128), (33, 1, 128), (64, 1, 128), (128, 1, 128), (200, 2, 128),
    (2, 1, 256), (16, 1, 256), (48, 2, 256), (64, 1, 256), (128, 1, 256),
])
@pytest.mark.parametrize("fp8", [True, False])
def test_shapes(lib, heads, kv_heads, dim, fp8):
    Case(heads + dim, LENGTHS, heads, kv_heads, dim, 10, fp8).check(lib)


@pytest.mark.parametrize("k", [0, 1, 2, 7, 10, 33])
@pytest.mark.parametrize("fp8,dim,heads,kv_heads", [(True, 128, 16, 2), (False, 128, 24, 4), (True, 64, 5, 5), (False, 256, 40, 2)])
def test_selected(lib, k, fp8, dim, heads, kv_heads):
    Case(k + dim, LENGTHS, heads, kv_heads, dim, 10, fp8, k=k, sinks=k % 2 == 0).check(lib)


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [1], [2], [31], [32], [33], [64], [128, 1], [-5, 2 ** 31 - 1, 3]])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("sinks", [True, False])
def test_lengths(lib, lengths, fp8, sinks):
    Case(len(lengths), lengths, 8, 2, 128, 4, fp8, sinks=sinks).check(lib)


@pytest.mark.parametrize("width", [0, 1, 2, 3])
def test_narrow_tables(lib, width):
    Case(width, [200, 64, 1, 0], 8, 2, 128, width, True).check(lib)
    Case(width, [200, 64, 1, 0], 8, 2, 128, width, False, sinks=True).check(lib)


@pytest.mark.parametrize("fp8,dim,heads,kv_heads,length", [(True, 128, 64, 8, 9000), (False, 128, 8, 1, 20011), (False, 64, 32, 4, 5000),
                                                          (True, 256, 4, 2, 7000), (False, 128, 64, 1, 10001)])
def test_one_long_row(lib, fp8, dim, heads, kv_heads, length):
    """A row that all workgroups share: many pieces to join."""
    Case(length, [length], heads, kv_heads, dim, -(-length // PAGE) + 3, fp8, sinks=True).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
def test_uneven_rows(lib, fp8):
    """Shares that hold the end of a row, whole rows and the start of another."""
    rng = np.random.default_rng(5)
    lengths = (rng.integers(0, 2, 50) * rng.integers(0, 3000, 50)).tolist() + [4000]
    Case(50, lengths, 12, 3, 64, 63, fp8).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
def test_more_units_than_workgroups(lib, fp8):
    """A unit a workgroup, nothing to join."""
    rng = np.random.default_rng(6)
    Case(6, rng.integers(0, 200, 300).tolist(), 16, 8, 64, 3, fp8, sinks=True, tables=1).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("layout", ["heads", "apart"])
def test_layouts(lib, fp8, layout):
    Case(7, LENGTHS, 24, 3, 128, 10, fp8, layout=layout).check(lib)
    Case(8, LENGTHS, 24, 3, 64, 10, fp8, layout=layout, k=3).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
def test_row_table(lib, fp8):
    """Rows of shared tables; table indexes out of range make their rows NaN."""
    Case(9, [200, 300, 5, 64, 100, 0, 640], 8, 2, 128, 10, fp8, row_table=[2, 0, 2, -1, 3, 7, 1], sinks=True).check(lib)
    Case(10, [200, 300, 5], 8, 2, 128, 10, fp8, tables=1).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
def test_bad_pages(lib, fp8):
    """A page id outside the pool makes the rows that have it NaN, others nothing."""
    bad = [(0, 2, -1), (1, 3, 1 << 30), (2, 5, -2 ** 31), (3, 1, 99)]
    Case(11, [300, 200, 300, 300], 8, 2, 128, 8, fp8, bad=bad).check(lib)
    Case(12, [300, 200, 300, 300], 8, 2, 128, 8, fp8, bad=bad, selected=[[[0, 2], [0, 1]], [[1, 2], [0, 3]], [[4, 5], [0, 1]], [[0, 2], [1, 3]]]).check(lib)
    Case(13, [300, 200], 8, 2, 64, 5, fp8, num_pages=6).check(lib)  # ids of the tensor, past num_pages


@pytest.mark.parametrize("fp8", [True, False])
def test_odd_selections(lib, fp8):
    """Out of order, twice, past the row's end, negative, behind as many as the row has."""
    listed = [[[3, 1, 0, 2]], [[1, 1, 1, 0]], [[9, 0, 5, -3]], [[-1, -1, 2, 0]], [[0, 0, 1, 2]], [[4, 4, 4, 4]], [[1, 2 ** 31 - 1, -2 ** 31, 0]]]
    Case(14, [256, 200, 190, 300, 100, 257, 400], 8, 1, 128, 7, fp8, selected=listed, sinks=True).check(lib)


def test_selection_as_the_topk_leaves_it(lib):
    """[rows * kv_heads, k] is taken too."""
    c = Case(15, LENGTHS, 8, 2, 128, 10, True, k=3)
    c.check(lib)
    c.selected = c.selected.flatten(0, 1)
    before = c.out.clone()
    c.run(lib)
    assert torch.equal(before, c.out)


@pytest.mark.parametrize("fp8", [True, False])
def test_slots_past_the_end(lib, fp8):
    """NaN and infinities past a row's length have no part, nor do those of other pages."""
    lengths = [1, 30, 32, 33, 63, 100, 127]

    def spoil(c):
        c.spoiled = True
    clean = Case(16, lengths, 8, 2, 128, 2, fp8, spoil=spoil)
    clean.run(lib)
    want = clean.out.clone()
    for word in (float("nan"), float("inf"), -float("inf")):
        for b, n in enumerate(lengths):
            for j in range(2):
                page, from_ = int(clean.table[b, j]), min(max(n - 64 * j, 0), 64)
                for i, pool in enumerate((clean.k, clean.v)):
                    if fp8:
                        pool.view(torch.uint8)[page, :, from_:] = 0x7F
                        clean.scales[i][page, :, from_:] = word
                    else:
                        pool[page, :, from_:] = word
        used = set(clean.table.flatten().tolist())
        for page in set(range(clean.k.shape[0])) - used:
            for pool in (clean.k, clean.v):
                pool.view(torch.uint8)[page] = 0x7F
        clean.out.fill_(3)
        clean.run(lib)
        assert torch.equal(clean.out, want)


@pytest.mark.parametrize("fp8", [True, False])
def test_values_that_are_no_numbers(lib, fp8):
    """A NaN key makes its heads' rows NaN, a NaN value its dim; nothing else."""
    c = Case(17, [200, 200, 100], 8, 2, 64, 4, fp8)
    c.run(lib)
    clean = c.out.clone()
    page = [int(x) for x in c.table[:, 1]]
    if fp8:
        c.k.view(torch.uint8)[page[0], 1, 5, 7] = 0x7F
        c.v.view(torch.uint8)[page[1], 0, 9, 11] = 0xFF
    else:
        c.k[page[0], 1, 5, 7] = float("nan")
        c.v[page[1], 0, 9, 11] = float("nan")
    c.run(lib)
    nan = c.out.isnan().cpu()
    want = torch.zeros_like(nan)
    want[0, 4:] = True
    want[1, :4, 11] = True
    assert torch.equal(nan, want)
    assert torch.equal(c.out[~nan.cuda()], clean[~nan.cuda()])


@pytest.mark.parametrize("fp8", [True, False])
def test_wide_scores(lib, fp8):
    """Scores that grow and fall by hundreds along a row move the reference again and
    again; those of all positions far below zero or a sink leave nothing but it."""
    c = Case(18, [640, 500, 333], 8, 2, 64, 10, fp8, scale=4.0, size=3.0, sinks=True)
    c.check(lib)
    ramp = torch.linspace(-40, 60, 640)
    for b in range(3):
        for j in range(10):
            page = int(c.table[b, j])
            by = (ramp if b < 2 else ramp.flip(0))[64 * j : 64 * j + 64]
            if fp8:
                c.k.view(torch.uint8)[page] = 0x38  # 1.0
                c.scales[0][page] = by.abs().cuda() / 60
            else:
                c.k[page] = (by / 60).to(BF16).cuda()[:, None]
    c.q.fill_(1.0)
    c.check(lib)
    c.q.fill_(-30.0)
    c.check(lib)
    c.sinks.fill_(10000.0)
    c.check(lib)
    c.sinks.fill_(-10000.0)
    c.check(lib)
    c.sinks.fill_(-float("inf"))
    c.check(lib)


def test_workspace(lib):
    """What a workspace holds before a call means nothing; too small a one is refused."""
    c = Case(19, [640, 10, 300], 16, 4, 128, 10, False)
    need = lib.idx_kv_attention_workspace(3, 16, 4, 128, 10)
    assert need > 0
    c.check(lib)
    want = c.out.clone()
    for byte in (0xFF, 0x7F, 0):
        c.out.zero_()
        c.run(lib, workspace=torch.full((need,), byte, dtype=torch.uint8, device="cuda"))
        assert torch.equal(c.out, want)
    with pytest.raises(lib.IdxError):
        c.run(lib, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="its own workspace"):
        c.run(lib, stream=torch.cuda.current_stream().cuda_stream)


def test_two_streams_at_once(lib):
    """Calls side by side, each with its own workspace, as one after the other."""
    cases = [Case(20 + i, [900, 64 * i, 500], 16, 2, 128, 15, i % 2 == 0) for i in range(4)]
    for c in cases:
        c.run(lib)
    want = [c.out.clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(lib, stream=s)
    torch.cuda.synchronize()
    for c, y in zip(cases, want):
        assert torch.equal(c.out, y)


def test_graph(lib):
    """Two captured calls, replayed in turn as lengths, tables and selections change in
    place, with eager work between, against the eager result each time."""
    dense = Case(30, [640, 0, 100, 333], 16, 2, 128, 10, True, sinks=True)
    picked = Case(31, [640, 64, 100, 333], 12, 3, 64, 10, False, k=3)
    graphs = []
    for c in (dense, picked):
        c.run(lib)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(lib)
        graphs.append(g)
    for step in range(4):
        for c, g in zip((dense, picked), graphs):
            c.lengths.copy_(torch.roll(c.lengths, 1))
            c.table.copy_(torch.roll(c.table, 3, 1))
            c.q.mul_(-1)
            c.out.fill_(9)
            g.replay()
            torch.cuda.synchronize()
            got, log = c.out.clone(), c.lse.clone()
            c.run(lib)
            assert torch.equal(got, c.out) and torch.equal(log, c.lse)
            c.check(lib)


def test_same_result_again(lib):
    """Bit for bit, whatever runs beside it."""
    c = Case(32, [5000, 100, 3000, 777], 40, 5, 128, 80, True)
    c.run(lib)
    want = c.out.clone()
    for _ in range(10):
        c.run(lib)
    assert torch.equal(c.out, want)


def test_split_results_join(lib):
    """Two calls over disjoint pages join by their log sums as the header says."""
    c = Case(33, [640, 640], 8, 2, 128, 10, False)
    c.check(lib)
    whole, lse = f64(c.out), f64(c.lse)
    parts = []
    for listed in ([0, 2, 4, 6, 8], [1, 3, 5, 7, 9]):
        c.selected = i32(np.broadcast_to(listed, (2, 2, 5)).copy())
        c.check(lib)
        parts.append((f64(c.out), f64(c.lse)))
    w = [np.exp(l - lse)[..., None] for _, l in parts]
    joined = sum(o * f for (o, _), f in zip(parts, w)) / sum(w)
    # a bf16 half step of each part, of the whole, and of the probabilities (v of 1 at most 5)
    assert np.abs(joined - whole).max() <= 3 * 2.0 ** -8 * 5 / 4
    assert np.allclose(np.logaddexp(parts[0][1], parts[1][1]), lse, atol=1e-5)


def test_a_run_of_them_together(lib):
    """Prompts, then decode steps, as a server has them: plan, rotation of keys, store,
    bounds, scores, top-k, attention over the selected pages; against float64 of the whole."""
    gen = torch.Generator().manual_seed(40)
    heads, kv_heads, dim, width, k = 16, 2, 128, 8, 3
    requests, pages = 4, 40
    prompts = [200, 1, 64, 390]
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    kp, vp, (ks, vs) = make_pools(gen, pages, kv_heads, dim, True)
    near = torch.zeros((pages, kv_heads, 2, dim), dtype=BF16, device="cuda")
    table = torch.full((requests, width), -1, dtype=I32, device="cuda")
    free = torch.randperm(pages, generator=gen).to(I32).cuda()
    cached = torch.zeros(requests, dtype=I32, device="cuda")
    added = i32(prompts)
    for step in range(4):
        n = sum(prompts) + 5 if step == 0 else requests
        slots, positions = (torch.empty(n, dtype=torch.int64, device="cuda") for _ in range(2))
        rows, lens = (torch.empty(n, dtype=I32, device="cuda") for _ in range(2))
        starts, taken = torch.empty(requests + 1, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda")
        lib.idx_plan_batch(cached, added, free, table, slots, positions, rows, lens, starts, taken)
        keys, values = (torch.randn((n, kv_heads, dim), generator=gen).to(BF16).cuda() for _ in range(2))
        lib.idx_norm_rope(keys, positions, freq, keys)
        lib.idx_store_kv_fp8(keys, values, slots, kp, vp, ks, vs)
        lib.idx_page_bounds_fp8(kp, ks, table, cached + added, near, first=cached)
        free = free[int(taken) :].contiguous()
        cached, added = cached + added, torch.ones_like(added)
        if step == 0:
            assert (slots[sum(prompts) :] == -1).all() and int(starts[-1]) == sum(prompts)
            continue
        q = torch.randn((requests, heads, dim), generator=gen).to(BF16).cuda()
        assert torch.equal(lens, cached) and rows.tolist() == [0, 1, 2, 3]
        scores = torch.empty((requests, kv_heads, width), device="cuda")
        counts = torch.empty((requests, kv_heads), dtype=I32, device="cuda")
        lib.idx_page_scores(q, near, table, lens, scores, counts, row_table=rows, last_pages=1)
        picked = torch.empty((requests * kv_heads, k), dtype=I32, device="cuda")
        lib.idx_topk_logits(scores.flatten(0, 1), counts.flatten(), picked)
        out, lse = torch.empty_like(q), torch.empty((requests, heads), device="cuda")
        lib.idx_kv_attention_fp8(q, kp, vp, ks, vs, table, picked, lens, out, lse, scale=dim ** -0.5, row_table=rows)
        torch.cuda.synchronize()
        picks = picked.cpu().numpy().reshape(requests, kv_heads, k)
        live = counts.cpu().numpy()
        for b in range(requests):
            for h in range(kv_heads):
                got = picks[b, h]
                assert (got >= 0).sum() == min(k, live[b, h]) and live[b, h] - 1 in got
        key_values, value_values = values_of(kp, ks), values_of(vp, vs)
        want_scores, _, want_live = ref.scores(f64(q), f64(near), table.cpu().numpy(), lens.cpu().numpy(), 0, 1, pages)
        assert (want_live == live).all() and np.allclose(f64(scores), want_scores, rtol=1e-5, atol=1e-4)
        want = ref.attention(f64(q), key_values, value_values, table.cpu().numpy(), picks, lens.cpu().numpy(), dim ** -0.5, pages)
        assert_near_attention(out, lse, want, dim, k * PAGE)


@pytest.mark.parametrize("seed", range(36))
def test_random_shapes(lib, seed):
    """Sizes across the ways of dividing a call: whole units, shares, units by themselves, few and many rows."""
    rng = np.random.default_rng(seed)
    dim = int(rng.choice([64, 128, 256]))
    kv_heads = int(rng.choice([1, 1, 2, 3, 8]))
    group = int(rng.choice([1, 3, 8, 16, 17, 30, 33, 64, 100, 128]))
    rows = int(rng.choice([1, 2, 7, 40, 64, 65, 100, 150]))
    width = int(rng.choice([1, 3, 9, 20, 33, 70]))
    while rows * kv_heads * width * dim > 1_500_000 or rows * kv_heads * group > 6000:
        rows, width = max(1, rows // 2), max(1, width * 2 // 3)
    lengths = (rng.random(rows) ** 2 * (64 * width + 1)).astype(int)
    lengths[rng.integers(rows)] = 64 * width
    if rows > 3:
        lengths[rng.integers(rows)] = 0
    k = None if rng.random() < 0.6 else int(rng.integers(0, width + 3))
    Case(seed, lengths.tolist(), kv_heads * group, kv_heads, dim, width, bool(rng.random() < 0.5), k=k, sinks=bool(rng.random() < 0.5),
         layout=str(rng.choice(["fused", "heads", "apart"]))).check(lib)


@pytest.mark.parametrize("rows,width,heads,kv_heads", [(65, 40, 8, 2), (100, 60, 2, 1), (200, 35, 3, 3), (130, 70, 64, 1)])
@pytest.mark.parametrize("fp8", [True, False])
def test_many_rows_shared_out(lib, rows, width, heads, kv_heads, fp8):
    """More rows than lanes, cut into shares; some empty, one far longer than the others."""
    rng = np.random.default_rng(rows)
    lengths = np.where(rng.random(rows) < 0.2, 0, rng.integers(1, 500, rows))
    lengths[rows // 2] = 64 * width
    assert lib.idx_kv_attention_workspace(rows, heads, kv_heads, 64, width) > 0
    Case(rows, lengths.tolist(), heads, kv_heads, 64, width, fp8, sinks=True).check(lib)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30])
def test_scales(lib, scale):
    """Nothing, turned round, next to nothing."""
    Case(41, LENGTHS, 8, 2, 128, 10, True, scale=scale).check(lib)
    Case(42, LENGTHS, 40, 1, 64, 10, False, scale=scale, sinks=True).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
def test_far_pages(lib, fp8):
    """Pages 2 GiB apart, heads in any order: offsets past 32 bits; stored, bounded and attended to."""
    gen = torch.Generator().manual_seed(50)
    pages, kv_heads, dim, apart = 4, 2, 128, 1 << 31
    size = 1 if fp8 else 2
    block = 64 * dim * size
    flat = torch.zeros(3 * apart + 8 * block, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn if fp8 else BF16)
    strides = (apart // size, 4 * block // size, dim, 1)
    k = flat.as_strided((pages, kv_heads, 64, dim), strides)
    v = flat.as_strided((pages, kv_heads, 64, dim), strides, 2 * block // size)
    scales = tuple(torch.zeros((pages, kv_heads, 64), device="cuda") for _ in range(2)) if fp8 else ()
    n = 200
    x = torch.randn((n, 2, kv_heads, dim), generator=gen).to(BF16).cuda()
    table = torch.tensor([[3, 1, 2, 0]], dtype=I32, device="cuda")
    at = torch.arange(n, device="cuda")
    slots = table[0].long()[at // 64] * 64 + at % 64
    store, bound, attend = ((lib.idx_store_kv_fp8, lib.idx_page_bounds_fp8, lib.idx_kv_attention_fp8) if fp8 else
                            (lib.idx_store_kv_bf16, lib.idx_page_bounds_bf16, lib.idx_kv_attention_bf16))
    store(x[:, 0], x[:, 1], slots, k, v, *scales)
    near = torch.zeros((pages, kv_heads, 2, dim), dtype=BF16, device="cuda")
    lengths = i32([n])
    bound(k, *scales[:1], table, lengths, near)
    q = torch.randn((1, 8, dim), generator=gen).to(BF16).cuda()
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    attend(q, k, v, *scales, table, None, lengths, out, lse, scale=0.1)
    torch.cuda.synchronize()
    keys, values = (values_of(p.contiguous(), s) for p, s in ((k, scales[0] if fp8 else None), (v, scales[1] if fp8 else None)))
    got = keys[slots.cpu().numpy() // 64, :, slots.cpu().numpy() % 64]
    want = f64(x[:, 0])
    assert (got == want).all() if not fp8 else (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 * 1.01 + 0.01).all()
    limits = ref.bounds(keys, table.cpu().numpy(), [0], [n], np.zeros((pages, kv_heads, 2, dim)), pages)
    assert (np.abs(f64(near) - limits) <= np.abs(limits) * 2.0 ** -7).all()
    assert_near_attention(out, lse, ref.attention(f64(q), keys, values, table.cpu().numpy(), None, [n], 0.1, pages), dim, n)


def test_heads_are_pools_of_the_other_operators(lib):
    """A head of the keys is a pool that idx_load_slots_fp8 reads and idx_norm_rope_store_fp8 writes."""
    gen = torch.Generator().manual_seed(51)
    pages, kv_heads, dim = 5, 3, 128
    k, v, (ks, vs) = make_pools(gen, pages, kv_heads, dim, True, "fused")
    slots = torch.randperm(pages * 64, generator=gen)[:100].cuda()
    stride = dict(num_pages=pages, kv_page_stride=k.stride(0), kscale_page_stride=4 * ks.stride(0))
    for h in range(kv_heads):
        x = torch.randn((100, dim), generator=gen).to(BF16).cuda()
        at, scale_at = k.data_ptr() + h * k.stride(1), ks.data_ptr() + 4 * h * ks.stride(1)
        lib.idx_norm_rope_store_fp8(x, None, None, slots, at, scale_at, norm=False, **stride)
        other, _, (other_scale, _) = make_pools(torch.Generator().manual_seed(0), pages, 1, dim, True, "apart")
        lib.idx_store_kv_fp8(x[:, None], x[:, None], slots, other, other.clone(), other_scale, other_scale.clone())
        page, pos = slots // 64, slots % 64
        assert torch.equal(k.view(torch.uint8)[page, h, pos], other.view(torch.uint8)[page, 0, pos])
        back = torch.empty((100, dim), dtype=BF16, device="cuda")
        lib.idx_load_slots_fp8(at, scale_at, slots, back, **stride)
        want = k.view(torch.uint8)[page, h, pos].view(torch.float8_e4m3fn).float() * ks[page, h, pos][:, None]
        assert torch.equal(back, want.to(BF16))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads,width,sinks", [(2, 2, False), (2, 60, True), (40, 2, False), (40, 60, False), (128, 60, False)])
def test_scores_at_the_low_end(lib, fp8, heads, width, sinks):
    """Logits next to float32's lowest value are numbers as others: positions of the same
    logit share the weight, a larger one has it all.  (A product of one value of q and one
    of k: -1.3125 * 2^127 with the scale, and log2(e) times that, -1.8935 * 2^127, in base
    2; float32 ends at -2 * 2^127.)"""
    n = 64 * width - 7
    c = Case(60, [n, n, 0], heads, 2, 64, width, fp8, scale=0.75, sinks=sinks)
    x = -1.3125 * 2.0 ** 127
    c.q.zero_()
    c.q[..., 5] = -1.75 * 2.0 ** 64
    if fp8:
        c.k.view(torch.uint8).zero_()
        c.k.view(torch.uint8)[..., 5] = 0x38  # 1.0
        c.scales[0].fill_(2.0 ** 63)
    else:
        c.k.zero_()
        c.k[..., 5] = 2.0 ** 63
    if sinks:
        c.sinks.fill_(-float("inf"))
    c.run(lib)
    keys = f64(c.v) if not fp8 else values_of(c.v, c.scales[1])
    for b in range(2):
        pages = [int(j) for j in c.table[b]]
        v = np.concatenate([keys[p] for p in pages], 1)[:, :n]  # [kv heads, n, dim]
        mean, size = v.mean(1).repeat(heads // 2, 0), np.abs(v).mean(1).repeat(heads // 2, 0)
        # float32 sums of n products (of probabilities 1 and, in e4m3, scales rounded to
        # bf16, 2^-8 of each), one rounding of the result to bf16
        err = size * ((2.0 ** -8 if fp8 else 0) + (n + 8) * 2.0 ** -24) + np.abs(mean) * 2.0 ** -8
        assert (np.abs(f64(c.out[b]) - mean) <= err).all()
        assert np.abs(f64(c.lse[b]) / x - 1).max() <= 2.0 ** -21
    assert (c.out[2] == 0).all() and torch.isneginf(c.lse[2]).all()
    page, at = int(c.table[1, width - 1]), 11  # a smaller amount: the largest logit of row 1
    if fp8:
        c.scales[0][page, :, at] *= 0.9375
    else:
        c.k[page, :, at, 5] *= 0.9375
    c.run(lib)
    want = keys[page, :, at].repeat(heads // 2, 0)
    assert (np.abs(f64(c.out[1]) - want) <= np.abs(want) * (2.0 ** -7 if fp8 else 0)).all()
    assert np.abs(f64(c.lse[1]) / (0.9375 * x) - 1).max() <= 2.0 ** -21


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lengths,width,k", [([100, 0, 300], 5, None), ([100, 0, 5000], 80, None), ([300, 0, 5000], 80, 3)])
def test_sink_of_infinity(lib, fp8, lengths, width, k):
    """exp(x) / inf = 0: nothing is left of the positions, and ln z is infinite; the
    other heads have the bits that they have without it."""
    c = Case(61, lengths, 8, 2, 64, width, fp8, k=k, sinks=True)
    c.run(lib)
    plain, plain_lse = c.out.clone(), c.lse.clone()
    c.sinks[5] = float("inf")
    c.run(lib)
    assert (c.out[:, 5] == 0).all() and torch.isposinf(c.lse[:, 5]).all()
    others = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(c.out[:, others], plain[:, others]) and torch.equal(c.lse[:, others], plain_lse[:, others])


def few_long_rows(rows, pages, width):
    """Rows of up to two pages, and some of up to `pages`."""
    lengths = [(37 * b) % 129 for b in range(rows)]
    for i, p in enumerate(pages):
        lengths[(i * rows) // len(pages) + 1] = 64 * p - 13 * i
    return lengths


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows,group,kv_heads,dim", [(260, 1, 8, 128), (260, 20, 8, 64), (260, 40, 8, 64), (260, 3, 8, 256), (131, 100, 8, 64)])
def test_whole_units_of_many_pages(lib, rows, group, kv_heads, dim, fp8):
    """More units than are cut, some of more pages than the 64 that are looked up
    early: all pages, and lists with entries to skip and pages outside the pool on
    both sides of the 64th."""
    width = 200
    lengths = few_long_rows(rows, [64, 65, 129, 200, 66], width)
    assert lib.idx_kv_attention_workspace(rows, kv_heads * group, kv_heads, dim, width) == 0
    Case(70, lengths, kv_heads * group, kv_heads, dim, width, fp8, tables=1, sinks=True).check(lib)
    Case(71, lengths, kv_heads * group, kv_heads, dim, width, fp8, tables=1, bad=[(0, 65, -1), (0, 199, 1 << 20)]).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("rows,group,kv_heads,dim", [(260, 2, 8, 128), (260, 33, 8, 64), (64, 8, 8, 128)])
def test_whole_units_of_long_lists(lib, rows, group, kv_heads, dim, fp8):
    width, k = 150, 140
    lengths = few_long_rows(rows, [150, 64, 141, 149, 100], width)
    rng = np.random.default_rng(rows)
    picks = np.full((rows, kv_heads, k), -1)
    for b, n in enumerate(lengths):
        count = -(-n // PAGE)
        for h in range(kv_heads):
            some = np.sort(rng.permutation(count)[:k])
            picks[b, h, : len(some)] = some
    long = int(np.argmax(lengths))
    for at in (3, 63, 64, 65, 127, 128, 139):  # to be skipped
        picks[long, at % kv_heads, at] = rng.choice([-1, -9, width, 2 ** 31 - 1])
    c = Case(72, lengths, kv_heads * group, kv_heads, dim, width, fp8, tables=1, selected=picks, sinks=True)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert lib.idx_kv_attention_workspace(rows, kv_heads * group, kv_heads, dim, width, k) == 0
    c.check(lib)
    picks[long, 1, 2], picks[long, 2, 100] = 70, 71  # pages that are outside the pool
    Case(73, lengths, kv_heads * group, kv_heads, dim, width, fp8, tables=1, selected=picks, bad=[(0, 70, 1 << 20), (0, 71, -5)]).check(lib)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("group,dim", [(1, 64), (8, 128), (16, 256), (32, 128), (20, 64), (64, 64), (64, 128), (50, 256)])
def test_past_the_caches(lib, group, dim, fp8):
    """Calls whose tables may name 256 MiB and more, few and many pages to a row, cut
    and whole."""
    kv_heads, rows = 2, 9
    page_bytes = 2 * PAGE * dim * (1 if fp8 else 2)
    width = -(-(1 << 28) // (rows * kv_heads * page_bytes))
    lengths = [1, 64 * 40 - 7, 0, 640, 65, 3000, 64, 31, 2000]
    gen_width = 48  # the pool has pages for these columns; the others of the table are never live
    for k in (None, 30):
        c = Case(80 + group, lengths, kv_heads * group, kv_heads, dim, gen_width, fp8, tables=1, k=k, sinks=True)
        wide = torch.full((1, width), -1, dtype=I32, device="cuda")
        wide[:, :gen_width] = c.table
        c.table = wide
        if k is not None:
            wider = torch.full((rows, kv_heads, width), -1, dtype=I32, device="cuda")
            wider[..., :k] = c.selected
            c.selected = wider
        assert rows * kv_heads * width * page_bytes >= 1 << 28
        c.check(lib)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads,kv_heads,dim,k", [(64, 8, 128, None), (16, 1, 64, None), (3, 3, 256, None), (40, 8, 64, 17), (32, 2, 128, 5)])
def test_probabilities_keep_16_bits(lib, heads, kv_heads, dim, k, fp8):
    """Up to 16 query heads a key head: a probability p goes into its product with the
    values as bf16(p) and bf16 of what that leaves, r = p - bf16(p), which float32 holds:
    |r| <= 2^-8 p, and off by 2^-8 |r| at most, 2^-16 p.  The rest as in
    assert_near_attention."""
    c = Case(90 + dim, [640, 1200, 64, 1000, 70, 1280], heads, kv_heads, dim, 20, fp8, k=k, sinks=True)
    c.run(lib)
    torch.cuda.synchronize()
    y, log, size, far = c.want()
    one = far * (dim + 8) * 2.0 ** -24 + 2.0 ** -22
    total = ((PAGE * k if k else 1280) / 4 + 64) * 2.0 ** -24
    err = size * (2.0 ** -16 + 2 * one + total)[..., None] * (1 + 2.0 ** -7) + np.abs(y) * 2.0 ** -8 + 2.0 ** -133
    d = np.abs(f64(c.out) - y)
    assert (d <= err).all(), f"{(d > err).sum()} of {d.size} off, {(d / err).max():.2f} times as far"
