"""Page tables and slot maps, store of keys and values, bounds and scores of pages on
the GPU against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
from kv_reference import PAGE, make_pools, values_of
from latent_reference import F32, assert_near_fp8, f64

pytestmark = pytest.mark.gpu

I32, I64, BF16 = torch.int32, torch.int64, torch.bfloat16


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32).cuda()


# --- page tables and slot maps


def plan_case(lib, cached, added, num_free, width, n, stride=None, stream=None):
    """Runs a plan over guarded buffers and checks every value and guard."""
    rng = np.random.default_rng(len(cached) * 1000 + n)
    requests = len(cached)
    order = rng.permutation(num_free + requests * width + 1).astype(np.int32)
    free, table = order[:num_free], order[num_free : num_free + requests * width].reshape(requests, width)
    want = ref.plan(cached, added, free, table, n)
    stride = width if stride is None else stride
    whole = torch.full((requests, stride), -7, dtype=I32)
    whole[:, :width] = torch.tensor(table.astype(np.int32))
    whole = whole.cuda()
    guard = [torch.full((size + 2,), -9, dtype=t, device="cuda") for size, t in ((n, I64), (n, I64), (n, I32), (n, I32),
                                                                                (requests + 1, I64), (1, I64))]
    inner = [g[1:-1] if g.dtype is I64 else g[1:-1] for g in guard]
    lib.idx_plan_batch(i32(cached).reshape(-1), i32(added).reshape(-1), i32(free).reshape(-1), whole[:, :width], *inner, stream=stream)
    torch.cuda.synchronize()
    assert (f64(whole[:, :width]) == want[0]).all()
    assert (whole[:, width:] == -7).all()
    for name, got, value in zip(("slots", "positions", "row_table", "seqlens", "starts"), inner, want[1:6]):
        assert (got.cpu().numpy() == value).all(), name
    assert int(inner[5]) == want[6]
    for g in guard:
        assert g[0] == -9 and g[-1] == -9


@pytest.mark.parametrize("cached,added,num_free,width,n", [
    ([0], [1], 1, 1, 1),
    ([5], [0], 0, 4, 3),
    ([63, 64, 65, 0], [1, 1, 1, 1], 8, 4, 4),
    ([0, 0, 0], [0, 0, 0], 2, 3, 5),
    ([0, 130, 64], [200, 1, 64], 5, 4, 300),       # padding rows
    ([0, 130, 64], [200, 1, 64], 5, 4, 100),       # more tokens than rows
    ([0, 10, 20], [300, 300, 300], 6, 8, 900),     # the free list runs out
    ([250, 100], [20, 10], 9, 4, 30),              # past the table
    ([-5, 3], [4, -6], 3, 2, 6),                   # negative lengths count as none
    ([300, 10], [5, 5], 3, 4, 10),                 # cached past the table already
    ([], [], 3, 4, 5),
    ([7, 9], [3, 0], 1, 0, 5),                     # a table without columns
    ([2 ** 31 - 1, 2 ** 31 - 10], [2, 2 ** 31 - 1], 1, 2, 9),  # lengths at int32's end
])
def test_plan(lib, cached, added, num_free, width, n):
    plan_case(lib, cached, added, num_free, width, n)


@pytest.mark.parametrize("requests,n,width", [(64, 64, 40), (255, 300, 9), (256, 5000, 9), (257, 5000, 9), (1023, 9000, 5), (1025, 12000, 5),
                                              (5000, 20000, 3), (65536, 70000, 2)])
def test_plan_many(lib, requests, n, width):
    rng = np.random.default_rng(requests)
    cached = rng.integers(0, 64 * width, requests)
    added = np.where(rng.random(requests) < 0.3, 0, rng.integers(0, 2 * n // requests + 2, requests))
    plan_case(lib, cached, added, requests, width, n, stride=width + 3)


def test_plan_optional_outputs(lib):
    """Each output may be left out."""
    cached, added, free = i32([10, 70]), i32([60, 3]), i32([5, 6, 7])
    full = [torch.empty(70, dtype=t, device="cuda") for t in (I64, I64, I32, I32)]
    full += [torch.empty(3, dtype=I64, device="cuda"), torch.empty(1, dtype=I64, device="cuda")]
    table = torch.zeros((2, 3), dtype=I32, device="cuda")
    lib.idx_plan_batch(cached, added, free, table, *full)
    for i in range(6):
        some = [torch.full_like(x, -3) for x in full]
        again = torch.zeros((2, 3), dtype=I32, device="cuda")
        lib.idx_plan_batch(cached, added, free, again, *[None if j == i else x for j, x in enumerate(some)])
        assert torch.equal(again, table)
        for j, (x, y) in enumerate(zip(some, full)):
            assert torch.equal(x, y) if j != i else (x == -3).all()
    none = torch.zeros((2, 3), dtype=I32, device="cuda")
    lib.idx_plan_batch(cached, added, free, none)  # pages alone
    assert torch.equal(none, table)


# --- store


@pytest.mark.parametrize("n,heads,dim,layout", [
    (1, 1, 64, "fused"), (1, 8, 128, "fused"), (3, 5, 256, "heads"), (64, 8, 128, "heads"), (257, 3, 64, "apart"), (100, 16, 256, "fused"),
    (1000, 7, 128, "apart"), (3001, 8, 128, "fused"),
])
@pytest.mark.parametrize("fp8", [True, False])
def test_store(lib, n, heads, dim, layout, fp8):
    gen = torch.Generator().manual_seed(n + heads)
    pages = -(-2 * n // PAGE) + 1
    k_pages, v_pages, scales = make_pools(gen, pages, heads, dim, fp8, layout)
    before = [x.clone() for x in (k_pages, v_pages, *scales)]
    size = torch.rand((n, 1, 1), generator=gen) * 4
    qkv = (torch.randn((n, 3 * heads, dim), generator=gen) * size).to(BF16)  # keys and values as parts of a wider row
    qkv[::7, heads] = 0  # keys of zeros
    whole = qkv.cuda()
    keys, values = whole[:, heads : 2 * heads], whole[:, 2 * heads :]
    slots = torch.randperm(pages * PAGE, generator=gen)[:n]
    if n > 2:
        slots[1], slots[2] = -1, pages * PAGE  # no slot of the pool
    call = lib.idx_store_kv_fp8 if fp8 else lib.idx_store_kv_bf16
    call(keys, values, slots.cuda(), k_pages, v_pages, *scales)
    torch.cuda.synchronize()
    kept = np.flatnonzero((slots.numpy() >= 0) & (slots.numpy() < pages * PAGE))
    at = slots.numpy()[kept]
    for i, (pool, x) in enumerate(((k_pages, qkv[:, heads : 2 * heads]), (v_pages, qkv[:, 2 * heads :]))):
        got = pool.cpu().view(torch.uint8 if fp8 else I32 if False else pool.dtype)
        old = before[i].cpu().view(got.dtype)
        if fp8:
            codes = got[at // PAGE, :, at % PAGE].reshape(-1, dim).numpy()
            stored = scales[i].cpu()[at // PAGE, :, at % PAGE].reshape(-1).numpy()
            y = f64(x)[kept].reshape(-1, dim)
            assert_near_fp8(codes, stored, y, np.zeros_like(y))
            left = scales[i].cpu().clone()
            left[at // PAGE, :, at % PAGE] = before[2 + i].cpu()[at // PAGE, :, at % PAGE]
            assert torch.equal(left, before[2 + i].cpu())
        else:
            assert torch.equal(got[at // PAGE, :, at % PAGE], x[kept])
        rest = got.clone()
        rest[at // PAGE, :, at % PAGE] = old[at // PAGE, :, at % PAGE]
        assert torch.equal(rest.view(torch.uint8), old.view(torch.uint8))


def test_store_agrees_with_the_key_store(lib):
    """Head by head the same bytes as idx_store_keys_fp8 (128 values)."""
    gen = torch.Generator().manual_seed(5)
    n, heads, pages = 200, 3, 8
    keys = (torch.randn((n, heads, 128), generator=gen) * torch.exp(6 * torch.randn((n, heads, 1), generator=gen))).to(BF16).cuda()
    slots = torch.randperm(pages * PAGE, generator=gen)[:n].cuda()
    k, v, (ks, vs) = make_pools(gen, pages, heads, 128, True, "heads")
    lib.idx_store_kv_fp8(keys, keys.flip(1), slots, k, v, ks, vs)
    for h in range(heads):
        one = torch.zeros((pages, PAGE * 132), dtype=torch.uint8, device="cuda")
        lib.idx_store_keys_fp8(keys[:, h].contiguous(), slots, one, one.data_ptr() + PAGE * 128, num_pages=pages)
        codes = one[:, : PAGE * 128].view(pages, PAGE, 128)
        scale = one[:, PAGE * 128 :].view(torch.float32)
        at, pos = slots // PAGE, slots % PAGE
        for got, s, head in ((k, ks, h), (v, vs, heads - 1 - h)):
            assert torch.equal(got.view(torch.uint8)[at, head, pos], codes[at, pos])
            assert torch.equal(s[at, head, pos], scale[at, pos])


def test_store_values_that_are_no_numbers(lib):
    """A NaN has no part in the amount and becomes +-448; huge and tiny vectors."""
    x = torch.zeros((6, 1, 64), dtype=BF16)
    x[0, 0, :4] = torch.tensor([float("nan"), 2.0, -4.0, 1.0])
    x[1, 0, :2] = torch.tensor([3.3e38, -3.3e38])
    x[2, 0, :2] = torch.tensor([1e-38, -2e-39])
    x[3] = float("nan")
    x[4, 0, :2] = torch.tensor([-0.0, 5.0])
    k, v, (ks, vs) = make_pools(torch.Generator().manual_seed(0), 1, 1, 64, True, "apart")
    lib.idx_store_kv_fp8(x.cuda(), x.cuda(), torch.arange(6).cuda(), k, v, ks, vs)
    got = values_of(k, ks)[0, 0]
    scale = f64(ks)[0, 0]
    assert scale[0] == np.float32(4) / np.float32(448) and abs(got[0, 0]) == 448 * scale[0] and got[0, 2] == -448 * scale[0]
    assert np.isclose(got[1, 0], f64(x)[1, 0, 0], rtol=2.0 ** -4) and np.isclose(got[2, 0], f64(x)[2, 0, 0], rtol=2.0 ** -4)
    assert scale[3] == 1 and (np.abs(got[3]) == 448).all() and scale[5] == 1 and (got[5] == 0).all()
    assert k.view(torch.uint8)[0, 0, 4, 0] == 0x80


@pytest.mark.parametrize("bits", [0x7F81, 0xFF81, 0x7FBF, 0x7FC0, 0xFFFF])
def test_store_nan_of_any_bits(lib, bits):
    """Wherever it stands in a vector, and whatever its bits, a NaN has no part in the amount."""
    x = torch.randn((64, 1, 64), generator=torch.Generator().manual_seed(9)).to(BF16)
    whole = x.clone()
    for t in range(64):
        x.view(torch.int16)[t, 0, t] = bits - 0x10000 if bits >= 0x8000 else bits
        whole[t, 0, t] = 0
    amax = whole.float().abs().amax(-1)[:, 0]
    k, v, (ks, vs) = make_pools(torch.Generator().manual_seed(0), 1, 1, 64, True, "apart")
    lib.idx_store_kv_fp8(x.cuda(), whole.cuda(), torch.arange(64).cuda(), k, v, ks, vs)
    assert torch.equal(ks.cpu()[0, 0], amax / 448) and torch.equal(vs.cpu()[0, 0], amax / 448)
    codes, others = k.view(torch.uint8).cpu()[0, 0], v.view(torch.uint8).cpu()[0, 0]
    at = torch.arange(64)
    assert (codes[at, at] == (0xFE if bits >= 0x8000 else 0x7E)).all()
    codes[at, at] = others[at, at]
    assert torch.equal(codes, others)  # (both ways round the quotient correctly)


# --- bounds


def bounds_case(lib, gen, lengths, first, heads, dim, fp8, width, layout="fused", row_table=None, spoil=None, num_pages=None):
    rows, tables = len(lengths), len(lengths) if row_table is None else 3
    pages = tables * width + 3
    k, _, scales = make_pools(gen, pages, heads, dim, fp8, layout)
    if spoil:
        spoil(k)
    table = torch.randperm(pages, generator=gen)[: tables * width].reshape(tables, width).to(I32)
    if num_pages is None:
        table[0, -1] = pages + 5  # outside the pool
        if width > 1:
            table[-1, 0] = -1
    near = torch.randn((pages, heads, 2, dim), generator=gen).to(BF16)
    out = near.cuda()
    args = dict(first=None if first is None else i32(first), row_table=None if row_table is None else i32(row_table), num_pages=num_pages)
    if fp8:
        lib.idx_page_bounds_fp8(k, scales[0], table.cuda(), i32(lengths), out, **args)
    else:
        lib.idx_page_bounds_bf16(k, table.cuda(), i32(lengths), out, **args)
    torch.cuda.synchronize()
    keys = values_of(k, scales[0] if fp8 else None)
    want = ref.bounds(keys, table.numpy(), np.zeros(rows) if first is None else first, lengths, f64(near),
                      pages if num_pages is None else num_pages, row_table)
    got = f64(out)
    if fp8:
        # outwards: no less (no more) than the float32 product, which is off by half a
        # step of 2^-24, and within a bf16 step of 2^-7 of it
        step = np.abs(want) * 2.0 ** -7 + 2.0 ** -133
        half = np.abs(want) * 2.0 ** -24
        touched = got != f64(near)
        lo, hi = got[:, :, 0], got[:, :, 1]
        assert (lo <= want[:, :, 0] + half[:, :, 0])[touched[:, :, 0]].all() and (hi >= want[:, :, 1] - half[:, :, 1])[touched[:, :, 1]].all()
        assert (np.abs(got - want) <= step + half).all()
    else:
        assert (got == want).all()


@pytest.mark.parametrize("lengths,first,heads,dim,width,layout", [
    ([1], None, 1, 64, 1, "fused"), ([64, 65, 0, 300], None, 3, 128, 5, "fused"), ([64, 65, 1, 300], [63, 64, 0, 250], 8, 256, 5, "heads"),
    ([500, 400, 320, 7], [500, 64, -3, 3], 2, 64, 5, "apart"), ([-4, 130], [0, 128], 5, 128, 3, "heads"),
    ([4000] * 3, [0, 3999, 2000], 16, 128, 60, "fused"),
])
@pytest.mark.parametrize("fp8", [True, False])
def test_bounds(lib, lengths, first, heads, dim, width, layout, fp8):
    bounds_case(lib, torch.Generator().manual_seed(len(lengths) + dim), lengths, first, heads, dim, fp8, width, layout)


@pytest.mark.parametrize("fp8", [True, False])
def test_bounds_row_table(lib, fp8):
    bounds_case(lib, torch.Generator().manual_seed(3), [200, 70, 190, 64], [0, 0, 64, 0], 4, 128, fp8, 4, row_table=[2, -1, 1, 3])


def test_bounds_pages_of_the_pool_alone(lib):
    """Ids of the pool's tensor but at or past num_pages are outside."""
    bounds_case(lib, torch.Generator().manual_seed(4), [640, 640], None, 2, 64, False, 10, num_pages=11)


def test_bounds_values_that_are_no_numbers(lib):
    """NaN has no part, infinities count as the largest finite value, what lies past a
    row's end has no part whatever it is."""
    def spoil(k):
        k[:, 0, 3, ::2] = float("nan")
        k[:, 1, :, 5] = float("nan")
        k[:, :, 7, 9] = float("inf")
        k[:, :, 8, 11] = -float("inf")
        k[:, :, 40:, 20:30] = float("inf")
        k[:, :, 40:, 30:] = float("nan")
        k[:, 0, :, 1] = float("inf")
    bounds_case(lib, torch.Generator().manual_seed(5), [40, 64 + 20, 3], None, 2, 64, False, 2, spoil=spoil)


def test_bounds_signalling_nan(lib):
    """Every bit pattern of a NaN, of either sign, is one."""
    def spoil(k):
        bits = k.view(torch.int16)
        bits[:, 0, 3, ::2] = 0x7F81
        bits[:, 0, 4, ::3] = 0xFF81 - 0x10000
        bits[:, 1, :, 5] = 0x7FBF
        bits[:, 1, 7, :] = 0xFFC0 - 0x10000
        bits[:, :, 60:, 1:9] = 0x7F81  # past the end of a row's last page
    bounds_case(lib, torch.Generator().manual_seed(6), [40, 64 + 20, 3], None, 2, 64, False, 2, spoil=spoil)


# --- scores


def scores_case(lib, gen, lengths, heads, kv_heads, dim, width, first=0, last=0, row_table=None, apart=None, spoil=None, tables=None):
    rows = len(lengths)
    tables = tables or (rows if row_table is None else 3)
    pages = tables * width + 2
    q = torch.randn((rows, heads, dim), generator=gen).to(BF16)
    lo = torch.randn((pages, kv_heads, dim), generator=gen)
    near = torch.stack((lo, lo + torch.rand((pages, kv_heads, dim), generator=gen) * 3), 2).to(BF16)
    table = torch.randperm(pages, generator=gen)[: tables * width].reshape(tables, width).to(I32)
    if width > 3:
        table[0, 2], table[-1, 3] = pages, -1
    if spoil:
        spoil(q, near)
    apart = -(-width // 4) * 4 if apart is None else apart
    whole = torch.full((rows, kv_heads, max(apart, 1)), -5.0, device="cuda")
    counts = torch.full((rows, kv_heads), -5, dtype=I32, device="cuda")
    lib.idx_page_scores(q.cuda(), near.cuda(), table.cuda(), i32(lengths), whole[:, :, :width], counts, first_pages=first, last_pages=last,
                        row_table=None if row_table is None else i32(row_table))
    torch.cuda.synchronize()
    want, size, live = ref.scores(f64(q), f64(near), table.numpy(), lengths, first, last, pages, row_table)
    got = f64(whole)
    assert (got[:, :, width:] == -5).all()
    got = got[:, :, :width]
    assert (counts.cpu().numpy() == live).all()
    assert (np.isposinf(got) == np.isposinf(want)).all() and (np.isneginf(got) == np.isneginf(want)).all()
    assert (np.isnan(got) == np.isnan(want)).all()
    fine = np.isfinite(want)
    # float32 sums of dim products, exact ones: a rounding each
    err = (dim + 2) * 2.0 ** -24 * size
    assert (np.abs(got - want)[fine] <= err[fine]).all(), np.abs(got - want)[fine].max()


@pytest.mark.parametrize("lengths,heads,kv_heads,dim,width,first,last", [
    ([1], 1, 1, 64, 1, 0, 0), ([0, 64, 65, 200], 8, 2, 128, 4, 0, 0), ([640, 100, 1, 320], 40, 8, 64, 10, 1, 2),
    ([64 * 40, 64 * 33, 64 * 129], 128, 1, 128, 131, 0, 1), ([64 * 20, 3], 34, 2, 256, 20, 0, 0), ([5000, 9000], 16, 16, 128, 300, 2, 0),
    ([300, 400], 7, 7, 128, 7, 5, 5), ([-3, 70], 4, 4, 64, 2, 0, 0),
])
def test_scores(lib, lengths, heads, kv_heads, dim, width, first, last):
    scores_case(lib, torch.Generator().manual_seed(heads + dim), lengths, heads, kv_heads, dim, width, first, last)


def test_scores_row_table_and_strides(lib):
    scores_case(lib, torch.Generator().manual_seed(1), [300, 70, 290, 64], 8, 4, 128, 5, row_table=[2, -1, 1, 3], apart=13)
    scores_case(lib, torch.Generator().manual_seed(2), [300, 70, 290, 64], 8, 4, 128, 5, tables=1)


def test_scores_without_columns(lib):
    scores_case(lib, torch.Generator().manual_seed(1), [300, 0], 8, 4, 128, 0)


def test_scores_many_rows(lib):
    """More rows than a grid's side holds, and more units than one round of it."""
    gen = torch.Generator().manual_seed(9)
    rows = 70000
    lengths = torch.randint(0, 65, (rows,), generator=gen).to(I32)
    q = torch.randn((rows, 16, 64), generator=gen).to(BF16)
    near = torch.randn((2, 16, 2, 64), generator=gen).sort(2).values.to(BF16)
    table = torch.tensor([[1]], dtype=I32)
    out = torch.empty((rows, 16, 1), device="cuda")
    lib.idx_page_scores(q.cuda(), near.cuda(), table.cuda(), lengths.cuda(), out)
    x = q.float()
    want = torch.maximum(x * near[1, :, 0].float(), x * near[1, :, 1].float()).double().sum(-1)
    want[lengths == 0] = -float("inf")
    got = out[..., 0].cpu().double()
    assert torch.equal(got.isinf(), want.isinf())
    fine = ~want.isinf()
    assert ((got - want)[fine].abs() <= 66 * 2.0 ** -24 * 64 * 16).all()


def test_scores_nan(lib):
    """A NaN of a query head or a page's bounds stays in its key head's scores."""
    gen = torch.Generator().manual_seed(3)
    q = torch.randn((2, 8, 128), generator=gen).to(BF16)
    near = torch.randn((12, 2, 2, 128), generator=gen).sort(2).values.to(BF16)
    q[0, 5, 17] = float("nan")
    near[4, 0, 1, 100] = float("nan")
    q[:, :4, 100] = q[:, :4, 100].abs() + 1
    table = torch.arange(12, dtype=I32).reshape(2, 6)
    out = torch.empty((2, 2, 6), device="cuda")
    lib.idx_page_scores(q.cuda(), near.cuda(), table.cuda(), i32([384, 384]), out)
    nan = out.isnan().cpu()
    assert nan[0, 1].all() and nan[0, 0].tolist() == [False] * 4 + [True, False] and not nan[1].any()


def test_scores_bound_every_key(lib):
    """The score of a page is at least that of each of its keys with each query head."""
    gen = torch.Generator().manual_seed(11)
    heads, kv_heads, dim, width = 24, 4, 128, 9
    for fp8 in (True, False):
        k, _, scales = make_pools(gen, width, kv_heads, dim, fp8)
        q = torch.randn((1, heads, dim), generator=gen).to(BF16)
        near = torch.zeros((width, kv_heads, 2, dim), dtype=BF16, device="cuda")
        table = torch.randperm(width, generator=gen).to(I32)[None].cuda()
        out = torch.empty((1, kv_heads, width), device="cuda")
        length = i32([64 * width - 20])
        if fp8:
            lib.idx_page_bounds_fp8(k, scales[0], table, length, near)
        else:
            lib.idx_page_bounds_bf16(k, table, length, near)
        lib.idx_page_scores(q.cuda(), near, table, length, out)
        keys = values_of(k, scales[0] if fp8 else None)[table[0].cpu().numpy()]  # [width, kv_heads, 64, dim]
        keys[-1, :, 44:] = 0
        x = f64(q).reshape(kv_heads, heads // kv_heads, dim)
        s = np.einsum("hgd,jhpd->hjgp", x, keys).reshape(kv_heads, width, -1)
        s[:, -1] = s[:, -1].reshape(kv_heads, -1, 64)[:, :, :44].max((1, 2))[:, None]
        size = np.einsum("hgd,jhpd->hjgp", np.abs(x), np.abs(keys)).max()
        assert (f64(out)[0] >= s.max(-1) - (dim + 2) * 2.0 ** -24 * size).all()


# --- together, on another stream, in a graph


def test_stream_of_another_device(lib):
    """A stream of another device than the tensors' is refused."""
    class Elsewhere:
        cuda_stream, device_index = 0, 1

    s = torch.zeros(1, dtype=I64, device="cuda")
    lens = torch.zeros(1, dtype=I32, device="cuda")
    table = torch.zeros((1, 1), dtype=I32, device="cuda")
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        lib.idx_plan_batch(lens, lens, lens, table, s, stream=Elsewhere())
    with pytest.raises(TypeError):
        lib.idx_plan_batch(lens, lens, lens, table, s, stream="elsewhere".split())


def test_on_another_stream_and_in_a_graph(lib):
    """A step's operators, captured once and replayed as the lengths grow, with eager
    work between the replays; every replay against the eager result on another stream."""
    gen = torch.Generator().manual_seed(21)
    requests, heads, kv_heads, dim, width = 5, 16, 4, 64, 6
    pages = requests * width
    free_all = torch.randperm(pages, generator=gen).to(I32).cuda()
    q = torch.randn((requests, heads, dim), generator=gen).to(BF16).cuda()
    kv = torch.randn((requests, 2, kv_heads, dim), generator=gen).to(BF16).cuda()
    start = torch.tensor([0, 63, 64, 100, 127], dtype=I32)

    def fresh():
        k, v, scales = make_pools(torch.Generator().manual_seed(1), pages, kv_heads, dim, True)
        table = torch.zeros((requests, width), dtype=I32, device="cuda")
        at = 0
        for r, c in enumerate(start.tolist()):  # pages of what is cached already
            for j in range(-(-c // PAGE)):
                table[r, j] = free_all[at]
                at += 1
        return dict(k=k, v=v, ks=scales[0], vs=scales[1], table=table, cached=start.cuda(), added=torch.ones(requests, dtype=I32, device="cuda"),
                    free=free_all[at:].clone(), slots=torch.zeros(requests, dtype=I64, device="cuda"),
                    rows=torch.zeros(requests, dtype=I32, device="cuda"), lens=torch.zeros(requests, dtype=I32, device="cuda"),
                    positions=torch.zeros(requests, dtype=I64, device="cuda"), taken=torch.zeros(1, dtype=I64, device="cuda"),
                    near=torch.zeros((pages, kv_heads, 2, dim), dtype=BF16, device="cuda"),
                    scores=torch.zeros((requests, kv_heads, 8), device="cuda")[..., :width],
                    counts=torch.zeros((requests, kv_heads), dtype=I32, device="cuda"))

    def step(s, stream=None):
        lib.idx_plan_batch(s["cached"], s["added"], s["free"], s["table"], s["slots"], s["positions"], s["rows"], s["lens"], None, s["taken"],
                           stream=stream)
        lib.idx_store_kv_fp8(kv[:, 0], kv[:, 1], s["slots"], s["k"], s["v"], s["ks"], s["vs"], stream=stream)
        lib.idx_page_bounds_fp8(s["k"], s["ks"], s["table"], s["lens"], s["near"], stream=stream)
        lib.idx_page_scores(q, s["near"], s["table"], s["lens"], s["scores"], s["counts"], row_table=s["rows"], last_pages=1, stream=stream)

    def advance(s):  # what a scheduler does between steps
        s["cached"] += 1
        s["free"].copy_(torch.roll(s["free"], -int(s["taken"])))

    eager, other = fresh(), torch.cuda.Stream()
    static = fresh()
    graph = torch.cuda.CUDAGraph()
    keep = {name: x.clone() for name, x in static.items()}
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(static)
    for name, x in static.items():
        x.copy_(keep[name])
    for _ in range(5):
        kv += 0.125
        kv.mul_(-1)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            step(eager, other)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(eager[name].contiguous().view(torch.uint8), static[name].contiguous().view(torch.uint8)), name
        assert (eager["lens"].cpu() == eager["cached"].cpu() + 1).all()
        advance(eager)
        advance(static)


# --- more work than a launch has workgroups: every loop goes round again


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("requests,n,each", [(1000, 140000, 13000), (2000, 600000, 600)])
def test_plan_of_more_rows_than_its_grid(lib, requests, n, each):
    """Rows, and for long prompts new pages, past those of the first round."""
    threads = 256 if requests <= 1024 else 1024
    round_ = 2 * cus() * threads
    rng = np.random.default_rng(requests)
    added = rng.integers(each // 2, each + 1, requests)
    cached = rng.integers(0, 200, requests)
    width = -(-(each + 200) // PAGE) + 1
    pages = int((-(-(cached + added) // PAGE) - -(-cached // PAGE)).sum())
    assert round_ < n <= added.sum() and (threads > 256 or pages > round_)
    plan_case(lib, cached, added, pages - 5, width, n)


def test_plan_of_pages_alone(lib):
    """More new pages than the threads of the one workgroup that hands them out."""
    requests, width = 300, 40
    added = np.full(requests, 64 * width - 3)
    cached = np.arange(requests) % 3
    free = np.random.default_rng(3).permutation(requests * width).astype(np.int32)
    table = torch.full((requests, width), -7, dtype=I32, device="cuda")
    lib.idx_plan_batch(i32(cached), i32(added), i32(free), table)
    want = ref.plan(cached, added, free, np.full((requests, width), -7), 0)
    assert want[6] > 1024 and (table.cpu().numpy() == want[0]).all()


@pytest.mark.parametrize("fp8,dim,heads", [(True, 64, 4), (True, 128, 8), (True, 256, 2), (False, 64, 4), (False, 128, 8), (False, 256, 2)])
@pytest.mark.parametrize("size", ["below", "at", "round"])
def test_store_of_many_tokens(lib, fp8, dim, heads, size):
    """Just below and just at the 16 MiB of outputs that pass the caches by, and more
    vectors than one round of the grid takes."""
    far = -(-(1 << 24) // (2 * dim if fp8 else 4 * dim))        # vectors
    round_ = 16 * cus() * 2 * 4 * (64 // (dim // 8))
    vectors = {"below": far - heads, "at": far, "round": round_ + 5 * heads}[size]
    n = vectors // heads
    assert n * heads == vectors and (vectors >= far) == (size != "below") and (vectors > round_) == (size == "round")
    gen = torch.Generator(device="cuda").manual_seed(dim + heads)
    pages = -(-n // PAGE) + 2
    if fp8:
        k, v = (torch.full((pages, heads, PAGE, dim), 0x3A, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        scales = tuple(torch.full((pages, heads, PAGE), -3.0, device="cuda") for _ in range(2))
    else:
        k, v = (torch.full((pages, heads, PAGE, dim), 77.0, dtype=BF16, device="cuda") for _ in range(2))
        scales = ()
    x = (torch.randn((n, 2, heads, dim), generator=gen, device="cuda") * (torch.rand((n, 2, heads, 1), generator=gen, device="cuda") * 4)).to(BF16)
    slots = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:n]
    slots[1], slots[n - 2] = -1, pages * PAGE
    (lib.idx_store_kv_fp8 if fp8 else lib.idx_store_kv_bf16)(x[:, 0], x[:, 1], slots, k, v, *scales)
    kept = (slots >= 0) & (slots < pages * PAGE)
    page, at = slots[kept] // PAGE, slots[kept] % PAGE
    rest = torch.ones((pages, PAGE), dtype=torch.bool, device="cuda")
    rest[page, at] = False
    rest = rest[:, None].expand(pages, heads, PAGE)
    for i, pool in enumerate((k, v)):
        want = x[kept, i]
        if not fp8:
            assert torch.equal(pool[page, :, at], want) and (pool[rest] == 77).all()
            continue
        assert_near_fp8(pool.view(torch.uint8)[page, :, at].reshape(-1, dim).cpu().numpy(), scales[i][page, :, at].reshape(-1).cpu().numpy(),
                        f64(want).reshape(-1, dim), np.zeros((want.shape[0] * heads, dim)))
        assert (pool.view(torch.uint8)[rest] == 0x3A).all() and (scales[i][rest] == -3).all()


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads,dim", [(4, 64), (3, 128), (5, 256)])
def test_bounds_of_more_pages_than_a_grid(lib, fp8, heads, dim):
    """So many rows that each has one column of workgroups, which go along its pages:
    rows of three tables, pages outside the pool among them."""
    rows, width = 16 * cus() // -(-heads // 4) + 200, 7
    assert rows * -(-heads // 4) >= 16 * cus() and width * heads > 4 * -(-heads // 4)
    rng = np.random.default_rng(heads)
    which = rng.integers(-1, 4, rows)
    lengths = np.choose(np.clip(which, 0, 2), [64 * width, 64 * width - 40, 130])  # (rows of a table agree)
    first = rng.integers(0, 130, rows)
    first[:6] = 0
    which[:6] = [0, 1, 2, 0, 1, 2]
    lengths[:6] = [64 * width, 64 * width - 40, 130] * 2
    bounds_case(lib, torch.Generator().manual_seed(heads), lengths, first, heads, dim, fp8, width, row_table=which)


def test_scores_of_more_units_than_a_grid(lib):
    """Units past the 2^20 of a round, whose bounds come to the LDS places of earlier ones."""
    rows, heads, kv_heads, dim, width, pages = 64, 16, 8, 64, 16 * 9000, 50
    blocks = -(-(-(-width // 16) * kv_heads) // 4)
    assert rows * blocks > 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((rows, heads, dim), generator=gen, device="cuda").to(BF16)
    near = torch.randn((pages, kv_heads, 2, dim), generator=gen, device="cuda").sort(2).values.to(BF16)
    table = torch.randint(0, pages + 1, (1, width), generator=gen, device="cuda").to(I32)  # (one id outside the pool)
    lengths = torch.full((rows,), 64 * width, dtype=I32, device="cuda")
    lengths[::3] -= 64 * 777 + 5
    out = torch.full((rows, kv_heads, width), -5.0, device="cuda")
    counts = torch.full((rows, kv_heads), -5, dtype=I32, device="cuda")
    lib.idx_page_scores(q, near, table, lengths, out, counts, last_pages=1)
    x = q.double().reshape(rows, kv_heads, 1, heads // kv_heads, dim)
    lo, hi = (near[:, :, i].double().transpose(0, 1)[None, :, :, None] for i in range(2))  # [1, kv heads, pages, 1, dim]
    best = torch.maximum(x * lo, x * hi)
    want = torch.cat((best.sum(-1).amax(-1), torch.full((rows, kv_heads, 1), float("nan"), device="cuda")), 2)
    err = (dim + 2) * 2.0 ** -24 * torch.cat((best.abs().sum(-1).amax(-1), torch.zeros((rows, kv_heads, 1), device="cuda")), 2)
    at = table[0].long()
    j = torch.arange(width, device="cuda")
    for b in range(rows):
        live = -(-int(lengths[b]) // PAGE)
        assert (counts[b] == live).all()
        assert torch.isneginf(out[b, :, live:]).all() and torch.isposinf(out[b, :, live - 1]).all()
        inside = (j < live - 1) & (at < pages)
        assert ((out[b].double() - want[b][:, at]).abs() <= err[b][:, at])[:, inside].all(), b
        assert out[b][:, (j < live - 1) & (at == pages)].isnan().all()
