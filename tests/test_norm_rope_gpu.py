"""Norm, rotation, paged store and read back on the GPU against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from latent_reference import F32, PAGE, assert_near_bf16, assert_near_fp8, e4m3_values, f64, inv_freq, norm_rope, vectors

pytestmark = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("n,heads,dim,rope,opts", [
    (1, 1, 128, 64, {}),
    (1, 64, 128, 64, {"halves": True}),
    (3, 5, 64, 64, {}),
    (7, 13, 256, 32, {"leading": True}),
    (5, 64, 512, 64, {}),
    (33, 17, 512, 512, {"halves": True}),
    (64, 64, 128, 96, {"halves": True, "leading": True}),
    (130, 65, 128, 16, {"weight": False}),
    (9, 3, 512, 0, {}),
    (9, 130, 512, 48, {"norm": False, "halves": True}),
    (700, 40, 512, 64, {}),
    (2000, 70, 128, 128, {}),
])
@pytest.mark.parametrize("strided", [False, True])
def test_norm_rope(lib, n, heads, dim, rope, opts, strided):
    rng = np.random.default_rng(n * heads + dim)
    opts = dict(opts)
    weight = torch.from_numpy(1 + rng.standard_normal(dim).astype(np.float32) * 0.3)
    if not opts.get("norm", True) or opts.pop("weight", None) is False:
        weight = None
    x = vectors(rng, (n, heads, dim))
    freq = inv_freq(rope // 2) if rope else None
    positions = torch.from_numpy(rng.integers(-5, 1 << 20, n)) if rope else None
    if n > 4 and rope:
        positions[1:4] = torch.tensor([0, 1, (1 << 31) + 12345])
    y, size = norm_rope(x, positions, freq, weight, eps=1e-5, **opts)
    xd = x.cuda()
    if strided:
        wide = torch.full((n, heads * dim + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        wide[:, :heads * dim] = xd.reshape(n, -1)
        xd = wide[:, :heads * dim].unflatten(1, (heads, dim))
    out = torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda")
    lib.idx_norm_rope(xd, dev(positions), dev(freq), out, weight=dev(weight), eps=1e-5, **opts)
    assert_near_bf16(out, y, size)
    if not strided:  # in place
        lib.idx_norm_rope(xd, dev(positions), dev(freq), xd, weight=dev(weight), eps=1e-5, **opts)
        assert torch.equal(xd.view(torch.int16), out.view(torch.int16))


def test_norm_rope_turns_back(lib):
    """A rotation with negated frequencies undoes one: off by two roundings to
    bf16 of the pair and both float32 parts."""
    rng = np.random.default_rng(5)
    x = vectors(rng, (50, 8, 128)).cuda()
    positions = torch.from_numpy(rng.integers(0, 1 << 20, 50)).cuda()
    freq = inv_freq(32).cuda()
    there, back = torch.empty_like(x), torch.empty_like(x)
    lib.idx_norm_rope(x, positions, freq, there, norm=False)
    lib.idx_norm_rope(there, positions, -freq, back, norm=False)
    a = f64(x)
    size = np.abs(a)
    size[..., 64:] = np.repeat(np.abs(a[..., 64::2]) + np.abs(a[..., 65::2]), 2, -1)
    # each of the pair's two values is within 2^-8 of itself after the first
    # rounding; the turn back passes their sum on, and rounds again
    assert (np.abs(f64(back) - a) <= size * (2 * 2.0 ** -8 + 2.0 ** -15) * 1.01 + 2.0 ** -130).all()


def pool_of(rng, pages, dim, fp8, layout):
    """(kv tensor, kscale or None, kv stride, kscale stride) of canary bytes."""
    if not fp8:
        stride = 2 * PAGE * dim + (32 if layout == "padded" else 0)
        return torch.from_numpy(rng.integers(0, 256, pages * stride, dtype=np.uint8)), None, stride, 0
    if layout == "fused":
        stride = PAGE * (dim + 4)
        return torch.from_numpy(rng.integers(0, 256, pages * stride, dtype=np.uint8)), None, stride, stride
    stride, ks = PAGE * dim + (48 if layout == "padded" else 0), 256 + (12 if layout == "padded" else 0)
    scales = torch.from_numpy(rng.random(pages * ks // 4 + 8).astype(np.float32))
    return torch.from_numpy(rng.integers(0, 256, pages * stride, dtype=np.uint8)), scales, stride, ks


def split_pool(kv, scales, pages, dim, fp8, stride, ks):
    """Values and scales by slot, and a copy of all bytes with the slots cleared."""
    kv = kv.cpu().numpy()
    width = dim if fp8 else 2 * dim
    rows = np.stack([kv[g * stride + i * width: g * stride + (i + 1) * width] for g in range(pages) for i in range(PAGE)])
    if not fp8:
        return rows.view(np.uint16), None
    src = kv.view(np.uint8) if scales is None else scales.cpu().numpy().view(np.uint8)
    at = PAGE * dim if scales is None else 0
    s = np.concatenate([src[at + g * ks: at + g * ks + 256].view(np.float32) for g in range(pages)])
    return rows, s


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("n,dim,rope,layout,opts", [
    (1, 128, 64, "fused", {"halves": True}),
    (1, 512, 64, "fused", {}),
    (3, 512, 0, "split", {}),
    (65, 128, 32, "padded", {"leading": True}),
    (1000, 512, 64, "fused", {}),
    (777, 512, 512, "padded", {"halves": True}),
    (700, 128, 128, "split", {"norm": False}),
    (9000, 512, 64, "fused", {}),
    (33000, 128, 64, "split", {"halves": True}),
])
def test_norm_rope_store_and_load(lib, fp8, n, dim, rope, layout, opts):
    """The stored slots hold the quantised vectors, every other byte of the pool
    is left as it was, and the read back gives their values."""
    rng = np.random.default_rng(n + dim)
    pages = n // PAGE + 3
    weight = None if not opts.get("norm", True) else torch.from_numpy(1 + rng.standard_normal(dim).astype(np.float32) * 0.3)
    x = vectors(rng, (n, dim))
    freq = inv_freq(rope // 2) if rope else None
    positions = torch.from_numpy(rng.integers(0, 1 << 20, n)) if rope else None
    slots = rng.permutation(pages * PAGE)[:n].astype(np.int64)
    if n > 10:
        slots[rng.random(n) < 0.05] = -1
        slots[rng.random(n) < 0.02] = pages * PAGE + rng.integers(0, 100)
        slots[4], slots[5] = np.iinfo(np.int64).max, np.iinfo(np.int64).min
    kept = (slots >= 0) & (slots < pages * PAGE)
    kv, scales, stride, ks = pool_of(rng, pages, dim, fp8, layout)
    kvd, sd, xd, slotd = kv.cuda(), dev(scales), x.cuda(), torch.from_numpy(slots).cuda()
    kscale = sd if sd is not None else kvd.data_ptr() + PAGE * dim
    common = dict(num_pages=pages, kv_page_stride=stride)
    if fp8:
        lib.idx_norm_rope_store_fp8(xd, dev(positions), dev(freq), slotd, kvd, kscale, weight=dev(weight),
                                    kscale_page_stride=ks, **common, **opts)
    else:
        lib.idx_norm_rope_store_bf16(xd, dev(positions), dev(freq), slotd, kvd, weight=dev(weight), **common, **opts)
    y, size = norm_rope(x, positions, freq, weight, **opts)
    got, got_s = split_pool(kvd, sd, pages, dim, fp8, stride, ks)
    if fp8:
        assert_near_fp8(got[slots[kept]], got_s[slots[kept]], y[kept], size[kept])
    else:
        bits = torch.from_numpy(got[slots[kept]].view(np.int16)).view(torch.bfloat16)
        assert_near_bf16(bits, y[kept], size[kept])
    # put the old bytes back into the stored slots: nothing else has changed
    back = kvd.cpu().numpy().copy()
    width = dim if fp8 else 2 * dim
    for s in slots[kept]:
        g, i = divmod(int(s), PAGE)
        a = g * stride + i * width
        back[a: a + width] = kv.numpy()[a: a + width]
        if fp8 and scales is None:
            a = g * ks + PAGE * dim + 4 * i
            back[a: a + 4] = kv.numpy()[a: a + 4]
    assert np.array_equal(back, kv.numpy())
    if scales is not None:
        other = np.ones(len(scales), bool)
        for s in slots[kept]:
            other[int(s) // PAGE * ks // 4 + int(s) % PAGE] = False
        assert np.array_equal(sd.cpu().numpy()[other], scales.numpy()[other])
    # read back, in another order, a slot twice, rows of skipped slots left
    take = np.concatenate([slots, slots[:3]])
    take = take[rng.permutation(len(take))]
    wide = torch.full((len(take), dim + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :dim]
    if fp8:
        lib.idx_load_slots_fp8(kvd, kscale, torch.from_numpy(take).cuda(), out, kscale_page_stride=ks, **common)
    else:
        lib.idx_load_slots_bf16(kvd, torch.from_numpy(take).cuda(), out, **common)
    ok = (take >= 0) & (take < pages * PAGE)
    w = wide.float().cpu().numpy()
    assert (w[:, dim:] == 3.0).all() and (w[~ok] == 3.0).all()
    if fp8:
        want = e4m3_values()[got[take[ok]]] * got_s[take[ok], None].astype(np.float64)
        # a float32 product, rounded to bf16
        assert (np.abs(w[ok][:, :dim] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -134).all()
    else:
        assert np.array_equal(out.cpu().view(torch.int16).numpy()[ok].view(np.uint16), got[take[ok]])


@pytest.mark.parametrize("n", [1, 1000, 5000])
def test_plain_store_gives_the_key_stores_bytes(lib, n):
    """Without norm and rotation the 128-value store writes what
    idx_store_keys_fp8 and the oracle's quantiser write, over all magnitudes."""
    rng = np.random.default_rng(n)
    k = rng.standard_normal((n, 128)).astype(np.float32) * np.float32(10.0) ** rng.integers(-30, 30, (n, 1)).astype(np.float32)
    k[rng.random(n) < 0.03] = 0.0
    k[rng.random((n, 128)) < 0.01] = -0.0
    x = torch.from_numpy(k).to(torch.bfloat16)
    pages = n // PAGE + 1
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n]).cuda()
    a = torch.zeros(pages * 8448, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    lib.idx_norm_rope_store_fp8(x.cuda(), None, None, slots, a, a.data_ptr() + 8192, norm=False, num_pages=pages)
    lib.idx_store_keys_fp8(x.cuda(), slots, b, b.data_ptr() + 8192, num_pages=pages)
    assert torch.equal(a, b)
    codes, scales = oracle.quantize_keys_fp8(x.view(torch.int16).numpy().view(np.uint16))
    got, got_s = split_pool(a, None, pages, 128, True, 8448, 8448)
    assert np.array_equal(got[slots.cpu().numpy()], codes) and np.array_equal(got_s[slots.cpu().numpy()], scales)


def test_plain_latent_store_is_the_float32_recipe(lib):
    """512 values: codes and scales are those of the recipe in float32, bit for
    bit (no norm, no rotation: no other rounding comes before)."""
    rng = np.random.default_rng(8)
    n, pages = 3000, 60
    x = (torch.from_numpy(rng.standard_normal((n, 512)) * 10.0 ** rng.integers(-30, 30, (n, 1)))).to(torch.bfloat16)
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n])
    kv = torch.zeros((pages, PAGE, 512), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((pages, PAGE), device="cuda")
    lib.idx_norm_rope_store_fp8(x.cuda(), None, None, slots.cuda(), kv, ks, norm=False, num_pages=pages,
                                kv_page_stride=PAGE * 512, kscale_page_stride=256)
    scale = x.float().abs().amax(-1) / 448
    codes = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ks.cpu().view(-1)[slots], scale)
    assert torch.equal(kv.cpu().view(-1, 512)[slots], codes)


def test_far_pages(lib):
    """Slots whose bytes lie past 4 GiB of the pool."""
    pages = 140000  # 4.6 GB
    kv = torch.empty(pages * 33024, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    x = vectors(rng, (40, 512))
    slots = torch.from_numpy(pages * PAGE - 1 - rng.permutation(4000)[:40])
    lib.idx_norm_rope_store_fp8(x.cuda(), None, None, slots.cuda(), kv, kv.data_ptr() + 32768, num_pages=pages)
    out = torch.zeros((40, 512), dtype=torch.bfloat16, device="cuda")
    lib.idx_load_slots_fp8(kv, kv.data_ptr() + 32768, slots.cuda(), out, num_pages=pages)
    y, size = norm_rope(x, None, None)
    scale = np.abs(y).max(-1, keepdims=True) / 448
    # e4m3's half step, the bf16 rounding of the product, the float32 part
    tol = np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * 1.01 + np.abs(y) * 2.0 ** -7
    assert (np.abs(f64(out) - y) <= tol).all()


def test_other_stream_and_graph(lib):
    """Calls follow the stream that they are given; a captured store and load
    replay on what their buffers hold then."""
    rng = np.random.default_rng(6)
    n, pages = 300, 8
    x = vectors(rng, (n, 512)).cuda()
    positions = torch.from_numpy(rng.integers(0, 1 << 20, n)).cuda()
    freq = inv_freq(32).cuda()
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n]).cuda()
    kv = torch.zeros(pages * 33024, dtype=torch.uint8, device="cuda")
    out = torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda")

    def both(stream=None):
        lib.idx_norm_rope_store_fp8(x, positions, freq, slots, kv, kv.data_ptr() + 32768, num_pages=pages, stream=stream)
        lib.idx_load_slots_fp8(kv, kv.data_ptr() + 32768, slots, out, num_pages=pages, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(side)
    side.synchronize()
    want = out.clone()
    both()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        x.copy_(vectors(np.random.default_rng(70 + k), (n, 512)))
        positions.add_(1000)
        kv.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        kv.zero_()
        out.zero_()
        both()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


@pytest.mark.parametrize("halves", [False, True])
def test_far_positions_still_turn(lib, halves):
    """Up to |p| = 2^53 the rotation is one, whatever is left of the angle: pairs
    keep their length.  Its cos and sin are float32 (3 2^-24 of the length), and
    the outputs are rounded to bf16 (2^-9 of it at most in each of two values)."""
    rng = np.random.default_rng(21)
    n, dim = 64, 128
    far = [2 ** 40, 2 ** 50 + 3, 2 ** 51 - 1, 2 ** 52 + 1, 2 ** 53, 2 ** 53 - 1]
    positions = torch.tensor([rng.choice(far) * rng.choice([-1, 1]) for _ in range(n)], dtype=torch.int64)
    freq = torch.cat([torch.tensor([1.0]), torch.from_numpy(rng.random(31).astype(np.float32))])
    x = torch.from_numpy(rng.standard_normal((n, 1, dim))).to(torch.bfloat16)
    out = torch.empty((n, 1, dim), dtype=torch.bfloat16, device="cuda")
    lib.idx_norm_rope(x.cuda(), positions.cuda(), freq.cuda(), out, norm=False, halves=halves)
    was, got = (t.double().cpu().numpy()[:, 0, dim - 64:] for t in (x, out))
    pairs = (lambda v: np.hypot(v[:, :32], v[:, 32:])) if halves else (lambda v: np.hypot(v[:, 0::2], v[:, 1::2]))
    assert (np.abs(pairs(got) - pairs(was)) <= pairs(was) * (2.0 ** -8 + 2.0 ** -21)).all()
    assert torch.equal(out[..., : dim - 64].cpu(), x[..., : dim - 64])


@pytest.mark.parametrize("n", [1, 7, 600])
def test_plain_store_of_nan_and_inf(lib, n):
    """Values next to the ends of the type, infinities and NaN: the scales and,
    where the quotient is a number, the codes are idx_store_keys_fp8's (which
    leaves the codes of NaN and infinities open); a quotient that is none (NaN,
    or infinity over infinity) becomes +-448 with the value's sign."""
    rng = np.random.default_rng(n)
    x = torch.from_numpy(rng.standard_normal((n, 128)) * 10.0 ** rng.integers(-38, 38, (n, 1))).to(torch.bfloat16)
    odd = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), 3.3e38, -3.3e38, 1e-38, -1e-40, 0.0, -0.0]).to(torch.bfloat16)
    where = torch.from_numpy(rng.random((n, 128)) < 0.01)
    x[where] = odd[torch.from_numpy(rng.integers(0, len(odd), int(where.sum())))]
    x[0, 5] = float("nan")
    pages = n // PAGE + 1
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n])
    a = torch.zeros(pages * 8448, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    lib.idx_norm_rope_store_fp8(x.cuda(), None, None, slots.cuda(), a, a.data_ptr() + 8192, norm=False, num_pages=pages)
    lib.idx_store_keys_fp8(x.cuda(), slots.cuda(), b, b.data_ptr() + 8192, num_pages=pages)
    (codes, scales), (keys, key_scales) = (split_pool(t, None, pages, 128, True, 8448, 8448) for t in (a, b))
    assert np.array_equal(scales, key_scales)
    none = (x.isnan() | (x.isinf() & torch.from_numpy(np.isinf(scales[slots.numpy()]))[:, None])).numpy()
    codes, keys = codes[slots.numpy()], keys[slots.numpy()]
    sign = ((x.view(torch.int16).numpy() >> 15) & 1).astype(np.uint8) << 7
    assert np.array_equal(codes[~none], keys[~none]) and np.array_equal(codes[none], (sign | 0x7E)[none])


def stored_bytes(lib, x, positions, freq, weight, slots, pages, dim, **opts):
    """Codes and scales by slot after a store into a pool of zeros."""
    kv = torch.zeros(pages * PAGE * (dim + 4), dtype=torch.uint8, device="cuda")
    lib.idx_norm_rope_store_fp8(x, positions, freq, slots, kv, kv.data_ptr() + PAGE * dim, num_pages=pages, weight=weight, **opts)
    return split_pool(kv, None, pages, dim, True, PAGE * (dim + 4), PAGE * (dim + 4))


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("neighbours", ["nan", "inf", "zero", "tiny", "huge", "none"])
@pytest.mark.parametrize("halves", [False, True])
def test_a_tokens_bytes_are_its_own(lib, dim, neighbours, halves):
    """What a token is stored as depends on nothing but the token: not on what
    stands beside it in the batch (padding without a slot included), nor on
    where the batch ends."""
    rng = np.random.default_rng(dim + len(neighbours))
    n, pages, eps = 203, 4, 0.0  # (eps 0: the factor of a zero vector is infinite)
    x = torch.from_numpy(rng.standard_normal((n, dim)) * np.exp(rng.standard_normal((n, 1)))).to(torch.bfloat16)
    weight = torch.from_numpy(1 + rng.standard_normal(dim).astype(np.float32) * 0.3).cuda()
    freq = inv_freq(32).cuda()
    positions = torch.from_numpy(rng.integers(0, 1 << 20, n))
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n])
    odd = torch.from_numpy(rng.random(n) < 0.25)
    odd[:8] = torch.tensor([1, 0, 0, 0, 0, 1, 0, 0]).bool()
    mixed = x.clone()
    fill = {"nan": float("nan"), "inf": float("inf"), "zero": 0.0, "tiny": 1e-30, "huge": 3e38}.get(neighbours)
    if fill is None:
        odd[:] = False
    else:
        mixed[odd] = fill
    skipped = slots.clone()
    skipped[odd & torch.from_numpy(rng.random(n) < 0.5)] = -1
    kept = ~odd
    call = dict(eps=eps, halves=halves)
    codes, scales = stored_bytes(lib, mixed.cuda(), positions.cuda(), freq, weight, skipped.cuda(), pages, dim, **call)
    for t in range(n):  # alone, a call each
        if kept[t]:
            one = [v[t: t + 1].cuda() for v in (x, positions, slots)]
            c, s = stored_bytes(lib, one[0], one[1], freq, weight, one[2], pages, dim, **call)
            at = int(slots[t])
            assert s[at] == scales[at] and np.array_equal(c[at], codes[at]), f"token {t}"
    at = slots[kept].numpy()
    y, size = norm_rope(x[kept], positions[kept], freq.cpu(), weight.cpu(), eps=eps, halves=halves)
    assert_near_fp8(codes[at], scales[at], y, size)


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("of_x,of_w", [(2.0 ** 50, 2.0 ** 90), (2.0 ** 50, 2.0 ** 62), (2.0 ** -55, 2.0 ** -90), (2.0 ** -55, 2.0 ** -30), (2.0 ** -59, 2.0 ** -95),
                                       (2.0 ** -40, 2.0 ** 100), (2.0 ** 40, 2.0 ** -100)])
def test_store_at_the_ends_of_the_range(lib, dim, halves, of_x, of_w):
    """x times the weight leaves float32's range, or its normal range, where the
    normed value times it does not: the stored values are those of the latter."""
    rng = np.random.default_rng(dim)
    n, pages = 101, 2
    # (magnitudes within 2^+-1 of one another: no value leaves the normal range)
    x = torch.from_numpy(of_x * (1 + rng.random((n, dim))) * rng.choice([-1, 1], (n, dim))).to(torch.bfloat16)
    weight = torch.from_numpy((of_w * (1 + rng.random(dim))).astype(np.float32))
    freq, positions = inv_freq(32), torch.from_numpy(rng.integers(0, 1 << 20, n))
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n])
    codes, scales = stored_bytes(lib, x.cuda(), positions.cuda(), freq.cuda(), weight.cuda(), slots.cuda(), pages, dim, eps=0.0, halves=halves)
    y, size = norm_rope(x, positions, freq, weight, eps=0.0, halves=halves)
    assert_near_fp8(codes[slots.numpy()], scales[slots.numpy()], y, size)


@pytest.mark.parametrize("halves", [False, True])
def test_frequencies_that_are_no_numbers(lib, halves):
    """A frequency that is NaN or infinite has no cos and sin: the values it
    turns become NaN, and no others.  (Position 0 times infinity is NaN too.)"""
    rng = np.random.default_rng(22)
    n, heads, dim = 9, 3, 128
    x = torch.from_numpy(rng.standard_normal((n, heads, dim))).to(torch.bfloat16)
    positions = torch.from_numpy(rng.integers(0, 1000, n))
    positions[2] = 0
    freq = inv_freq(16)
    for j, v in ((1, float("nan")), (4, float("inf")), (9, -float("inf"))):
        freq[j] = v
    out = torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda")
    lib.idx_norm_rope(x.cuda(), positions.cuda(), freq.cuda(), out, halves=halves)
    none = torch.zeros(dim, dtype=torch.bool)
    for j in (1, 4, 9):
        none[[dim - 32 + j, dim - 16 + j] if halves else [dim - 32 + 2 * j, dim - 31 + 2 * j]] = True
    assert torch.equal(out.isnan().cpu(), none.expand(n, heads, dim))


@pytest.mark.parametrize("n,heads,dim,rope,opts", [
    (2050, 130, 64, 0, {}),
    (2100, 70, 128, 64, {"halves": True}),
    (2060, 40, 256, 64, {}),
    (1400, 33, 512, 64, {"leading": True}),
    (4200, 1, 128, 64, {"halves": True}),
    (4200, 3, 512, 48, {}),
    (4200, 5, 512, 48, {}),
])
def test_norm_rope_of_many_tokens(lib, n, heads, dim, rope, opts):
    """Batches that fill the device, with heads that fill a workgroup's steps,
    or the last of them in part, or few of their places; in place too."""
    rng = np.random.default_rng(n + heads)
    weight = torch.from_numpy(1 + rng.standard_normal(dim).astype(np.float32) * 0.3)
    x = vectors(rng, (n, heads, dim))
    freq = inv_freq(rope // 2) if rope else None
    positions = torch.from_numpy(rng.integers(0, 1 << 20, n)) if rope else None
    xd = x.cuda()
    out = torch.empty_like(xd)
    lib.idx_norm_rope(xd, dev(positions), dev(freq), out, weight=dev(weight), **opts)
    lib.idx_norm_rope(xd, dev(positions), dev(freq), xd, weight=dev(weight), **opts)
    assert torch.equal(xd.view(torch.int16), out.view(torch.int16))
    for a in range(0, n, 500):  # (a part at a time: float64 takes four times the room)
        b = min(n, a + 500)
        y, size = norm_rope(x[a:b], None if positions is None else positions[a:b], freq, weight, **opts)
        assert_near_bf16(out[a:b], y, size)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("power", [20, 31, 36, 40, 43])
def test_far_positions_keep_what_float64_leaves(lib, halves, power):
    """The angle is off by |theta| 2^-51 + 2^-25 at most (its product and its
    reduction by float64's 2 / pi, each within 2^-53 of itself or so, and the
    fraction of a quarter turn rounded to float32): values are off by as much of
    their pair's length, besides the roundings of any position."""
    rng = np.random.default_rng(power)
    n, dim = 200, 64
    positions = torch.from_numpy(rng.integers(1 << (power - 1), 1 << power, n) * rng.choice([-1, 1], n))
    freq = torch.cat([torch.tensor([1.0, 0.5]), torch.from_numpy(rng.random(30).astype(np.float32))])
    x = torch.from_numpy(rng.standard_normal((n, 1, dim))).to(torch.bfloat16)
    out = torch.empty((n, 1, dim), dtype=torch.bfloat16, device="cuda")
    lib.idx_norm_rope(x.cuda(), positions.cuda(), freq.cuda(), out, norm=False, halves=halves)
    y, size = norm_rope(x, positions, freq, norm=False, halves=halves)
    theta = np.abs(f64(positions))[:, None] * f64(freq)
    off = theta * 2.0 ** -51 + 2.0 ** -25
    off = np.concatenate([off, off], -1) if halves else np.repeat(off, 2, -1)
    # (assert_near_bf16 takes F32 of `size`)
    assert_near_bf16(out, y, size * (1 + off[:, None] / F32))


@pytest.mark.parametrize("bits", [0x7F81, 0xFF81, 0x7FBF, 0x7FC0, 0xFFFF])
@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("opts", [None, {}, {"halves": True}, {"leading": True}])
def test_store_nan_of_any_bits(lib, dim, opts, bits):
    """Without a norm, and where no rotation touches it: a NaN has no part in the
    amount, whatever its bits and wherever it stands, and becomes +-448; the other
    values are stored as without it.  (The largest value of each vector stands
    before the NaN, among the 8 that a lane has.)"""
    rng = np.random.default_rng(dim)
    rope = 0 if opts is None else 64
    first = 64 if opts and opts.get("leading") else 0  # of the values that are not rotated
    at = torch.arange(first, first + dim - rope)
    n, pages = len(at), -(-dim // PAGE)
    x = torch.from_numpy(rng.standard_normal((n, dim))).to(torch.bfloat16)
    t = torch.arange(n)
    x[t, at // 8 * 8] = 10.0
    whole = x.clone()
    whole[t, at] = 0.0
    x.view(torch.int16)[t, at] = bits - 0x10000 if bits >= 0x8000 else bits
    freq = inv_freq(32).cuda() if rope else None
    positions = torch.from_numpy(rng.integers(0, 1 << 20, n)).cuda() if rope else None
    slots = torch.from_numpy(rng.permutation(pages * PAGE)[:n])
    call = dict(norm=False, **(opts or {}))
    codes, scales = stored_bytes(lib, x.cuda(), positions, freq, None, slots.cuda(), pages, dim, **call)
    others, want = stored_bytes(lib, whole.cuda(), positions, freq, None, slots.cuda(), pages, dim, **call)
    assert np.array_equal(scales, want)
    s, i = slots.numpy(), at.numpy()
    assert (codes[s, i] == (0xFE if bits >= 0x8000 else 0x7E)).all()
    codes[s, i] = others[s, i]
    assert np.array_equal(codes, others)
