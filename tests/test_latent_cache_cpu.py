"""Host-side checks of the latent cache's entry points: exports, argument
validation (every call here returns before any HIP call) and the binding's
refusals."""
from __future__ import annotations

import ctypes
import re
import subprocess
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parent.parent
HEADER = ROOT / "include" / "latent_cache.h"
LIB = ROOT / "paged_mqa_logits_idx_amd" / "libidx_paged_mqa.so"

OK, NULL, UNSUPPORTED, SHAPE, ALIGN = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def raw():
    import paged_mqa_logits_idx_amd as b

    return b._lib


def declared():
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    return sorted(set(re.findall(r"\b(idx_[a-z0-9_]+)\s*\(", text)))


def test_declared_symbols_are_exported_and_bound(raw):
    import paged_mqa_logits_idx_amd as b

    dyn = subprocess.run(["nm", "-D", "--defined-only", str(LIB)], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (idx_[a-z0-9_]+)$", dyn, flags=re.M))
    names = declared()
    assert names
    for name in names:
        assert name in exported, name
        assert name in b.__all__ and callable(getattr(b, name))
        assert getattr(raw, name).argtypes is not None


def call(raw, name, order, base, **kw):
    a = dict(base)
    a.update(kw)
    return getattr(raw, name)(*[a[k] for k in order.split()])


ROPE_ORDER = "x w pos freq out n heads dim rope flags eps xs stream"
ROPE = dict(x=16, w=16, pos=8, freq=4, out=16, n=1, heads=2, dim=128, rope=64, flags=0, eps=1e-6, xs=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=96), UNSUPPORTED), (dict(dim=1024), UNSUPPORTED), (dict(dim=0), UNSUPPORTED),
    (dict(rope=8), UNSUPPORTED), (dict(rope=-16), UNSUPPORTED), (dict(rope=144), UNSUPPORTED), (dict(flags=8), UNSUPPORTED),
    (dict(n=-1), SHAPE), (dict(n=(1 << 40) + 1), SHAPE), (dict(heads=-1), SHAPE), (dict(xs=248), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(n=0, x=None, out=None, pos=None, freq=None), OK), (dict(heads=0, x=None, out=None), OK),
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(pos=None), NULL), (dict(freq=None), NULL), (dict(flags=1), NULL),
    (dict(x=8), ALIGN), (dict(w=4), ALIGN), (dict(pos=4), ALIGN), (dict(freq=2), ALIGN), (dict(out=8), ALIGN), (dict(xs=260), ALIGN),
])
def test_norm_rope_validation(raw, kw, status):
    assert call(raw, "idx_norm_rope", ROPE_ORDER, ROPE, **kw) == status


STORE8_ORDER = "x w pos freq slots n dim rope flags eps xs kv ks pages kvs kss stream"
STORE16_ORDER = "x w pos freq slots n dim rope flags eps xs kv pages kvs stream"
STORE = dict(x=16, w=16, pos=8, freq=4, slots=8, n=1, dim=512, rope=64, flags=0, eps=1e-6, xs=512, kv=16, ks=4, pages=1, kvs=33024,
             kss=33024, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=256), UNSUPPORTED), (dict(dim=64), UNSUPPORTED), (dict(rope=8), UNSUPPORTED), (dict(flags=16), UNSUPPORTED),
    (dict(n=-1), SHAPE), (dict(xs=504), SHAPE), (dict(pages=-1), SHAPE), (dict(pages=(1 << 40) + 1), SHAPE),
    (dict(kvs=32767), SHAPE), (dict(kvs=(1 << 32) + 16), SHAPE), (dict(kss=255), SHAPE),
    (dict(n=0, x=None, slots=None, kv=None, ks=None), OK),
    (dict(x=None), NULL), (dict(slots=None), NULL), (dict(kv=None), NULL), (dict(ks=None), NULL), (dict(pos=None), NULL),
    (dict(slots=4), ALIGN), (dict(kv=8), ALIGN), (dict(ks=2), ALIGN), (dict(kvs=33032), ALIGN), (dict(kss=33026), ALIGN), (dict(xs=516), ALIGN),
])
def test_store_fp8_validation(raw, kw, status):
    assert call(raw, "idx_norm_rope_store_fp8", STORE8_ORDER, STORE, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kvs=33024), SHAPE), (dict(dim=64), UNSUPPORTED), (dict(n=0, x=None), OK), (dict(kv=None), NULL), (dict(kv=8), ALIGN),
    (dict(slots=12), ALIGN),
])
def test_store_bf16_validation(raw, kw, status):
    assert call(raw, "idx_norm_rope_store_bf16", STORE16_ORDER, STORE, **{"kvs": 65536, **kw}) == status


LOAD8_ORDER = "kv ks slots n dim pages kvs kss out os stream"
LOAD16_ORDER = "kv slots n dim pages kvs out os stream"
LOAD = dict(kv=16, ks=4, slots=8, n=1, dim=512, pages=1, kvs=65536, kss=256, out=16, os=512, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=64), UNSUPPORTED), (dict(n=-1), SHAPE), (dict(os=511), SHAPE), (dict(kvs=32000), SHAPE), (dict(pages=-1), SHAPE),
    (dict(n=0, kv=None, ks=None, slots=None, out=None), OK),
    (dict(kv=None), NULL), (dict(slots=None), NULL), (dict(out=None), NULL),
    (dict(kv=8), ALIGN), (dict(slots=4), ALIGN), (dict(out=8), ALIGN), (dict(os=516), ALIGN),
])
def test_load_validation(raw, kw, status):
    assert call(raw, "idx_load_slots_fp8", LOAD8_ORDER, LOAD, **kw) == status
    assert call(raw, "idx_load_slots_bf16", LOAD16_ORDER, LOAD, **kw) == status


def test_load_fp8_scales(raw):
    assert call(raw, "idx_load_slots_fp8", LOAD8_ORDER, LOAD, ks=None) == NULL
    assert call(raw, "idx_load_slots_fp8", LOAD8_ORDER, LOAD, kss=128) == SHAPE
    assert call(raw, "idx_load_slots_fp8", LOAD8_ORDER, LOAD, ks=6) == ALIGN


def test_binding_refuses():
    """Wrong types, shapes, layouts and host tensors, before any library call."""
    import paged_mqa_logits_idx_amd as b

    bf = dict(dtype=torch.bfloat16)
    x, out = torch.zeros(4, 2, 128, **bf), torch.zeros(4, 2, 128, **bf)
    pos, freq = torch.zeros(4, dtype=torch.int64), torch.zeros(32)
    for match, args, kw in [
        ("x must be torch.bfloat16", (x.float(), pos, freq, out), {}),
        ("x must have 3 dims", (x[0], pos, freq, out), {}),
        ("dense behind its first dim", (x.transpose(0, 1).contiguous().transpose(0, 1), pos, freq, out), {}),
        ("out must be", (x, pos, freq, out[:2]), {}),
        ("out must be torch.bfloat16", (x, pos, freq, out.half()), {}),
        ("go together", (x, pos, None, out), {}),
        ("positions must be torch.int64", (x, pos.int(), freq, out), {}),
        ("positions must be", (x, pos[:3], freq, out), {}),
        ("inv_freq must be torch.float32", (x, pos, freq.double(), out), {}),
        ("weight must be", (x, pos, freq, out), dict(weight=torch.zeros(64))),
        ("weight goes with the norm", (x, pos, freq, out), dict(weight=torch.zeros(128), norm=False)),
        ("must be device tensors", (x, pos, freq, out), {}),
    ]:
        with pytest.raises(ValueError, match=match):
            b.idx_norm_rope(*args, **kw)
    v, slots, kv = torch.zeros(4, 512, **bf), torch.zeros(4, dtype=torch.int64), torch.zeros(33024, dtype=torch.uint8)
    for match, args, kw in [
        ("x must have 2 dims", (x, pos, freq, slots, kv, 4), dict(num_pages=1)),
        ("slots must be torch.int64", (v, pos, freq, slots.int(), kv, 4), dict(num_pages=1)),
        ("slots must be", (v, pos, freq, slots[:2], kv, 4), dict(num_pages=1)),
        ("kv_pages is shorter", (v, pos, freq, slots, kv, 4), dict(num_pages=2)),
        ("kscale is shorter", (v, pos, freq, slots, kv, torch.zeros(63)), dict(num_pages=1)),
        ("kscale must be torch.float32", (v, pos, freq, slots, kv, torch.zeros(64).half()), dict(num_pages=1)),
        ("must be device tensors", (v, pos, freq, slots, kv, 4), dict(num_pages=1)),
    ]:
        with pytest.raises(ValueError, match=match):
            b.idx_norm_rope_store_fp8(*args, **kw)
    with pytest.raises(ValueError, match="kv_pages is shorter"):
        b.idx_norm_rope_store_bf16(v, pos, freq, slots, kv, num_pages=1)
    with pytest.raises(ValueError, match="out must have 2 dims"):
        b.idx_load_slots_fp8(kv, 4, slots, x, num_pages=1)
    with pytest.raises(ValueError, match="kv_pages must be contiguous"):
        b.idx_load_slots_bf16(kv[::2], slots, v, num_pages=0)


ATT8_ORDER = "q kv ks pt rt nt idx sl sinks out lse rows heads dim width pages kvs kss pts k scale ws wb stream"
ATT16_ORDER = "q kv pt rt nt idx sl sinks out lse rows heads dim width pages kvs pts k scale ws wb stream"
ATT = dict(q=16, kv=16, ks=4, pt=4, rt=None, nt=0, idx=4, sl=4, sinks=None, out=16, lse=4, rows=1, heads=64, dim=512, width=1,
           pages=1, kvs=65536, kss=33024, pts=1, k=8, scale=0.5, ws=None, wb=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=576), UNSUPPORTED), (dict(heads=129), UNSUPPORTED),
    (dict(rows=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(width=-1), SHAPE), (dict(width=(1 << 24) + 1), SHAPE), (dict(k=-2), SHAPE),
    (dict(pages=-1), SHAPE), (dict(kvs=32000), SHAPE), (dict(pts=-1), SHAPE), (dict(nt=-1), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("-inf")), SHAPE), (dict(wb=-1), SHAPE),
    (dict(rows=0, q=None, out=None), OK), (dict(heads=0, q=None, out=None), OK),
    (dict(q=None), NULL), (dict(kv=None), NULL), (dict(pt=None), NULL), (dict(sl=None), NULL), (dict(out=None), NULL),
    (dict(idx=None), NULL), (dict(k=-1), NULL),           # a list without its length, a length without its list
    (dict(q=8), ALIGN), (dict(kv=8), ALIGN), (dict(pt=2), ALIGN), (dict(rt=2), ALIGN), (dict(idx=2), ALIGN), (dict(sl=2), ALIGN),
    (dict(sinks=2), ALIGN), (dict(out=8), ALIGN), (dict(lse=2), ALIGN), (dict(ws=8), ALIGN), (dict(kvs=65544), ALIGN),
    (dict(k=4096, width=64), NULL),                       # splits its rows: a workspace is needed
    (dict(k=4096, width=64, ws=16, wb=1000), SHAPE),      # too small a one
    (dict(idx=None, k=-1, width=4097), NULL),
])
def test_attention_validation(raw, kw, status):
    assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, **kw) == status
    assert call(raw, "idx_latent_attention_bf16", ATT16_ORDER, ATT, **kw) == status


def test_attention_fp8_scales(raw):
    assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, ks=None) == NULL
    assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, kss=252) == SHAPE
    assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, ks=6) == ALIGN


def test_attention_workspace_sizes():
    import paged_mqa_logits_idx_amd as b

    assert b.idx_latent_attention_workspace(0, 64, 32, 2048) == 0
    assert b.idx_latent_attention_workspace(4096, 64, 88, 2048) == 0       # rows enough to fill the device
    assert b.idx_latent_attention_workspace(1, 64, 512, 2048) > 0
    assert b.idx_latent_attention_workspace(1, 64, 512) >= b.idx_latent_attention_workspace(1, 64, 512, 2048)
    assert b.idx_latent_attention_workspace(1, 64, 512, 16) == 0           # one tile
    for bad in [(-1, 64, 32, 1), (1, 129, 32, 1), (1, 64, -1, 1), (1, 64, (1 << 24) + 1, 1)]:
        assert b.idx_latent_attention_workspace(*bad) == -1


def test_attention_binding_refuses():
    import paged_mqa_logits_idx_amd as b

    q = torch.zeros(3, 8, 512, dtype=torch.bfloat16)
    kv = torch.zeros((2, 33024), dtype=torch.uint8)
    table, sl = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    idx = torch.zeros((3, 4), dtype=torch.int32)
    for match, args, kw in [
        ("q must be torch.bfloat16", (q.float(), kv, 4, table, idx, sl, q), {}),
        ("q and out must be", (q, kv, 4, table, idx, sl, q[:2]), {}),
        ("page_table must be torch.int32", (q, kv, 4, table.long(), idx, sl, q), {}),
        ("page_table must have two dims", (q, kv, 4, table[0], idx, sl, q), {}),
        ("holds 2 tables for 3 rows", (q, kv, 4, table[:2], idx, sl, q), {}),
        ("topk_idx must be", (q, kv, 4, table, idx[:2], sl, q), {}),
        ("topk_idx must be contiguous", (q, kv, 4, table, idx.t().contiguous().t(), sl, q), {}),
        ("seqlens must be", (q, kv, 4, table, idx, sl[:2], q), {}),
        ("lse must be", (q, kv, 4, table, idx, sl, q, torch.zeros(3, 9)), {}),
        ("sinks must be", (q, kv, 4, table, idx, sl, q), dict(sinks=torch.zeros(9))),
        ("row_table must be", (q, kv, 4, table, idx, sl, q), dict(row_table=sl[:1])),
        ("kv_pages is shorter", (q, kv, 4, table, idx, sl, q), dict(num_pages=3)),
        ("must be device tensors", (q, kv, 4, table, idx, sl, q), {}),
    ]:
        with pytest.raises(ValueError, match=match):
            b.idx_latent_attention_fp8(*args, scale=1.0, **{"num_pages": 2, **kw})


def test_attention_size_limits(raw):
    """A launch has fewer than 2^32 threads."""
    import paged_mqa_logits_idx_amd as b

    for rows, heads in [(8_000_001, 64), (4_000_001, 65), ((1 << 31) - 1, 128)]:
        assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, rows=rows, heads=heads) == SHAPE
        assert call(raw, "idx_latent_attention_bf16", ATT16_ORDER, ATT, rows=rows, heads=heads) == SHAPE
        assert b.idx_latent_attention_workspace(rows, heads, 1, 8) == -1
    assert b.idx_latent_attention_workspace(8_000_000, 64, 1, 8) == 0
    assert b.idx_latent_attention_workspace(4_000_000, 65, 1, 8) == 0


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_attention_scale_in_base_2(raw, scale):
    """The kernels take the scale times log2(e): one that overflows there would
    make every row NaN."""
    assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, scale=scale) == SHAPE
    assert call(raw, "idx_latent_attention_bf16", ATT16_ORDER, ATT, scale=scale) == SHAPE


def test_attention_scale_below_the_limit(raw):
    for scale in (2.35e38, -2.35e38):  # (3.4028e38 / 1.4427 = 2.3587e38)
        assert call(raw, "idx_latent_attention_fp8", ATT8_ORDER, ATT, scale=scale, rows=0) == OK
