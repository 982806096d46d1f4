"""Host-side checks of the entry points of the cache of keys and values by head:
exports, argument validation (every call here returns before any HIP call) and
the binding's refusals."""
from __future__ import annotations

import re
import subprocess
import sys
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parent.parent
HEADER = ROOT / "include" / "kv_cache.h"
LIB = ROOT / "paged_mqa_logits_idx_amd" / "libidx_paged_mqa.so"

OK, NULL, UNSUPPORTED, SHAPE, ALIGN = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def raw():
    import paged_mqa_logits_idx_amd as b

    return b._lib


def test_declared_symbols_are_exported_and_bound(raw):
    import paged_mqa_logits_idx_amd as b

    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = sorted(set(re.findall(r"\b(idx_[a-z0-9_]+)\s*\(", text)))
    dyn = subprocess.run(["nm", "-D", "--defined-only", str(LIB)], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (idx_[a-z0-9_]+)$", dyn, flags=re.M))
    assert len(names) == 9
    for name in names:
        assert name in exported, name
        assert name in b.__all__ and callable(getattr(b, name))
        assert getattr(raw, name).argtypes is not None


def call(raw, name, order, base, **kw):
    a = dict(base)
    a.update(kw)
    order = order.split()
    assert len(order) == len(getattr(raw, name).argtypes)
    return getattr(raw, name)(*[a[k] for k in order])


PLAN_ORDER = "cached added requests free num_free pt width pts n slots positions rows lens starts taken stream"
PLAN = dict(cached=4, added=4, requests=2, free=4, num_free=1, pt=4, width=4, pts=4, n=2, slots=8, positions=8, rows=4,
            lens=4, starts=8, taken=8, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(requests=-1), SHAPE), (dict(requests=65537), SHAPE), (dict(num_free=-1), SHAPE), (dict(width=-1), SHAPE),
    (dict(width=(1 << 24) + 1, pts=1 << 25), SHAPE), (dict(n=-1), SHAPE), (dict(pts=3), SHAPE), (dict(pts=-1, requests=1), SHAPE),
    (dict(requests=0, n=0, cached=None, added=None, pt=None, starts=None, taken=None), OK),
    (dict(cached=None), NULL), (dict(added=None), NULL), (dict(pt=None), NULL), (dict(free=None), NULL),
    (dict(cached=2), ALIGN), (dict(added=2), ALIGN), (dict(free=2), ALIGN), (dict(pt=6), ALIGN), (dict(slots=4), ALIGN),
    (dict(positions=12), ALIGN), (dict(rows=2), ALIGN), (dict(lens=2), ALIGN), (dict(starts=4), ALIGN), (dict(taken=4), ALIGN),
])
def test_plan_validation(raw, kw, status):
    assert call(raw, "idx_plan_batch", PLAN_ORDER, PLAN, **kw) == status


STORE8 = "keys values slots n heads dim kst vst k v ks vs pages kvp kvh ksp ksh stream"
STORE16 = "keys values slots n heads dim kst vst k v pages kvp kvh stream"
STORE = dict(keys=16, values=16, slots=8, n=1, heads=2, dim=128, kst=256, vst=256, k=16, v=16, ks=4, vs=4, pages=1, kvp=65536,
             kvh=16384, ksp=512, ksh=256, stream=None)
STORE_CASES = [
    (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(n=-1), SHAPE),
    (dict(n=(1 << 32) + 1), SHAPE), (dict(heads=-1), SHAPE), (dict(kst=255), SHAPE), (dict(vst=248), SHAPE),
    (dict(pages=-1), SHAPE), (dict(kvp=8191), SHAPE), (dict(kvh=8191), SHAPE), (dict(kvp=(1 << 32) + 16), SHAPE),
    (dict(kvh=(1 << 38) + 16), SHAPE), (dict(n=0, keys=None, values=None, k=None, v=None, slots=None), OK),
    (dict(heads=0, keys=None, k=None), OK),
    (dict(keys=None), NULL), (dict(values=None), NULL), (dict(slots=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(keys=8), ALIGN), (dict(values=24), ALIGN), (dict(kst=260), ALIGN), (dict(vst=260), ALIGN), (dict(slots=4), ALIGN),
    (dict(k=8), ALIGN), (dict(v=8), ALIGN), (dict(kvp=65544), ALIGN), (dict(kvh=16392), ALIGN),
]


@pytest.mark.parametrize("kw,status", STORE_CASES)
def test_store_validation(raw, kw, status):
    assert call(raw, "idx_store_kv_fp8", STORE8, STORE, **kw) == status
    assert call(raw, "idx_store_kv_bf16", STORE16, STORE, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ksp=255), SHAPE), (dict(ksh=252), SHAPE), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(ks=2), ALIGN),
    (dict(vs=6), ALIGN), (dict(ksp=514), ALIGN), (dict(ksh=258), ALIGN),
])
def test_store_scale_validation(raw, kw, status):
    assert call(raw, "idx_store_kv_fp8", STORE8, STORE, **kw) == status


BOUNDS8 = "k ks pt rt tables first sl out rows heads dim width pages kvp kvh ksp ksh pts stream"
BOUNDS16 = "k pt rt tables first sl out rows heads dim width pages kvp kvh pts stream"
BOUNDS = dict(k=16, ks=4, pt=4, rt=4, tables=1, first=4, sl=4, out=16, rows=1, heads=2, dim=128, width=2, pages=1, kvp=65536,
              kvh=16384, ksp=512, ksh=256, pts=2, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=32), UNSUPPORTED), (dict(rows=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(rows=1 << 30, heads=2), SHAPE),
    (dict(width=-1), SHAPE), (dict(width=(1 << 24) + 1), SHAPE), (dict(tables=-1), SHAPE), (dict(pts=-1), SHAPE),
    (dict(pages=-1), SHAPE), (dict(kvp=100), SHAPE), (dict(kvh=100), SHAPE),
    (dict(rows=0, k=None, pt=None, sl=None, out=None), OK), (dict(width=0, pt=None, k=None), OK), (dict(heads=0, k=None), OK),
    (dict(k=None), NULL), (dict(pt=None), NULL), (dict(sl=None), NULL), (dict(out=None), NULL),
    (dict(k=8), ALIGN), (dict(pt=2), ALIGN), (dict(rt=2), ALIGN), (dict(first=2), ALIGN), (dict(sl=2), ALIGN), (dict(out=8), ALIGN),
    (dict(kvp=65544), ALIGN), (dict(kvh=16392), ALIGN),
])
def test_bounds_validation(raw, kw, status):
    assert call(raw, "idx_page_bounds_fp8", BOUNDS8, BOUNDS, **kw) == status
    assert call(raw, "idx_page_bounds_bf16", BOUNDS16, BOUNDS, **kw) == status


@pytest.mark.parametrize("rows,heads", [((1 << 24), 1), (1 << 22, 16), (1 << 30, 1)])
def test_bounds_of_more_rows_than_a_launch_has(raw, rows, heads):
    assert call(raw, "idx_page_bounds_fp8", BOUNDS8, BOUNDS, rows=rows, heads=heads) == SHAPE
    assert call(raw, "idx_page_bounds_bf16", BOUNDS16, BOUNDS, rows=rows, heads=heads) == SHAPE


SCORES_ORDER = "q near pt rt tables sl out counts rows heads kvheads dim width pages pts stride first last stream"
SCORES = dict(q=16, near=16, pt=4, rt=4, tables=1, sl=4, out=4, counts=4, rows=1, heads=8, kvheads=2, dim=128, width=2, pages=1,
              pts=2, stride=4, first=0, last=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=96), UNSUPPORTED), (dict(heads=258), UNSUPPORTED), (dict(kvheads=0), UNSUPPORTED), (dict(heads=7), SHAPE),
    (dict(heads=-2), SHAPE), (dict(rows=-1), SHAPE), (dict(width=-1), SHAPE), (dict(stride=1), SHAPE), (dict(pages=-1), SHAPE),
    (dict(first=-1), SHAPE), (dict(last=-1), SHAPE), (dict(tables=-1), SHAPE), (dict(pts=-1), SHAPE),
    (dict(rows=0, q=None, near=None), OK), (dict(heads=0, kvheads=0, q=None), OK),
    (dict(q=None), NULL), (dict(near=None), NULL), (dict(pt=None), NULL), (dict(sl=None), NULL), (dict(out=None), NULL),
    (dict(q=8), ALIGN), (dict(near=8), ALIGN), (dict(pt=2), ALIGN), (dict(rt=2), ALIGN), (dict(sl=2), ALIGN), (dict(out=2), ALIGN),
    (dict(counts=2), ALIGN),
])
def test_scores_validation(raw, kw, status):
    assert call(raw, "idx_page_scores", SCORES_ORDER, SCORES, **kw) == status


ATTEND8 = ("q k v ks vs pt rt tables idx sl sinks out lse rows heads kvheads dim width pages kvp kvh ksp ksh pts topk scale "
           "space bytes stream")
ATTEND16 = "q k v pt rt tables idx sl sinks out lse rows heads kvheads dim width pages kvp kvh pts topk scale space bytes stream"
ATTEND = dict(q=16, k=16, v=16, ks=4, vs=4, pt=4, rt=4, tables=1, idx=4, sl=4, sinks=4, out=16, lse=4, rows=1, heads=8, kvheads=2,
              dim=128, width=512, pages=1, kvp=65536, kvh=16384, ksp=512, ksh=256, pts=512, topk=512, scale=0.1, space=None, bytes=0,
              stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dim=512), UNSUPPORTED), (dict(heads=258), UNSUPPORTED), (dict(kvheads=0), UNSUPPORTED), (dict(heads=7), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=1000001), SHAPE), (dict(width=-1), SHAPE), (dict(width=(1 << 24) + 1), SHAPE),
    (dict(topk=-2), SHAPE), (dict(tables=-1), SHAPE), (dict(pts=-1), SHAPE), (dict(bytes=-1), SHAPE), (dict(pages=-1), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=3e38), SHAPE), (dict(kvp=100), SHAPE),
    (dict(kvh=100), SHAPE),
    (dict(rows=0, q=None, k=None, out=None), OK), (dict(heads=0, kvheads=0, q=None), OK),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(pt=None), NULL), (dict(idx=None), NULL),
    (dict(topk=-1), NULL), (dict(sl=None), NULL), (dict(out=None), NULL), (dict(), NULL), (dict(space=16, bytes=16), SHAPE),
    (dict(q=8), ALIGN), (dict(k=8), ALIGN), (dict(v=8), ALIGN), (dict(pt=2), ALIGN), (dict(rt=2), ALIGN), (dict(idx=2), ALIGN),
    (dict(sl=2), ALIGN), (dict(sinks=2), ALIGN), (dict(out=8), ALIGN), (dict(lse=2), ALIGN), (dict(space=8, bytes=1 << 30), ALIGN),
    (dict(kvp=65544), ALIGN), (dict(kvh=16392), ALIGN),
])
def test_attention_validation(raw, kw, status):
    """The base call lacks only its workspace, which is asked for last."""
    assert call(raw, "idx_kv_attention_fp8", ATTEND8, ATTEND, **kw) == status
    assert call(raw, "idx_kv_attention_bf16", ATTEND16, ATTEND, **kw) == status


def test_workspace_sizes(raw):
    size = raw.idx_kv_attention_workspace
    assert size(0, 8, 2, 128, 8, -1) == 0 and size(1, 0, 0, 128, 8, -1) == 0
    assert size(1, 8, 2, 96, 8, -1) == size(1, 7, 2, 128, 8, -1) == size(-1, 8, 2, 128, 8, -1) == size(1, 258, 2, 128, 8, -1) == -1
    assert size(1, 8, 2, 128, 8, -2) == size(1, 8, 2, 128, -1, -1) == size(1, 8, 0, 128, 8, -1) == -1
    assert size(64, 64, 8, 128, 512, -1) > 0
    assert size(100000, 64, 8, 128, 512, -1) == 0  # a unit a workgroup


# --- the binding's own checks, on CPU tensors: the first of them that fails speaks

I32, I64, BF16, F32, U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def attend(**kw):
    import paged_mqa_logits_idx_amd as b

    a = dict(q=zeros(2, 8, 128), k_pages=zeros(3, 2, 64, 128), v_pages=zeros(3, 2, 64, 128), page_table=zeros(2, 4, dtype=I32),
             page_idx=None, seqlens=zeros(2, dtype=I32), out=zeros(2, 8, 128), lse=None, scale=0.1)
    a.update(kw)
    return b.idx_kv_attention_bf16(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(q=zeros(2, 8, 128, dtype=F32)), "q must be torch.bfloat16"), (dict(out=zeros(2, 8, 64)), "q and out"),
    (dict(q=zeros(2, 1024)), "q and out"), (dict(k_pages=zeros(3, 2, 64, 128, dtype=U8)), "k_pages must be torch.bfloat16"),
    (dict(k_pages=zeros(3, 2, 64, 64)), "k_pages must be"), (dict(v_pages=zeros(3, 1, 64, 128)), "v_pages must be torch.bfloat16"),
    (dict(v_pages=zeros(3, 4, 64, 128)[:, ::2]), "v_pages must have the strides"), (dict(k_pages=zeros(3, 2, 128, 64).transpose(2, 3)), "dense"),
    (dict(page_table=zeros(2, 4, dtype=I64)), "page_table must be torch.int32"), (dict(page_table=zeros(3, 4, dtype=I32)[:, ::2]), "unit-stride"),
    (dict(q=zeros(3, 8, 128), out=zeros(3, 8, 128), seqlens=zeros(3, dtype=I32)), "2 tables for 3 rows"),
    (dict(seqlens=zeros(3, dtype=I32)), "seqlens must be"), (dict(page_idx=zeros(2, 2, 4, dtype=I64)), "page_idx must be torch.int32"),
    (dict(page_idx=zeros(3, 4, dtype=I32)), "page_idx must be"), (dict(sinks=zeros(7, dtype=F32)), "sinks must be"),
    (dict(lse=zeros(2, 7, dtype=F32)), "lse must be"), (dict(row_table=zeros(3, dtype=I32)), "row_table must be"),
    (dict(workspace=zeros(8, 8, dtype=U8)[:, ::2]), "workspace must be contiguous"), (dict(num_pages=4), "holds 3 pages"),
    (dict(), "must be device tensors"),
])
def test_binding_refusals_attention(kw, text):
    with pytest.raises(ValueError, match=text):
        attend(**kw)


@pytest.mark.parametrize("kw,text", [
    (dict(cached=zeros(2, dtype=I64)), "cached must be torch.int32"), (dict(added=zeros(3, dtype=I32)), "added must be"),
    (dict(page_table=zeros(3, 4, dtype=I32)), "3 tables for 2 requests"), (dict(page_table=zeros(2, 4, dtype=I64)), "page_table must be torch.int32"),
    (dict(page_table=zeros(2, 8, dtype=I32)[:, ::2]), "unit-stride"), (dict(slots=zeros(4, dtype=I32)), "slots must be torch.int64"),
    (dict(seqlens=zeros(5, dtype=I32)), "seqlens must be"), (dict(starts=zeros(2, dtype=I64)), "starts must be"),
    (dict(taken=zeros(1, dtype=I32)), "taken must be"), (dict(free_pages=zeros(4, dtype=I64)), "free_pages must be"),
    (dict(), "must be device tensors"),
])
def test_binding_refusals_plan(kw, text):
    import paged_mqa_logits_idx_amd as b

    a = dict(cached=zeros(2, dtype=I32), added=zeros(2, dtype=I32), free_pages=zeros(4, dtype=I32), page_table=zeros(2, 4, dtype=I32),
             slots=zeros(4, dtype=I64), positions=zeros(4, dtype=I64), row_table=zeros(4, dtype=I32), seqlens=zeros(4, dtype=I32),
             starts=zeros(3, dtype=I64), taken=zeros(1, dtype=I64))
    a.update(kw)
    with pytest.raises(ValueError, match=text):
        b.idx_plan_batch(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(keys=zeros(4, 256)), "keys must have 3 dims"), (dict(values=zeros(4, 1, 128)), "values must be"),
    (dict(keys=zeros(4, 2, 128, dtype=F32)), "keys must be torch.bfloat16"), (dict(slots=zeros(4, dtype=I32)), "slots must be"),
    (dict(k_pages=zeros(3, 4, 64, 128, dtype=U8), v_pages=zeros(3, 4, 64, 128, dtype=U8), kscale=zeros(3, 4, 64, dtype=F32),
          vscale=zeros(3, 4, 64, dtype=F32)), "k_pages must have 2 heads"),
    (dict(kscale=zeros(3, 2, 64)), "kscale must be torch.float32"), (dict(vscale=zeros(2, 2, 64, dtype=F32)), "vscale must be torch.float32"),
    (dict(vscale=zeros(3, 2, 128, dtype=F32)[..., :64]), "vscale must have the strides"), (dict(num_pages=4), "holds 3 pages"),
    (dict(), "must be device tensors"),
])
def test_binding_refusals_store(kw, text):
    import paged_mqa_logits_idx_amd as b

    a = dict(keys=zeros(4, 2, 128), values=zeros(4, 2, 128), slots=zeros(4, dtype=I64), k_pages=zeros(3, 2, 64, 128, dtype=U8),
             v_pages=zeros(3, 2, 64, 128, dtype=U8), kscale=zeros(3, 2, 64, dtype=F32), vscale=zeros(3, 2, 64, dtype=F32))
    a.update(kw)
    with pytest.raises(ValueError, match=text):
        b.idx_store_kv_fp8(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(bounds=zeros(2, 2, 2, 128)), "bounds must be"), (dict(bounds=zeros(3, 2, 2, 64)), "bounds must be"),
    (dict(bounds=zeros(3, 2, 2, 128, dtype=F32)), "bounds must be torch.bfloat16"), (dict(first=zeros(3, dtype=I32)), "first must be"),
    (dict(seqlens=zeros(2, dtype=I64)), "seqlens must be"), (dict(page_table=zeros(3, 4, dtype=I32)[0]), "two dims"),
    (dict(), "must be device tensors"),
])
def test_binding_refusals_bounds(kw, text):
    import paged_mqa_logits_idx_amd as b

    a = dict(k_pages=zeros(3, 2, 64, 128), page_table=zeros(2, 4, dtype=I32), seqlens=zeros(2, dtype=I32), bounds=zeros(3, 2, 2, 128))
    a.update(kw)
    with pytest.raises(ValueError, match=text):
        b.idx_page_bounds_bf16(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(q=zeros(2, 1024)), "q must be"), (dict(bounds=zeros(3, 2, 128)), "q must be"), (dict(bounds=zeros(3, 2, 2, 64)), "q must be"),
    (dict(scores=zeros(2, 2, 4)), "scores must be torch.float32"), (dict(scores=zeros(2, 2, 5, dtype=F32)), "scores must be"),
    (dict(scores=zeros(2, 2, 8, dtype=F32)[..., ::2]), "unit-stride"), (dict(scores=zeros(4, 2, 4, dtype=F32)[::2]), "evenly apart"),
    (dict(page_counts=zeros(2, dtype=I32)), "page_counts must be"), (dict(), "must be device tensors"),
])
def test_binding_refusals_scores(kw, text):
    import paged_mqa_logits_idx_amd as b

    a = dict(q=zeros(2, 8, 128), bounds=zeros(3, 2, 2, 128), page_table=zeros(2, 4, dtype=I32), seqlens=zeros(2, dtype=I32),
             scores=zeros(2, 2, 4, dtype=F32))
    a.update(kw)
    with pytest.raises(ValueError, match=text):
        b.idx_page_scores(**a)


def test_binding_takes_tensors_alone():
    """What is no tensor, or too few of them, is refused by name."""
    import paged_mqa_logits_idx_amd as b

    with pytest.raises(ValueError, match="q must be a tensor"):
        attend(q=[1.0])
    with pytest.raises(ValueError, match="page_table must be a tensor"):
        attend(page_table=None)
    with pytest.raises(TypeError):
        attend(scale="half")
    with pytest.raises(TypeError):
        attend(num_pages=1.5)
    with pytest.raises(TypeError, match="arguments"):
        b._binding.plan_batch(1)


def test_other_operators_without_the_compiled_marshalling():
    """The indexer's and the latent cache's calls do not need _binding.so; those that do
    say so when they are called."""
    code = """
import sys
sys.modules["paged_mqa_logits_idx_amd._binding"] = None  # as if it were not built
import torch
import paged_mqa_logits_idx_amd as b
assert b.idx_abi_version() > 0 and b.idx_kv_attention_workspace(0, 8, 2, 128, 8) == 0
try:
    b.idx_topk_logits(torch.zeros((1, 8)), torch.zeros((1,), dtype=torch.int64), torch.zeros((1, 2), dtype=torch.int32))
except ValueError as e:
    assert "lens" in str(e) or "int32" in str(e), e
else:
    raise AssertionError("a wrong type went through")
z = torch.zeros((1, 1), dtype=torch.int32)
for call in (lambda: b.idx_plan_batch(z[0], z[0], z[0], z), lambda: b.idx_store_kv_bf16(z, z, z, z, z),
             lambda: b.idx_page_bounds_bf16(z, z, z, z), lambda: b.idx_page_scores(z, z, z, z, z),
             lambda: b.idx_kv_attention_bf16(z, z, z, z, None, z, z, scale=1.0)):
    try:
        call()
    except ImportError as e:
        assert "_binding.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("went on without it")
print("fine")
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert done.returncode == 0 and done.stdout.strip().endswith("fine"), done.stderr
