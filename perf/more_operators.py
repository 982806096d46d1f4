"""Measured cases of serving with a paged cache of keys and values by head: the
block tables and slot maps of a batch, the store of new keys and values, the
bounds of each page's keys, the score of a page by its bounds, and attention of
one new token over all pages or over the selected ones.

    plan     request r has cached[r] tokens and gets added[r] more: new pages
             from the free list, then slot, position, request and length of
             every new token
    store    keys and values to their slots; e4m3: scale = amax / 448 and codes
    bounds   lo_d = min, hi_d = max over a page's live keys, rounded outwards
    scores   s_j = max_h sum_d max(q_hd lo_jd, q_hd hi_jd) over the query heads
             h of a key head, +inf for the first and last pages of a row
    attend   out_h = sum_p softmax_p(scale * <q_h, k_p>) v_p over the positions
             below the row's length, of all pages or of those selected, with
             an optional sink logit a head, and the log of the denominator

`own` chooses between the plain form, elementary torch operations in 32 bits,
and the library's own entry points.  Sizes: 64-position pages, 64 query heads,
heads of 128 values, the batches, the contexts of 8192, 32768 and 262208
positions and the 2048 selected positions (32 pages) are the indexer's and the
benchmark's; 8 key heads and heads of 64 and 256 values are generic.
"""
import math

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
BF16_MAX = 3.3895313892515355e38


def listed():
    return [
        # one decode step: 64 requests, a new token each
        {"name": "plan decode", "op": "plan", "requests": 64, "n": 64, "context": 32768, "prompts": False},
        # a large mixed step: prompts and decoding requests, 65536 token places
        {"name": "plan mixed", "op": "plan", "requests": 1024, "n": 65536, "context": 32768, "prompts": True},
        # keys and values of one decode step
        {"name": "store decode fp8", "op": "store", "n": 64, "kv_heads": 8, "dim": 128, "fp8": True},
        # keys and values of long prompts
        {"name": "store prompt bf16", "op": "store", "n": 32768, "kv_heads": 8, "dim": 128, "fp8": False},
        # a decode step renews the bounds of each row's last page
        {"name": "bounds decode fp8", "op": "bounds", "rows": 64, "context": 8192, "fresh": 1, "kv_heads": 8, "dim": 128, "fp8": True},
        # bounds of all pages of four prompts
        {"name": "bounds prompts bf16", "op": "bounds", "rows": 4, "context": 32768, "fresh": 0, "kv_heads": 8, "dim": 128, "fp8": False},
        # pages of the longest single request
        {"name": "scores long context", "op": "scores", "rows": 1, "context": 262208, "heads": 64, "kv_heads": 8, "dim": 128},
        # pages of a decode batch
        {"name": "scores decode", "op": "scores", "rows": 64, "context": 32768, "heads": 64, "kv_heads": 8, "dim": 128},
        # one request decoding alone
        {"name": "attend one row", "op": "attend", "rows": 1, "context": 8192, "heads": 64, "kv_heads": 8, "dim": 128, "k": 0, "fp8": False, "sinks": False},
        # odd batch, group and selection, small heads
        {"name": "attend odd selected", "op": "attend", "rows": 33, "context": 8191, "heads": 40, "kv_heads": 8, "dim": 64, "k": 17, "fp8": True, "sinks": True},
        # a decode batch over 32 selected pages of up to 512
        {"name": "attend selected fp8", "op": "attend", "rows": 64, "context": 32768, "heads": 64, "kv_heads": 8, "dim": 128, "k": 32, "fp8": True, "sinks": False},
        # the same batch over everything cached
        {"name": "attend decode bf16", "op": "attend", "rows": 64, "context": 32768, "heads": 64, "kv_heads": 8, "dim": 128, "k": 0, "fp8": False, "sinks": False},
    ]


def _between(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["plan", "store", "bounds", "scores", "attend", "attend", "attend"])
    if op == "plan":
        requests = _between(rng, 1, 1024)
        prompts = rng.random() < 0.6
        return {"op": op, "requests": requests, "n": _between(rng, requests, 65536) if prompts else requests + rng.randint(0, 7),
                "context": _between(rng, 64, 32768), "prompts": prompts}
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, rng.randint(1, 16)])
    fp8 = rng.random() < 0.5
    if op == "store":
        return {"op": op, "n": _between(rng, 1, 32768 * 8 * 128 // (kv_heads * dim)), "kv_heads": kv_heads, "dim": dim, "fp8": fp8}
    rows, context = _between(rng, 1, 64), _between(rng, 1, 32768)
    if rows == 1 and rng.random() < 0.5:  # a long context
        context = _between(rng, 32768, 262208)
    if op == "bounds":
        rows = max(1, min(rows, 4 * 32768 * 8 * 128 // (context * kv_heads * dim)))
        return {"op": op, "rows": rows, "context": context, "fresh": rng.choice([0, 1, _between(rng, 1, context)]), "kv_heads": kv_heads,
                "dim": dim, "fp8": fp8}
    heads = kv_heads * rng.choice([1, 4, 8, rng.randint(1, 16), max(1, 64 // kv_heads), max(1, 128 // kv_heads)])
    if op == "scores":
        rows = max(1, min(rows, 64 * 32768 * 8 * 128 // (context * kv_heads * dim)))
        return {"op": op, "rows": rows, "context": context, "heads": heads, "kv_heads": kv_heads, "dim": dim}
    k = rng.choice([0, _between(rng, 1, 64)])
    rows = max(1, min(rows, 48 * 32768 * 8 * 128 // (context * kv_heads * dim)))
    return {"op": op, "rows": rows, "context": context, "heads": heads, "kv_heads": kv_heads, "dim": dim, "k": k, "fp8": fp8,
            "sinks": rng.random() < 0.5}


def _lengths(case):
    """Positions of each row: a spread from a quarter of the context up."""
    rows, context = case["rows"], case["context"]
    return [context - (3 * context * b // 4) // rows for b in range(rows)]


def _pages(n):
    return -(-n // PAGE)


def work(case):
    op = case["op"]
    if op == "plan":
        n, requests = case["n"], case["requests"]
        return {"bytes": 24 * n + 16 * requests + 8 * (n // PAGE + requests), "flops": 0}
    heads, d = case["kv_heads"], case["dim"]
    if op == "store":
        n = case["n"]
        return {"bytes": n * (heads * (4 * d + 2 * (d + 4 if case["fp8"] else 2 * d)) + 8), "flops": 4 * n * heads * d}
    lengths = _lengths(case)
    if op == "bounds":
        positions = sum(n - (max(0, n - case["fresh"]) // PAGE * PAGE if case["fresh"] else 0) for n in lengths)
        pages = sum(_pages(n) - (max(0, n - case["fresh"]) // PAGE if case["fresh"] else 0) for n in lengths)
        return {"bytes": heads * (positions * (d + 4 if case["fp8"] else 2 * d) + pages * 4 * d) + 4 * pages, "flops": 2 * heads * positions * d}
    if op == "scores":
        pages, columns = sum(_pages(n) for n in lengths), case["rows"] * _pages(case["context"])
        return {"bytes": heads * (pages * 4 * d + columns * 4) + 4 * pages + case["rows"] * case["heads"] * 2 * d,
                "flops": 4 * pages * case["heads"] * d}
    seen = sum(min(n, case["k"] * PAGE) if case["k"] else n for n in lengths)
    per_position = 2 * (d + 4 if case["fp8"] else 2 * d)
    return {"bytes": heads * seen * per_position + case["rows"] * (case["heads"] * (4 * d + 4) + 4 * case["k"] * heads) + seen // PAGE * 4,
            "flops": 4 * seen * case["heads"] * d}


def _codes(shape, gen):
    """e4m3 codes of normal values over their largest of 448."""
    return (torch.randn(shape, generator=gen, device="cuda") * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _pool(state, pages, gen):
    """Keys and values of a pool: [pages, 2, heads] blocks of 64 positions, the
    e4m3 blocks with their scales behind the codes."""
    case = state["case"]
    heads, d = case["kv_heads"], case["dim"]
    if case["fp8"]:
        pool = torch.empty((pages, 2, heads, PAGE * (d + 4)), dtype=torch.uint8, device="cuda")
        pool[..., : PAGE * d] = _codes((pages, 2, heads, PAGE * d), gen).view(torch.uint8)
        scales = pool[..., PAGE * d :].view(torch.float32)
        scales.copy_((torch.rand(scales.shape, generator=gen, device="cuda") + 0.6) / 110.0)
        values = pool[..., : PAGE * d].view(torch.float8_e4m3fn).unflatten(-1, (PAGE, d))
        state["k_pages"], state["v_pages"] = values[:, 0], values[:, 1]
        state["kscale"], state["vscale"] = scales[:, 0], scales[:, 1]
    else:
        values = _normal((pages, 2, heads, PAGE, d), gen)
        state["k_pages"], state["v_pages"] = values[:, 0], values[:, 1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    op = case["op"]

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def ints(x, dtype=torch.int32):
        return x.floor().to(dtype)

    if op == "plan":
        requests, n, context = case["requests"], case["n"], case["context"]
        width = _pages(context)
        if case["prompts"]:  # every eighth request decodes, the others bring what is left of the token places, unevenly
            share = uniform(requests) ** 2
            added = ints(share / share.sum() * (n - requests) * 0.97) + 1
            added[::8] = 1
        else:
            added = torch.ones((requests,), dtype=torch.int32, device="cuda")
        added = added.clamp(max=context)
        state["added"] = added
        state["cached"] = ints(uniform(requests) * (context - added + 1)).clamp(min=0)
        free = requests + n // PAGE + 1
        order = torch.randperm(free + requests * width, generator=gen, device="cuda").to(torch.int32)
        state["free"] = order[:free].contiguous()
        state["table"] = order[free:].reshape(requests, width).contiguous()
        state["slots"] = torch.empty((n,), dtype=torch.int64, device="cuda")
        state["positions"] = torch.empty((n,), dtype=torch.int64, device="cuda")
        state["row_table"] = torch.empty((n,), dtype=torch.int32, device="cuda")
        state["seqlens"] = torch.empty((n,), dtype=torch.int32, device="cuda")
        state["starts"] = torch.empty((requests + 1,), dtype=torch.int64, device="cuda")
        state["taken"] = torch.empty((1,), dtype=torch.int64, device="cuda")
        return state
    heads, d = case["kv_heads"], case["dim"]
    if op == "store":
        # slots in random order over a pool with as many again, a few tokens
        # without a slot; the page behind the pool takes what the plain form
        # has to put somewhere
        n = case["n"]
        pages = _pages(2 * n)
        size = uniform(n, 1, 1) * 3 + 0.2
        state["keys"] = (torch.randn((n, heads, d), generator=gen, device="cuda") * size).to(torch.bfloat16)
        state["values"] = (torch.randn((n, heads, d), generator=gen, device="cuda") * size).to(torch.bfloat16)
        slots = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:n].contiguous()
        if n > 8:
            slots[torch.randint(0, n, (n // 64 + 1,), generator=gen, device="cuda")] = -1
        state["slots"], state["pages"] = slots, pages
        _pool(state, pages + 1, gen)
        return state
    rows, width = case["rows"], _pages(case["context"])
    pages = rows * width
    state["table"] = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).reshape(rows, width)
    order = torch.randperm(rows, generator=gen, device="cuda")
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order].contiguous()
    state["lengths"], state["pages"] = lengths, pages
    if op == "bounds":
        if case["fp8"]:
            block = torch.empty((pages, heads, PAGE * (d + 4)), dtype=torch.uint8, device="cuda")
            block[..., : PAGE * d] = _codes((pages, heads, PAGE * d), gen).view(torch.uint8)
            state["kscale"] = block[..., PAGE * d :].view(torch.float32)
            state["kscale"].copy_((uniform(pages, heads, PAGE) + 0.6) / 110.0)
            state["k_pages"] = block[..., : PAGE * d].view(torch.float8_e4m3fn).unflatten(-1, (PAGE, d))
        else:
            state["k_pages"] = _normal((pages, heads, PAGE, d), gen)
        state["first"] = (lengths - case["fresh"]).clamp(min=0) if case["fresh"] else torch.zeros_like(lengths)
        state["bounds"] = _normal((pages + 1, heads, 2, d), gen)  # the page behind: as above
        return state
    state["q"] = (1.5 * torch.randn((rows, case["heads"], d), generator=gen, device="cuda")).to(torch.bfloat16)
    if op == "scores":
        # bounds of 64 normal keys: about two and a half on either side, less a common part
        middle = 0.5 * torch.randn((pages, heads, 1, d), generator=gen, device="cuda")
        away = uniform(pages, heads, 2, d) + 1.9
        away[:, :, 0] *= -1
        state["bounds"] = (middle + away).to(torch.bfloat16)
        state["scores"] = torch.empty((rows, heads, -(-width // 4) * 4), device="cuda")[:, :, :width]
        state["counts"] = torch.empty((rows, heads), dtype=torch.int32, device="cuda")
        return state
    _pool(state, pages, gen)
    state["sinks"] = torch.randn((case["heads"],), generator=gen, device="cuda") if case["sinks"] else None
    state["selected"] = _select((lengths + PAGE - 1) // PAGE, heads, width, case["k"], gen) if case["k"] else None
    state["out"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty((rows, case["heads"]), device="cuda")
    return state


def _select(counts, heads, width, k, gen):
    """k distinct pages of each row below its count in ascending order for each
    key head, -1 behind them: what a top-k leaves."""
    counts, none = counts.long()[:, None, None], 1 << 30
    keys = torch.rand((counts.shape[0], heads, max(width, k)), generator=gen, device="cuda")
    keys = keys.masked_fill(torch.arange(keys.shape[2], device="cuda") >= counts, 2.0)
    at = keys.topk(k, dim=2, largest=False).indices
    at = at.masked_fill(at >= counts, none).sort(dim=2).values
    return at.masked_fill(at == none, -1).to(torch.int32)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _planned(state):
    return tuple(state[name] for name in ("table", "slots", "positions", "row_table", "seqlens", "starts", "taken"))


def _stored(state):
    """The pool after a store, without the page behind it."""
    pages = state["pages"]
    values = (state["k_pages"][:pages], state["v_pages"][:pages])
    return values + (state["kscale"][:pages], state["vscale"][:pages]) if state["case"]["fp8"] else values


# --- the library's entry points


def _run_own(state):
    import paged_mqa_logits_idx_amd as lib

    case = state["case"]
    op = case["op"]
    if op == "plan":
        lib.idx_plan_batch(state["cached"], state["added"], state["free"], state["table"], state["slots"], state["positions"],
                           state["row_table"], state["seqlens"], state["starts"], state["taken"])
        return _planned(state)
    if op == "store":
        if case["fp8"]:
            lib.idx_store_kv_fp8(state["keys"], state["values"], state["slots"], state["k_pages"], state["v_pages"], state["kscale"],
                                 state["vscale"], num_pages=state["pages"])
        else:
            lib.idx_store_kv_bf16(state["keys"], state["values"], state["slots"], state["k_pages"], state["v_pages"],
                                  num_pages=state["pages"])
        return _stored(state)
    if op == "bounds":
        if case["fp8"]:
            lib.idx_page_bounds_fp8(state["k_pages"], state["kscale"], state["table"], state["lengths"], state["bounds"],
                                    first=state["first"], num_pages=state["pages"])
        else:
            lib.idx_page_bounds_bf16(state["k_pages"], state["table"], state["lengths"], state["bounds"], first=state["first"],
                                     num_pages=state["pages"])
        return state["bounds"][: state["pages"]]
    if op == "scores":
        lib.idx_page_scores(state["q"], state["bounds"], state["table"], state["lengths"], state["scores"], state["counts"],
                            first_pages=1, last_pages=2)
        return state["scores"], state["counts"]
    if case["fp8"]:
        lib.idx_kv_attention_fp8(state["q"], state["k_pages"], state["v_pages"], state["kscale"], state["vscale"], state["table"],
                                 state["selected"], state["lengths"], state["out"], state["lse"], scale=case["dim"] ** -0.5,
                                 sinks=state["sinks"])
    else:
        lib.idx_kv_attention_bf16(state["q"], state["k_pages"], state["v_pages"], state["table"], state["selected"], state["lengths"],
                                  state["out"], state["lse"], scale=case["dim"] ** -0.5, sinks=state["sinks"])
    return state["out"], state["lse"]


# --- the plain form


def _plan_plain(state):
    table, n = state["table"], state["slots"].shape[0]
    cached, added, free = state["cached"].long(), state["added"].long(), state["free"]
    width = table.shape[1]
    low = (cached + PAGE - 1) // PAGE
    high = ((cached + added + PAGE - 1) // PAGE).clamp(max=width)
    need = (high - low).clamp(min=0)
    ends, last = need.cumsum(0), added.cumsum(0)
    j = torch.arange(width, device="cuda")
    rank = (ends - need)[:, None] + j - low[:, None]
    fresh = (j >= low[:, None]) & (j < high[:, None])
    got = torch.where(rank < free.shape[0], free[rank.clamp(0, free.shape[0] - 1)], -1)
    table.copy_(torch.where(fresh, got, table))
    t = torch.arange(n, device="cuda")
    request = torch.searchsorted(last, t, right=True)
    live = request < added.shape[0]
    request = torch.where(live, request, 0)
    position = torch.where(live, cached[request] + t - (last - added)[request], 0)
    column = position // PAGE
    page = torch.where(live & (column < width), table[request, column.clamp(max=width - 1)].long(), -1)
    starts = torch.cat((last.new_zeros(1), last))
    return (table, torch.where(page >= 0, page * PAGE + position % PAGE, -1), position, request.int(),
            torch.where(live, position + 1, 0).int(), starts, ends[-1:])


def _quantised(x):
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _store_plain(state):
    to = torch.where(state["slots"] >= 0, state["slots"], state["pages"] * PAGE)  # tokens without a slot: the page behind
    page, at = to // PAGE, to % PAGE
    if not state["case"]["fp8"]:
        state["k_pages"][page, :, at] = state["keys"]
        state["v_pages"][page, :, at] = state["values"]
        return _stored(state)
    codes, state["kscale"][page, :, at] = _quantised(state["keys"].float())
    state["k_pages"].view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
    codes, state["vscale"][page, :, at] = _quantised(state["values"].float())
    state["v_pages"].view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
    return _stored(state)


def _outwards(x, up):
    """The bf16 next to float32 x that is no less (up) or no more, and finite."""
    bits = x.contiguous().view(torch.int32)
    away = (bits >= 0) if up else (bits < 0)
    bits = torch.where(away, bits + 0xFFFF, bits) & -0x10000
    return bits.view(torch.float32).clamp(-BF16_MAX, BF16_MAX).to(torch.bfloat16)


def _bounds_plain(state):
    case, lengths = state["case"], state["lengths"].long()
    width = state["table"].shape[1]
    most = min(width, case["fresh"] // PAGE + 2) if case["fresh"] else width
    j = state["first"].long()[:, None] // PAGE + torch.arange(most, device="cuda")
    live = j * PAGE < lengths[:, None]
    page = torch.where(live, state["table"].long().gather(1, j.clamp(max=width - 1)), 0)
    if case["fp8"]:
        keys = state["k_pages"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * state["kscale"][page][..., None]
    else:
        keys = state["k_pages"][page].float()
    dead = (j[:, :, None] * PAGE + torch.arange(PAGE, device="cuda") >= lengths[:, None, None])[:, :, None, :, None]
    low, high = keys.masked_fill(dead, math.inf).amin(3), keys.masked_fill(dead, -math.inf).amax(3)
    state["bounds"][torch.where(live, page, state["pages"])] = torch.stack((_outwards(low, False), _outwards(high, True)), 3)
    return state["bounds"][: state["pages"]]


def _scores_plain(state):
    case = state["case"]
    heads, width = case["kv_heads"], state["table"].shape[1]
    bounds = state["bounds"][state["table"].long()].permute(0, 2, 1, 3, 4).float()  # [rows, key heads, pages, 2, D]
    q = state["q"].float().unflatten(1, (heads, -1))
    s = torch.matmul(q.clamp(max=0), bounds[:, :, :, 0].transpose(2, 3)) + torch.matmul(q.clamp(min=0), bounds[:, :, :, 1].transpose(2, 3))
    s = s.amax(2)
    counts = (state["lengths"].long() + PAGE - 1) // PAGE
    j = torch.arange(width, device="cuda")
    left = (counts[:, None] - j)[:, None]
    s = s.masked_fill((j < 1) | (left <= 2), math.inf)
    return s.masked_fill(left <= 0, -math.inf), counts.int()[:, None].expand(-1, heads).contiguous()


def _listed_pages(state):
    """Pages to attend to, as columns of the table, their ids and their live positions."""
    case, width = state["case"], state["table"].shape[1]
    rows, heads = case["rows"], case["kv_heads"]
    j = state["selected"].long() if case["k"] else torch.arange(width, device="cuda").expand(rows, heads, width)
    live = (j >= 0)[..., None] & (j[..., None] * PAGE + torch.arange(PAGE, device="cuda") < state["lengths"].long()[:, None, None, None])
    page = state["table"].long()[torch.arange(rows, device="cuda")[:, None, None], j.clamp(min=0)]
    return page, live.flatten(2)


def _gathered(state, which, page):
    """Keys or values of the pages in 32 bits, [rows, key heads, positions, D]."""
    head = torch.arange(state["case"]["kv_heads"], device="cuda")[:, None]
    if not state["case"]["fp8"]:
        return state[which + "_pages"][page, head].flatten(2, 3).float()
    codes = state[which + "_pages"].view(torch.uint8)[page, head].view(torch.float8_e4m3fn)
    return codes.flatten(2, 3).float() * state[which + "scale"][page, head].flatten(2)[..., None]


def _attend_plain(state):
    case = state["case"]
    page, live = _listed_pages(state)
    q = state["q"].float().unflatten(1, (case["kv_heads"], -1))
    s = torch.matmul(q, _gathered(state, "k", page).transpose(2, 3)) * case["dim"] ** -0.5
    s = s.masked_fill(~live[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    sinks = state["sinks"].view(case["kv_heads"], -1, 1) if case["sinks"] else None
    if sinks is not None:
        top = torch.maximum(top, sinks)
    e = (s - top).exp()
    total = e.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + (sinks - top).exp()
    out = torch.matmul(e, _gathered(state, "v", page)) / total
    return out.flatten(1, 2).to(torch.bfloat16), (top + total.log()).flatten(1)


def _run_plain(state):
    op = state["case"]["op"]
    if op == "plan":
        return _plan_plain(state)
    if op == "store":
        return _store_plain(state)
    if op == "bounds":
        return _bounds_plain(state)
    return _scores_plain(state) if op == "scores" else _attend_plain(state)


# --- the definition in 64 bits


def _e4m3_table():
    """The 256 values of the e4m3 codes: four exponent bits of bias 7, three of
    mantissa, subnormals, no infinities, 0x7F and 0xFF not numbers."""
    code = torch.arange(256, dtype=torch.float64)
    sign, e, m = 1 - 2 * (code >= 128).double(), (code % 128) // 8, code % 8
    value = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)
    value[torch.tensor([0x7F, 0xFF])] = math.nan
    return (sign * value).cuda()


def _to_e4m3(v):
    """The e4m3 values nearest to v (ties to even)."""
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return ((v / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def _wide(values, scales=None):
    """Stored blocks [..., 64, D] in 64 bits, without the scale where none is given."""
    if values.dtype == torch.bfloat16:
        return values.double()
    wide = _e4m3_table()[values.view(torch.uint8).long()]
    return wide if scales is None else wide * scales.double()[..., None]


def exact(case, seed):
    op = case["op"]
    if op == "plan":  # whole numbers only
        return None
    state = prepare(case, seed)
    if op == "store":
        kept = state["slots"] >= 0
        at = state["slots"][kept]
        pages, found = state["pages"], []
        for which, name in (("k", "keys"), ("v", "values")):
            pool, x = _wide(state[which + "_pages"][:pages]), state[name].double()[kept]
            if case["fp8"]:
                scales = state[which + "scale"][:pages].double()
                size = x.abs().amax(-1) / E4M3_MAX
                scales[at // PAGE, :, at % PAGE] = size
                x = _to_e4m3(x / size[..., None])
                found.append(scales)
            pool[at // PAGE, :, at % PAGE] = x
            found.append(pool)
        return (found[1], found[3], found[0], found[2]) if case["fp8"] else tuple(found)
    lengths = state["lengths"].tolist()
    if op == "bounds":
        bounds = state["bounds"][: state["pages"]].double()
        for b, length in enumerate(lengths):
            j = torch.arange(int(state["first"][b]) // PAGE, _pages(length), device="cuda")
            page = state["table"][b].long()[j]
            keys = _wide(state["k_pages"][page], state["kscale"][page] if case["fp8"] else None)
            live = (j[:, None] * PAGE + torch.arange(PAGE, device="cuda") < length)[:, None, :, None]
            bounds[page, :, 0] = torch.where(live, keys, math.inf).min(2).values
            bounds[page, :, 1] = torch.where(live, keys, -math.inf).max(2).values
        return bounds
    heads, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    if op == "scores":
        width = state["table"].shape[1]
        scores = torch.full((case["rows"], heads, width), -math.inf, dtype=torch.float64, device="cuda")
        for b, length in enumerate(lengths):
            count = _pages(length)
            bounds = state["bounds"][state["table"][b, :count].long()].double()
            for h in range(heads):
                q = state["q"][b, h * group : (h + 1) * group].double()
                for part in range(0, count, 1024):
                    lo, hi = bounds[part : part + 1024, h, 0], bounds[part : part + 1024, h, 1]
                    some = scores[b, h, part : part + lo.shape[0]]
                    for one in q:
                        some.copy_(torch.maximum(some, torch.maximum(one * lo, one * hi).sum(-1)))
            scores[b, :, 0] = math.inf
            scores[b, :, max(0, count - 2) : count] = math.inf
        return scores, None
    outs, logs = [], []
    for b, length in enumerate(lengths):
        for h in range(heads):
            j = state["selected"][b, h].long() if case["k"] else torch.arange(_pages(length), device="cuda")
            j = j[j >= 0]
            page = state["table"][b].long()[j]
            live = (j[:, None] * PAGE + torch.arange(PAGE, device="cuda") < length).flatten()
            keys, values = (_wide(state[w + "_pages"][page, h], state[w + "scale"][page, h] if case["fp8"] else None).flatten(0, 1)[live]
                            for w in ("k", "v"))
            s = (state["q"][b, h * group : (h + 1) * group].double() @ keys.T) / case["dim"] ** 0.5
            if case["sinks"]:
                s = torch.cat((s, state["sinks"][h * group : (h + 1) * group].double()[:, None]), 1)
            logs.append(torch.logsumexp(s, 1))
            outs.append(torch.exp(s[:, : keys.shape[0]] - logs[-1][:, None]) @ values)
    shape = (case["rows"], case["heads"])
    return torch.stack(outs).view(*shape, case["dim"]), torch.stack(logs).view(shape)
