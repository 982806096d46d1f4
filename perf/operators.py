"""Measured cases of the operators around the indexer: the norm and rotation of
queries, the norm, rotation and paged store of keys and latents, the read back
of stored slots, and the attention over a paged cache of latents.

    y        = x / sqrt(mean(x^2) + eps) * weight, then the last `rope` values
               rotated pairwise by the angles position * inv_freq
    store    scale = amax / 448, code = e4m3(y / scale), at the page slots given
    load     code * scale of the slots given
    attend   out_h = sum_p softmax_p(scale * <q_h, c_p>) c_p over the selected
             positions p of a row, with an optional sink logit per head in the
             softmax's denominator, and the log of that denominator

`own` chooses between the plain form, elementary torch operations in 32 bits
(angles in 64), and the library's own entry points.  Sizes: 64 query heads,
128-value keys and 64-position pages are the indexer's; 512 is the width of a
latent vector; batches, contexts and the 2048 selected positions are those of
the benchmark's decode and prefill.
"""
import math

import torch

own = False

PAGE = 64
LATENT = 512
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # index queries of one decode step: 64 requests, 64 heads of 128
        {"name": "rotate decode", "op": "rotate", "n": 64, "heads": 64, "dim": 128, "rope": 64, "halves": True, "weight": False},
        # attention queries of one 4096-token prefill: 64 heads of 512
        {"name": "rotate prefill", "op": "rotate", "n": 4096, "heads": 64, "dim": 512, "rope": 64, "halves": False, "weight": True},
        # index keys of one decode step
        {"name": "store decode keys", "op": "store", "n": 64, "dim": 128, "rope": 64, "halves": True, "fp8": True},
        # latents of one long prompt
        {"name": "store prompt latents", "op": "store", "n": 65536, "dim": 512, "rope": 64, "halves": False, "fp8": True},
        # latents of an odd-sized chunk kept in bf16
        {"name": "store chunk bf16", "op": "store", "n": 5633, "dim": 512, "rope": 64, "halves": False, "fp8": False},
        # cached prefix of one request read back: a 22K-token context
        {"name": "load prefix", "op": "load", "n": 5632, "dim": 512, "fp8": True},
        # a whole 1M-token context read back
        {"name": "load long context", "op": "load", "n": 262208, "dim": 512, "fp8": True},
        # one request decoding alone
        {"name": "attend one row", "op": "attend", "rows": 1, "heads": 64, "k": 2048, "context": 8192, "shared": False, "fp8": True, "sinks": True},
        # decode batch over the top-2048 of up to 32768 positions each
        {"name": "attend decode", "op": "attend", "rows": 64, "heads": 64, "k": 2048, "context": 32768, "shared": False, "fp8": True, "sinks": True},
        # odd batch, head count and selection, bf16 cache
        {"name": "attend odd bf16", "op": "attend", "rows": 33, "heads": 40, "k": 777, "context": 8191, "shared": False, "fp8": False, "sinks": False},
        # every cached position (no selection): short contexts, 128 heads
        {"name": "attend whole context", "op": "attend", "rows": 16, "heads": 128, "k": 0, "context": 8192, "shared": False, "fp8": False, "sinks": False},
        # one 4096-token prefill, causal, top-2048 of up to 5632 positions
        {"name": "attend prefill", "op": "attend", "rows": 4096, "heads": 64, "k": 2048, "context": 5632, "shared": True, "fp8": True, "sinks": True},
    ]


def _between(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "store", "load", "attend", "attend"])
    dim = rng.choice([128, 512])
    if op == "rotate":
        heads = rng.randint(1, 128)
        return {"op": op, "n": _between(rng, 1, 4096 * 64 * 512 // (heads * dim)), "heads": heads, "dim": dim,
                "rope": rng.choice([32, 64]), "halves": rng.random() < 0.5, "weight": rng.random() < 0.5}
    if op == "store":
        return {"op": op, "n": _between(rng, 1, 65536), "dim": dim, "rope": rng.choice([32, 64]), "halves": rng.random() < 0.5,
                "fp8": rng.random() < 0.7}
    if op == "load":
        fp8 = rng.random() < 0.7
        return {"op": op, "n": _between(rng, 1, 262208 if fp8 else 196608), "dim": dim, "fp8": fp8}
    shared = rng.random() < 0.4
    heads = rng.choice([64, 128, rng.randint(1, 128)])
    if shared:  # a prefill chunk of one request
        rows, context, k = _between(rng, 64, 4096), _between(rng, 64, 5632), _between(rng, 16, 2048)
    else:  # a decode batch
        rows, context, k = _between(rng, 1, 64), _between(rng, 1, 32768), rng.choice([0, _between(rng, 1, 2048)])
    seen = min(k, context) if k else context
    rows = max(1, min(rows, 4096 * 64 * 2048 // (seen * max(heads, 64))))
    return {"op": "attend", "rows": rows, "heads": heads, "k": k, "context": context, "shared": shared, "fp8": rng.random() < 0.6,
            "sinks": rng.random() < 0.5}


def _lengths(case):
    """Positions that each row sees: a causal ramp in a prefill, a spread from a
    quarter of the context up in a decode batch."""
    rows, context = case["rows"], case["context"]
    if case["shared"]:
        return [-(-context * (b + 1) // rows) for b in range(rows)]
    return [context - (3 * context * b // 4) // rows for b in range(rows)]


def work(case):
    op = case["op"]
    if op == "rotate":
        n, values = case["n"], case["n"] * case["heads"] * case["dim"]
        return {"bytes": 4 * values + 8 * n + 2 * case["rope"] + (4 * case["dim"] if case["weight"] else 0), "flops": 4 * values}
    if op == "store":
        n, d = case["n"], case["dim"]
        return {"bytes": n * (2 * d + 16 + (d + 4 if case["fp8"] else 2 * d)) + 4 * d + 2 * case["rope"], "flops": 6 * n * d}
    if op == "load":
        n, d = case["n"], case["dim"]
        return {"bytes": n * (2 * d + 8 + (d + 4 if case["fp8"] else 2 * d)), "flops": n * d}
    rows, heads, k, lengths = case["rows"], case["heads"], case["k"], _lengths(case)
    seen = sum(min(k, n) for n in lengths) if k else sum(lengths)
    # of a shared cache each position is read once, of others what each row selects
    read = min(seen, case["context"]) if case["shared"] else seen
    per_position = LATENT + 4 if case["fp8"] else 2 * LATENT
    return {"bytes": read * per_position + rows * heads * (4 * LATENT + 4) + 4 * rows * (k + 1) + (4 * heads if case["sinks"] else 0)
            + read // PAGE * 4, "flops": 4 * seen * heads * LATENT}


def _inv_freq(rope):
    return (10000.0 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)).float()


def _codes(shape, gen):
    """e4m3 codes of normal values over their largest of 448."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    op = case["op"]
    if op in ("rotate", "store"):
        shape = (case["n"], case["heads"], case["dim"]) if op == "rotate" else (case["n"], case["dim"])
        size = torch.rand((case["n"],) + (1,) * (len(shape) - 1), generator=gen, device="cuda") * 3 + 0.2
        state["x"] = (torch.randn(shape, generator=gen, device="cuda") * size).to(torch.bfloat16)
        state["positions"] = torch.randint(0, 1 << 20, (case["n"],), generator=gen, device="cuda")
        state["inv_freq"] = _inv_freq(case["rope"])
        weight = 1 + 0.1 * torch.randn((case["dim"],), generator=gen, device="cuda")
        state["weight"] = weight if op == "store" or case["weight"] else None
    if op == "rotate":
        state["out"] = torch.empty_like(state["x"])
    if op in ("store", "load"):
        # slots in random order over a pool with as many again, a few tokens
        # without a slot in a stored batch; the page behind the pool takes
        # what the plain form has to put somewhere
        n, d = case["n"], case["dim"]
        pages = -(-2 * n // PAGE)
        slots = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:n].contiguous()
        if op == "store" and n > 8:
            slots[torch.randint(0, n, (n // 64 + 1,), generator=gen, device="cuda")] = -1
        state["slots"], state["pages"] = slots, pages
        if case["fp8"]:
            state["pool"] = _codes((pages + 1, PAGE, d), gen).view(torch.uint8)
            state["scales"] = torch.rand((pages + 1, PAGE), generator=gen, device="cuda") * 0.01 + 0.005
        else:
            state["pool"] = torch.randn((pages + 1, PAGE, d), generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        if op == "load":
            state["out"] = torch.empty((n, d), device="cuda", dtype=torch.bfloat16)
    if op == "attend":
        rows, context, k = case["rows"], case["context"], case["k"]
        width = -(-context // PAGE)
        pages = width if case["shared"] else rows * width
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        state["table"] = order.reshape(1 if case["shared"] else rows, width)
        lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        if not case["shared"]:
            lengths = lengths[torch.randperm(rows, generator=gen, device="cuda")].contiguous()
        state["lengths"] = lengths
        # latents and queries as their norms leave them: about one per value
        if case["fp8"]:
            fused = torch.empty((pages, PAGE * (LATENT + 4)), dtype=torch.uint8, device="cuda")
            fused[:, : PAGE * LATENT] = _codes((pages, PAGE * LATENT), gen).view(torch.uint8)
            scales = (torch.rand((pages, PAGE), generator=gen, device="cuda") + 0.6) / 110.0
            fused[:, PAGE * LATENT :] = scales.view(torch.uint8)
            state["pool"] = fused
        else:
            state["pool"] = torch.randn((pages, PAGE, LATENT), generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        state["q"] = (1.5 * torch.randn((rows, case["heads"], LATENT), generator=gen, device="cuda")).to(torch.bfloat16)
        state["sinks"] = torch.randn((case["heads"],), generator=gen, device="cuda") if case["sinks"] else None
        state["selected"] = _select(lengths, context, k, gen) if k else None
        state["out"] = torch.empty_like(state["q"])
        state["lse"] = torch.empty((rows, case["heads"]), device="cuda", dtype=torch.float32)
    return state


def _select(lengths, context, k, gen):
    """k distinct positions of each row below its length in ascending order, -1
    behind them: what a top-k leaves."""
    lengths, none = lengths.long()[:, None], 1 << 30
    keys = torch.rand((lengths.shape[0], max(context, k)), generator=gen, device="cuda")
    keys = keys.masked_fill(torch.arange(keys.shape[1], device="cuda") >= lengths, 2.0)
    at = keys.topk(k, dim=1, largest=False).indices
    at = at.masked_fill(at >= lengths, none).sort(dim=1).values
    return at.masked_fill(at == none, -1).to(torch.int32)


_SCALE = LATENT ** -0.5


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --- the library's entry points


def _run_own(state):
    import paged_mqa_logits_idx_amd as lib

    case = state["case"]
    op = case["op"]
    if op == "rotate":
        lib.idx_norm_rope(state["x"], state["positions"], state["inv_freq"], state["out"], weight=state["weight"], eps=EPS,
                          halves=case["halves"])
        return state["out"]
    if op == "store":
        d, pages = case["dim"], state["pages"]
        if case["fp8"]:
            lib.idx_norm_rope_store_fp8(state["x"], state["positions"], state["inv_freq"], state["slots"], state["pool"], state["scales"],
                                        weight=state["weight"], eps=EPS, halves=case["halves"], num_pages=pages,
                                        kv_page_stride=PAGE * d, kscale_page_stride=PAGE * 4)
        else:
            lib.idx_norm_rope_store_bf16(state["x"], state["positions"], state["inv_freq"], state["slots"], state["pool"],
                                         weight=state["weight"], eps=EPS, halves=case["halves"], num_pages=pages)
        return _stored(state)
    if op == "load":
        if case["fp8"]:
            lib.idx_load_slots_fp8(state["pool"], state["scales"], state["slots"], state["out"], num_pages=state["pages"],
                                   kv_page_stride=PAGE * case["dim"], kscale_page_stride=PAGE * 4)
        else:
            lib.idx_load_slots_bf16(state["pool"], state["slots"], state["out"], num_pages=state["pages"])
        return state["out"]
    pages = state["pool"].shape[0]
    if case["fp8"]:
        lib.idx_latent_attention_fp8(state["q"], state["pool"], state["pool"].data_ptr() + PAGE * LATENT, state["table"],
                                     state["selected"], state["lengths"], state["out"], state["lse"], sinks=state["sinks"],
                                     scale=_SCALE, num_pages=pages)
    else:
        lib.idx_latent_attention_bf16(state["q"], state["pool"], state["table"], state["selected"], state["lengths"], state["out"],
                                      state["lse"], sinks=state["sinks"], scale=_SCALE, num_pages=pages)
    return state["out"], state["lse"]


def _stored(state):
    """The pool after a store, without the page behind it."""
    pages = state["pages"]
    if state["case"]["fp8"]:
        return state["pool"][:pages].view(torch.float8_e4m3fn), state["scales"][:pages]
    return state["pool"][:pages]


# --- the plain form


def _normed(state):
    """The normed and rotated vectors in 32 bits."""
    case = state["case"]
    x = state["x"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if state["weight"] is not None:
        y = y * state["weight"]
    angle = state["positions"].double()[:, None] * state["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if y.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    rope = case["rope"]
    head, tail = y[..., :-rope], y[..., -rope:]
    if case["halves"]:
        a, b = tail[..., : rope // 2], tail[..., rope // 2 :]
        tail = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = tail[..., 0::2], tail[..., 1::2]
        tail = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((head, tail), -1)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "rotate":
        return _normed(state).to(torch.bfloat16)
    if op == "store":
        y = _normed(state)
        to = torch.where(state["slots"] >= 0, state["slots"], state["pages"] * PAGE)  # tokens without a slot: the page behind
        flat = state["pool"].view(-1, case["dim"])
        if case["fp8"]:
            amax = y.abs().amax(-1)
            scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            flat[to] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            state["scales"].view(-1)[to] = scale
        else:
            flat[to] = y.to(torch.bfloat16)
        return _stored(state)
    if op == "load":
        got = state["pool"].view(-1, case["dim"])[state["slots"]]
        if case["fp8"]:
            got = got.view(torch.float8_e4m3fn).float() * state["scales"].view(-1)[state["slots"]][:, None]
        return got.to(torch.bfloat16)
    lengths = state["lengths"].long()[:, None]
    at = state["selected"].long() if state["selected"] is not None else torch.arange(case["context"], device="cuda")[None]
    at = at.expand(case["rows"], -1)
    live = (at >= 0) & (at < lengths)
    at = at.clamp(min=0)
    page = state["table"].long().expand(case["rows"], -1).gather(1, at // PAGE)
    if case["fp8"]:
        pool = state["pool"]
        codes = pool[:, : PAGE * LATENT].unflatten(1, (PAGE, LATENT))[page, at % PAGE]
        c = codes.view(torch.float8_e4m3fn).float() * pool[:, PAGE * LATENT :].view(torch.float32)[page, at % PAGE][..., None]
    else:
        c = state["pool"][page, at % PAGE].float()
    s = torch.matmul(state["q"].float(), c.transpose(1, 2)) * _SCALE
    s = s.masked_fill(~live[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    if state["sinks"] is not None:
        top = torch.maximum(top, state["sinks"][:, None])
    e = (s - top).exp()
    total = e.sum(-1, keepdim=True)
    if state["sinks"] is not None:
        total = total + (state["sinks"][:, None] - top).exp()
    out = torch.matmul(e, c) / total
    return out.to(torch.bfloat16), (top + total.log())[..., 0]


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


def _exact_vectors(state):
    case, x = state["case"], state["x"].double()
    x = x if x.dim() == 3 else x[:, None]
    y = x / ((x * x).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
    if state["weight"] is not None:
        y = y * state["weight"].double()
    first, rope = case["dim"] - case["rope"], case["rope"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), state["positions"].double()[:, None, None] * state["inv_freq"].double())
    pair = torch.arange(rope // 2, device="cuda")
    one = first + (pair if case["halves"] else 2 * pair)
    two = one + (rope // 2 if case["halves"] else 1)
    turned = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = turned.real, turned.imag
    return y if case["op"] == "rotate" else y[:, 0]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return _exact_vectors(state)
    if op in ("store", "load"):
        flat, pages, d = state["pool"].view(-1, case["dim"]), state["pages"], case["dim"]
        slots = state["slots"]
        if case["fp8"]:
            values, scales = _e4m3_table()[flat.long()], state["scales"].double().view(-1)
        else:
            values, scales = flat.double(), None
        if op == "load":
            return values[slots] * scales[slots, None] if case["fp8"] else values[slots]
        y, kept = _exact_vectors(state)[slots >= 0], slots[slots >= 0]
        if not case["fp8"]:
            values[kept] = y
            return values[: pages * PAGE].view(pages, PAGE, d)
        scales[kept] = y.abs().amax(-1) / E4M3_MAX
        values[kept] = _to_e4m3(y / scales[kept, None])
        return values[: pages * PAGE].view(pages, PAGE, d), scales[: pages * PAGE].view(pages, PAGE)
    table, lengths = _e4m3_table(), state["lengths"].tolist()
    outs, logs = [], []
    for b, length in enumerate(lengths):
        at = state["selected"][b].long() if state["selected"] is not None else torch.arange(length, device="cuda")
        live = (at >= 0) & (at < length)
        at = torch.where(live, at, 0)
        page = state["table"][0 if case["shared"] else b].long()[at // PAGE]
        slot = at % PAGE
        if case["fp8"]:
            rows = state["pool"][page[:, None], slot[:, None] * LATENT + torch.arange(LATENT, device="cuda")]
            c = table[rows.long()] * state["pool"].view(torch.float32)[page, PAGE * LATENT // 4 + slot].double()[:, None]
        else:
            c = state["pool"][page, slot].double()
        s = (state["q"][b].double() @ c.T) / LATENT ** 0.5
        s = torch.where(live, s, -math.inf)
        if state["sinks"] is not None:
            s = torch.cat((s, state["sinks"].double()[:, None]), 1)
        logs.append(torch.logsumexp(s, 1))
        outs.append(torch.exp(s[:, : c.shape[0]] - logs[-1][:, None]) @ c)
    return torch.stack(outs), torch.stack(logs)
