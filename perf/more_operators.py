"""What a server does around the decode step, as measured cases:

  prompt  causal attention over whole prompts, or over pieces of them behind earlier tokens: packed sequences of
          different lengths, several query heads a key head
  tree    attention of a tree of drafted tokens over the paged cache (16-bit, or quantised to 8 or 4 bits)
  plan    page tables, slots, positions and row starts from the sequences' lengths, and the pages' way back

``run`` computes them in plain torch operations, or, where ``own`` is true, through the library's calls.  Head counts
are those of Llama-3.1-8B (32 query heads, 8 key heads), Qwen3-14B (40/8), Llama-3.3-70B and Qwen3-32B (64/8), with 128
columns a head; a few cases and the drawn ones have others.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
BITS = {"16": 16, "mx8": 8, "mx4": 4}
BLOCK = 32                                  # columns of a cached row that share one power-of-two scale
TOP = {"mx8": 448.0, "mx4": 6.0}            # largest e4m3 and e2m1 values
MX4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _prompt(name, B, hq, hk, D, dtype, longest, past, ragged, fused):
    return {"name": name, "op": "prompt", "B": B, "hq": hq, "hk": hk, "D": D, "dtype": dtype, "longest": longest,
            "past": past, "ragged": ragged, "fused": fused}


def _tree(name, B, N, hq, hk, D, dtype, fmt, page, longest, ragged):
    return {"name": name, "op": "tree", "B": B, "N": N, "hq": hq, "hk": hk, "D": D, "dtype": dtype, "fmt": fmt,
            "page": page, "longest": longest, "ragged": ragged}


def _plan(name, B, page, held, add, ragged, mixed):
    return {"name": name, "op": "plan", "B": B, "page": page, "held": held, "add": add, "ragged": ragged, "mixed": mixed}


def listed():
    return [
        # a conversation's first words: one short prompt, latency
        _prompt("prompt_short", 1, 32, 8, 128, "fp16", 37, 0, False, False),
        # a batch of new requests of every length
        _prompt("prompt_batch", 16, 32, 8, 128, "bf16", 1024, 0, True, False),
        # odd prompts of a small model with narrow heads, rows inside a fused q+k+v buffer
        _prompt("prompt_odd", 3, 12, 4, 64, "fp16", 1237, 0, True, True),
        # pieces of prompts, cut so that decoding goes on beside them: most keys lie before the piece
        _prompt("prompt_piece", 4, 40, 8, 128, "fp16", 500, 8192, True, False),
        # one long document on 64 query heads
        _prompt("prompt_long", 1, 64, 8, 128, "bf16", 8192, 0, False, False),
        # one conversation with a few drafted tokens: latency
        _tree("tree_small", 1, 8, 32, 8, 128, "fp16", "16", 16, 300, False),
        # an ordinary verification step of sequences of all lengths, quantised cache
        _tree("tree_step", 16, 24, 32, 8, 128, "bf16", "mx8", 64, 8192, True),
        # many conversations with small trees, unquantised cache
        _tree("tree_batch", 32, 12, 40, 8, 128, "bf16", "16", 64, 2048, True),
        # one long document held in 4 bits, the largest tree
        _tree("tree_long", 1, 64, 64, 8, 128, "fp16", "mx4", 128, 131071, False),
        # a decode step of 32 sequences: a row each, now and then a page
        _plan("plan_step", 32, 64, 8192, 1, True, False),
        # new prompts and finished sequences of every length
        _plan("plan_prompts", 48, 64, 0, 8192, True, True),
        # a large server's verification step: a tree a sequence, small pages
        _plan("plan_drafts", 4096, 16, 4096, 16, False, False),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    op = rng.choice(("prompt", "prompt", "tree", "tree", "plan"))
    dtype = rng.choice(("fp16", "bf16"))
    D = rng.choice((64, 128, 128, 256))
    hk = rng.choice((1, 2, 4, 8, 8, 16))
    hq = hk * rng.choice((1, 2, 3, 4, 5, 8))
    if op == "prompt":
        # pairs of a query and a key on all heads, and their columns, stay below the longest listed case's
        B = size(1, 32)
        pairs = 64 * 8192 * 8192 * 128 // (B * hq * max(D, 128))
        longest = size(1, min(8192, math.isqrt(pairs)))
        past = rng.choice((0, 0, 1)) * size(1, max(1, min(16384, pairs // longest - longest)))
        c = _prompt("", B, hq, hk, D, dtype, longest, past, rng.random() < 0.7, rng.random() < 0.4)
    elif op == "tree":
        B, N = size(1, 48), size(1, 64)
        # rows of the cache, and drafts times tokens, stay below the longest listed case's
        tokens = min(131072 * 8 * 128 // (hk * D), 64 * 64 * 131072 * 128 // (N * hq * D))
        longest = max(N, size(1, max(1, tokens // B)))
        c = _tree("", B, N, hq, hk, D, dtype, rng.choice(("16", "mx8", "mx4")), rng.choice((16, 32, 64, 128, 256)),
                  longest, rng.random() < 0.7)
    else:
        B = size(1, 4096)
        add = size(1, min(8192, 262144 // B))
        c = _plan("", B, rng.choice((16, 32, 64, 128, 256)), rng.choice((0, 1)) * size(1, 4096), add,
                  rng.random() < 0.7, rng.random() < 0.5)
    del c["name"]
    return c


# ---- what a case says beside its numbers: lengths and trees, the same for every seed --------------------------------

def _rng(case):
    return random.Random(" ".join(str(case[k]) for k in sorted(case) if k != "name"))


def _pieces(case):
    """(queries, keys) of each sequence of a prompt case."""
    r, B, longest = _rng(case), case["B"], case["longest"]
    nq = [r.randint(1, longest) if case["ragged"] else longest for _ in range(B)]
    nq[0] = longest
    past = [r.randint(0, case["past"]) if case["ragged"] else case["past"] for _ in range(B)]
    past[-1] = case["past"]
    return nq, [a + b for a, b in zip(nq, past)]


def _drafts(case):
    """Tokens of each sequence of a tree case, drafts included, and the trees' masks: bit j of row i is set where
    draft j is i or leads to it."""
    r, B, N, longest = _rng(case), case["B"], case["N"], case["longest"]
    lens = [r.randint(N, longest) if case["ragged"] else longest for _ in range(B)]
    lens[0] = longest
    masks = []
    for _ in range(B):
        row = []
        for i in range(N):
            parent = r.randint(max(-1, i - 6), i - 1)
            row.append((row[parent] if parent >= 0 else 0) | 1 << i)
        masks.append(row)
    return lens, masks


def _requests(case):
    """Tokens held and asked for by each sequence of a plan case: with `mixed` a third of the sequences end, giving
    back what they hold, and some are padding."""
    r, B = _rng(case), case["B"]
    held = [r.randint(0, case["held"]) for _ in range(B)]
    adds = [r.randint(0, case["add"]) if case["ragged"] and case["add"] > 1 else case["add"] for _ in range(B)]
    if case["mixed"]:
        for b in range(B):
            kind = r.random()
            if kind < 0.3:                                      # ends
                held[b] = r.randint(1, case["held"] + case["add"])
                adds[b] = -held[b]
            elif kind < 0.35:                                   # padding
                held[b], adds[b] = -1, 3
    return held, adds


def _plan_sizes(case):
    """Rows of the two calls of a pass (what is asked for, and its undoing), pages a sequence, pages in all."""
    held, adds = _requests(case)
    rows = sum(a for h, a in zip(held, adds) if h >= 0 and a > 0)
    back = sum(-a for h, a in zip(held, adds) if h >= 0 and a < 0)
    page = case["page"]
    width = max(1, -(-(case["held"] + case["add"]) // page))
    pages = sum(-(-(max(h, 0) + max(a, 0)) // page) for h, a in zip(held, adds))
    return rows, back, width, pages + 5


def _row_bytes(case):
    """Bytes of one token's row of one key head in the cache."""
    D, bits = case["D"], BITS[case["fmt"]]
    return D * bits // 8 + (D // BLOCK if bits < 16 else 0)


def work(case):
    if case["op"] == "prompt":
        nq, nk = _pieces(case)
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(nq, nk))
        return {"bytes": 4 * case["D"] * (case["hq"] * sum(nq) + case["hk"] * sum(nk)),
                "flops": 4 * case["D"] * case["hq"] * pairs}
    if case["op"] == "tree":
        lens, masks = _drafts(case)
        N, rows = case["N"], 2 * case["hk"] * sum(lens)
        seen = sum(N * (n - N) + sum(bin(m).count("1") for m in row) for n, row in zip(lens, masks))
        return {"bytes": rows * _row_bytes(case) + case["B"] * N * (case["hq"] * case["D"] * 4 + 8),
                "flops": 4 * case["D"] * case["hq"] * seen}
    rows, back, _, pages = _plan_sizes(case)
    return {"bytes": 2 * 20 * case["B"] + 12 * (rows + back) + 8 * 2 * ((rows + back) // case["page"]),
            "flops": 20 * case["B"] + 6 * (rows + back)}


# ---- inputs -------------------------------------------------------------------------------------------------------

def _kv_rows(g, T, hk, D, dt):
    """Keys and values as projections give them: keys with a few strong columns, values without."""
    k = torch.randn((T, hk, D), generator=g, device="cuda")
    k *= torch.exp(0.5 * torch.randn((1, hk, D), generator=g, device="cuda"))
    v = torch.randn((T, hk, D), generator=g, device="cuda")
    return k.to(dt), v.to(dt)


def _starts(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).int()


def _inputs(case, seed):
    """The case's tensors from the seed alone, the same for every side."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "plan":
        held, adds = _requests(case)
        page, (rows, back, width, n_pages) = case["page"], _plan_sizes(case)
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        table = torch.full((case["B"], width), -1, dtype=torch.int32)
        at, host = 0, order.cpu()
        for b, h in enumerate(held):
            c = -(-max(h, 0) // page)
            table[b, :c] = host[at:at + c]
            at += c
        return {"table": table.cuda(), "lens": torch.tensor(held, dtype=torch.int32, device="cuda"),
                "free": torch.cat((order[at:], torch.full((at,), -1, dtype=torch.int32, device="cuda"))),
                "n_free": torch.tensor([n_pages - at], dtype=torch.int32, device="cuda"),
                "adds": torch.tensor(adds, dtype=torch.int32, device="cuda")}
    dt, D, hq, hk = DTYPES[case["dtype"]], case["D"], case["hq"], case["hk"]
    if case["op"] == "prompt":
        nq, nk = _pieces(case)
        T, Tk = sum(nq), sum(nk)
        q = (1.5 * torch.randn((T, hq, D), generator=g, device="cuda")).to(dt)
        k, v = _kv_rows(g, Tk, hk, D, dt)
        if case["fused"]:
            if T == Tk:
                qkv = torch.cat((q.flatten(1), k.flatten(1), v.flatten(1)), 1)
                q = qkv[:, :hq * D].unflatten(1, (hq, D))
                k = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
                v = qkv[:, (hq + hk) * D:].unflatten(1, (hk, D))
            else:
                kv = torch.cat((k.flatten(1), v.flatten(1)), 1)
                k, v = kv[:, :hk * D].unflatten(1, (hk, D)), kv[:, hk * D:].unflatten(1, (hk, D))
        return {"q": q, "k": k, "v": v, "starts": _starts(nq), "k_starts": _starts(nk)}
    (lens, masks), page, B = _drafts(case), case["page"], case["B"]
    n_pages = sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.zeros((B, -(-case["longest"] // page)), dtype=torch.int32, device="cuda")
    at, chunks = 0, []
    for b, n in enumerate(lens):
        c = -(-n // page)
        table[b, :c] = order[at:at + c]
        i = torch.arange(n, device="cuda")
        chunks.append(order[at + i // page].long() * page + i % page)
        at += c
    slots = torch.cat(chunks)
    k, v = _kv_rows(g, slots.shape[0], hk, D, dt)
    q = (1.5 * torch.randn((B, case["N"], hq, D), generator=g, device="cuda")).to(dt)
    visible = [[m - (1 << 64) if m >> 63 else m for m in row] for row in masks]
    return {"pages": n_pages, "slots": slots, "k": k, "v": v, "q": q, "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "visible": torch.tensor(visible, dtype=torch.int64, device="cuda")}


def prepare(case, seed):
    x = _inputs(case, seed)
    state = {"case": case}
    if case["op"] == "plan":
        rows, back, width, n_pages = _plan_sizes(case)
        state.update({"adds": x["adds"], "undo": -x["adds"], "rows": rows, "back": back})
        if own:
            import sparse_matrix_vector_amd as nm
            state["pages"] = nm.KVPages(case["B"], width, n_pages, case["page"])
            for name in ("table", "lens", "free", "n_free"):
                getattr(state["pages"], name).copy_(x[name])
        else:
            state["pages"] = {name: x[name] for name in ("table", "lens", "free", "n_free")}
    elif case["op"] == "tree":
        if own:
            import sparse_matrix_vector_amd as nm
            cache = nm.KVCache(x["pages"], case["page"], case["hk"], case["D"], DTYPES[case["dtype"]], case["fmt"])
            nm.kv_write(cache, x["k"], x["v"], x["slots"])
        else:
            cache = [_plain_cached(case, t, x["slots"], x["pages"] * case["page"]) for t in (x["k"], x["v"])]
        state.update({n: x[n] for n in ("q", "table", "lens", "visible")}, cache=cache)
    else:
        state.update(x)
        state["nq"], state["nk"] = _pieces(case)
    torch.cuda.synchronize()
    return state


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if case["op"] == "plan":
        # a step and its undoing (drafts that are refused; sequences that end), so that a state can be used again
        p = state["pages"]
        if own:
            import sparse_matrix_vector_amd as nm
            out = nm.kv_plan(p, state["adds"], state["rows"])
            back = nm.kv_plan(p, state["undo"], state["back"])
            return (*out, *back, p.table, p.lens, p.free, p.n_free)
        out = _plain_plan(case, p, state["adds"], state["rows"])
        back = _plain_plan(case, p, state["undo"], state["back"])
        return (*out, *back, p["table"], p["lens"], p["free"], p["n_free"])
    if own:
        import sparse_matrix_vector_amd as nm
        if case["op"] == "prompt":
            return nm.attn_prompt(state["q"], state["k"], state["v"], state["starts"],
                                  k_starts=state["k_starts"] if case["past"] else None)
        return nm.attn_tree(state["q"], state["cache"], state["table"], state["lens"], state["visible"],
                            max_len=case["longest"])
    return _plain_prompt(case, state) if case["op"] == "prompt" else _plain_tree(case, state)


# ---- plain forms --------------------------------------------------------------------------------------------------

def _softmax_times(s, v):
    """softmax(s) v over the last axis of s, zeros where a row is all -inf."""
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_prompt(case, state):
    B, hq, hk, D = (case[n] for n in ("B", "hq", "hk", "D"))
    G, L, M = hq // hk, case["longest"], max(state["nk"])
    i, j = torch.arange(L, device="cuda"), torch.arange(M, device="cuda")
    qs, ks = state["starts"].long(), state["k_starts"].long()
    nq, nk = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    qi = (qs[:-1, None] + i).clamp_(max=state["q"].shape[0] - 1)                       # [B][L]
    kj = (ks[:-1, None] + j).clamp_(max=state["k"].shape[0] - 1)
    q = (state["q"].float()[qi] / math.sqrt(D)).view(B, L, hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, hk, G * L, D)
    k = state["k"].float()[kj].permute(0, 2, 3, 1).contiguous()                        # [B][hk][D][M]
    v = state["v"].float()[kj].transpose(1, 2).contiguous()                            # [B][hk][M][D]
    s = torch.matmul(q, k).view(B, hk, G, L, M)
    seen = j <= (i[None, :] + (nk - nq)[:, None])[:, :, None]                          # [B][L][M]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    o = _softmax_times(s.view(B, hk, G * L, M), v)
    o = o.view(B, hk, G, L, D).permute(0, 3, 1, 2, 4).reshape(B * L, hq, D)
    at = torch.repeat_interleave(torch.arange(B, device="cuda") * L - qs[:-1], nq, output_size=state["q"].shape[0])
    return o[at + torch.arange(state["q"].shape[0], device="cuda")].to(state["q"].dtype)


def _plain_quantise(x, fmt):
    """Codes and scales (the powers of two themselves): the scale is the least one under which the block's largest
    magnitude does not pass the largest code."""
    blocks = x.float().unflatten(-1, (-1, BLOCK))
    amax = blocks.abs().amax(-1)
    m, e = torch.frexp(amax)
    top, shift = (0.875, 9) if fmt == "mx8" else (0.75, 3)           # 448 = 0.875 * 2^9, 6 = 0.75 * 2^3
    e = torch.where(m <= top, e - shift, e - shift + 1)
    e = torch.where(amax == 0, torch.full_like(e, -126), e.clamp(-126, 127))
    scale = torch.ldexp(torch.ones_like(amax), e)
    y = blocks / scale[..., None]
    if fmt == "mx8":
        return y.to(torch.float8_e4m3fn).flatten(-2), scale
    a = y.abs()                                                      # nearest e2m1 value, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + 8 * (y < 0)).to(torch.uint8).flatten(-2), scale


def _plain_cached(case, x, slots, n_slots):
    """What a cache of n_slots slots holds of the rows x: 16-bit values, or codes and scales."""
    hk, D, fmt = case["hk"], case["D"], case["fmt"]
    if fmt == "16":
        held = torch.zeros((n_slots, hk, D), dtype=x.dtype, device="cuda")
        held[slots] = x
        return held
    codes, scale = _plain_quantise(x, fmt)
    held = torch.zeros((n_slots, hk, D), dtype=torch.uint8, device="cuda"), \
        torch.zeros((n_slots, hk, D // BLOCK), device="cuda")
    held[0][slots] = codes.view(torch.uint8)
    held[1][slots] = scale
    return held


def _plain_read(case, held, slots):
    if case["fmt"] == "16":
        return held[slots].float()
    codes = held[0][slots]
    if case["fmt"] == "mx8":
        y = codes.view(torch.float8_e4m3fn).float()
    else:
        values = torch.tensor(MX4_VALUES + tuple(-x for x in MX4_VALUES), device="cuda")
        y = values[codes.int()]
    return (y.unflatten(-1, (-1, BLOCK)) * held[1][slots][..., None]).flatten(-2)


def _plain_tree(case, state):
    B, N, hq, hk, D, L, page = (case[n] for n in ("B", "N", "hq", "hk", "D", "longest", "page"))
    G = hq // hk
    q = (state["q"].float() / math.sqrt(D)).view(B, N, hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, hk, N * G, D)
    t = torch.arange(L, device="cuda")
    slots = state["table"].long()[:, t // page] * page + t % page                     # [B][L]
    k, v = (_plain_read(case, held, slots) for held in state["cache"])                # [B][L][hk][D]
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(B, hk, N, G, L)
    j = t - (state["lens"].long()[:, None] - N)                                       # [B][L]: which draft, if any
    bit = state["visible"][:, :, None] >> j.clamp(0, 63)[:, None, :] & 1              # [B][N][L]
    seen = (j < 0)[:, None, :] | (j < N)[:, None, :] & (bit == 1)
    s.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    o = _softmax_times(s.view(B, hk, N * G, L), v.transpose(1, 2).contiguous())
    return o.view(B, hk, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D).to(state["q"].dtype)


def _owner(ends, count, last):
    """Which sequence each of 0 .. count - 1 belongs to, by the sequences' ends (the last one for those behind)."""
    return torch.searchsorted(ends, torch.arange(count, device="cuda"), right=True).clamp_(max=last)


def _plain_plan(case, p, adds, rows):
    """One planned step: pages of dropped tokens go back, then each sequence in turn gets what it asks for."""
    page, B = case["page"], case["B"]
    n_pages, width = p["free"].shape[0], p["table"].shape[1]
    lens, adds, n_free = p["lens"].long(), adds.long(), p["n_free"].long()
    k, zero = torch.arange(n_pages, device="cuda"), torch.zeros_like(lens)
    live = lens >= 0
    held = torch.where(live, (lens + page - 1) // page, zero)
    drop = torch.where(live & (adds < 0), torch.minimum(-adds, lens), zero)
    grow = torch.where(live & (adds > 0) & ((lens + adds + page - 1) // page <= width), adds, zero)
    freed = torch.where(drop > 0, held - (lens - drop + page - 1) // page, zero)
    # freed pages onto the list, the first one on top
    ends = freed.cumsum(0)
    b = _owner(ends, n_pages, B - 1)
    given = p["table"][b, (held[b] - ends[b] + k).clamp_(0, width - 1)]
    free = torch.cat((p["free"], p["free"][:1]))
    free[torch.where(k < ends[-1], n_free + ends[-1] - 1 - k, n_pages)] = given
    free, room = free[:n_pages], n_free + ends[-1]
    # what is asked for, as long as pages and rows last
    want = torch.where(grow > 0, (lens + grow + page - 1) // page - held, zero)
    ok = (want.cumsum(0) <= room) & (grow.cumsum(0) <= rows)
    grow, want = torch.where(ok, grow, zero), torch.where(ok, want, zero)
    ends = want.cumsum(0)
    b = _owner(ends, n_pages, B - 1)
    at = b * width + held[b] + want[b] - ends[b] + k
    table = torch.cat((p["table"].flatten(), p["table"].flatten()[:1]))
    table[torch.where(k < ends[-1], at, B * width)] = free[(room - 1 - k).clamp_(min=0)]
    p["table"], p["free"], p["n_free"] = table[:-1].view(B, width), free, (room - ends[-1]).int()
    p["lens"] = (lens + grow - drop).int()
    # the rows
    starts = torch.cat((grow.new_zeros(1), grow.cumsum(0)))
    r = torch.arange(rows, device="cuda")
    b = _owner(starts[1:], rows, B - 1)
    pos = lens[b] + r - starts[b]
    slot = p["table"][b, (pos // page).clamp_(0, width - 1)].long() * page + pos % page
    inside = r < starts[-1]
    return (starts.int(), torch.where(inside, slot, torch.full_like(slot, -1)),
            torch.where(inside, pos, torch.zeros_like(pos)).int(), (grow - drop).int())


# ---- from the definitions, in 64 bits -----------------------------------------------------------------------------

def _exact_cached(x, fmt):
    """The value that the cache holds for each element of x: the nearest of the format's grid."""
    x = x.double()
    if fmt == "16":
        return x
    if fmt == "mx8":
        grid = [n * 2.0 ** -9 for n in range(8)] + [(8 + n) * 2.0 ** (e - 10) for e in range(1, 16) for n in range(8)]
        grid = grid[:-1]
    else:
        grid = list(MX4_VALUES)
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    shape = x.shape
    x = x.reshape(-1, BLOCK)
    out = torch.empty_like(x)
    for r0 in range(0, x.shape[0], 1 << 20):
        b = x[r0:r0 + (1 << 20)]
        top = b.abs().amax(1)
        e = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -140) / TOP[fmt])) - 1
        for _ in range(3):                                            # the least power of two that holds the block
            e = torch.where(top > TOP[fmt] * torch.exp2(e), e + 1, e)
        scale = torch.exp2(e.clamp(-126, 127))[:, None]
        a = b.abs() / scale
        below, upto = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
        code = torch.where(below % 2 == 0, below, upto)               # they differ on a tie only: the even one
        out[r0:r0 + (1 << 20)] = torch.copysign(grid[code] * scale, b)
    return out.view(shape)


def _exact_plan(case, x):
    """The two steps of a pass, one sequence after the other."""
    page, (rows, back, width, _) = case["page"], _plan_sizes(case)
    table, lens, free = x["table"].cpu().numpy(), x["lens"].cpu().numpy().astype(np.int64), x["free"].cpu().numpy()
    n_free, width = int(x["n_free"][0]), table.shape[1]
    adds, out = x["adds"].cpu().numpy().astype(np.int64), []
    for asked, capacity in ((adds, rows), (-adds, back)):
        before, granted, given = lens.copy(), np.zeros_like(lens), []
        for b in np.flatnonzero((lens > 0) & (asked < 0)):
            granted[b] = -min(-asked[b], lens[b])
            first, last = -(-(lens[b] + granted[b]) // page), -(-lens[b] // page)
            given += table[b, first:last].tolist()
        free[n_free:n_free + len(given)] = given[::-1]
        n_free += len(given)
        starts, open_ = [0], True
        slots, positions = np.full(capacity, -1, np.int64), np.zeros(capacity, np.int32)
        for b in range(case["B"]):
            first, last = -(-max(lens[b], 0) // page), -(-(lens[b] + asked[b]) // page)
            if lens[b] >= 0 and asked[b] > 0 and last <= width:
                open_ = open_ and last - first <= n_free and starts[-1] + asked[b] <= capacity
                if open_:
                    granted[b] = asked[b]
                    table[b, first:last] = free[n_free - (last - first):n_free][::-1]
                    n_free -= last - first
                    at = np.arange(lens[b], lens[b] + asked[b])
                    slots[starts[-1]:starts[-1] + asked[b]] = table[b, at // page].astype(np.int64) * page + at % page
                    positions[starts[-1]:starts[-1] + asked[b]] = at
            starts.append(starts[-1] + max(int(granted[b]), 0))
        lens = before + granted
        out += [np.array(starts, np.int32), slots, positions, granted.astype(np.int32)]
    return (*out, table, lens.astype(np.int32), free, np.array([n_free], np.int32))


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, x)
    hq, hk, D = case["hq"], case["hk"], case["D"]
    G, scale = hq // hk, 1 / math.sqrt(D)
    if case["op"] == "prompt":
        out, at, k_at = torch.empty_like(x["q"], dtype=torch.float64), 0, 0
        for n, m in zip(*_pieces(case)):
            i = torch.arange(n, device="cuda")[:, None] + (m - n)
            hidden = torch.arange(m, device="cuda") > i
            for h in range(hq):
                k, v = (x[name][k_at:k_at + m, h // G].double() for name in ("k", "v"))
                s = x["q"][at:at + n, h].double() @ k.T * scale
                out[at:at + n, h] = torch.softmax(s.masked_fill_(hidden, -math.inf), -1) @ v
            at, k_at = at + n, k_at + m
        return out
    lens, masks = _drafts(case)
    k, v = _exact_cached(x["k"], case["fmt"]), _exact_cached(x["v"], case["fmt"])
    N, out, at = case["N"], torch.empty_like(x["q"], dtype=torch.float64), 0
    for b, n in enumerate(lens):
        seen = torch.ones((N, n), dtype=torch.bool)
        seen[:, n - N:] = torch.tensor([[bool(m >> j & 1) for j in range(N)] for m in masks[b]])
        seen = seen.cuda()
        for h in range(hq):
            s = x["q"][b, :, h].double() @ k[at:at + n, h // G].T * scale
            out[b, :, h] = torch.softmax(s.masked_fill_(~seen, -math.inf), -1) @ v[at:at + n, h // G]
        at += n
    return out
