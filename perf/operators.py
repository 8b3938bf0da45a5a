"""The paged-cache operators as measured work: planning a step's pages and
slots on the GPU, appending its keys and values to the cache, and attention
of its tokens over the cache.

``run`` computes an operator in plain torch operations (``own`` false) or
through the framework's entry points (``own`` true); ``exact`` is its
definition in 64 bits, written apart from the plain form.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _attention(name, requests, chunk, chunks, lo, hi, heads, kv_heads, dim, page, dtype, window=0):
    """`chunks` of the requests bring `chunk` new tokens, the others one;
    every request holds between lo and hi tokens before the step."""
    return {"op": "attention", "name": name, "requests": requests, "chunk": chunk, "chunks": chunks, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "window": window}


def _append(name, tokens, requests, heads, kv_heads, dim, page, source, dtype, rotary, interleaved=False):
    """`tokens` new tokens of `requests` requests; the first `rotary` values
    of every head are rotated."""
    return {"op": "append", "name": name, "tokens": tokens, "requests": requests, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "source": source, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved}


def _plan(name, requests, chunk, chunks, lo, hi, page):
    return {"op": "plan", "name": name, "requests": requests, "chunk": chunk, "chunks": chunks, "lo": lo, "hi": hi,
            "page": page}


def listed():
    return [
        # one conversation answering token by token, Llama-3-8B heads: latency of the smallest call
        _attention("decode 1 x 700", 1, 1, 1, 700, 700, 32, 8, 128, 16, "bf16"),
        # a full decode batch of the fused product (64 vectors) with ragged contexts: cache bandwidth
        _attention("decode 64 ragged to 8191", 64, 1, 64, 1, 8191, 32, 8, 128, 16, "bf16"),
        # one long document: the split over the keys and its join
        _attention("decode 1 x 131072", 1, 1, 1, 131071, 131071, 32, 8, 128, 64, "f16"),
        # a few drafted tokens checked at once for 16 requests
        _attention("draft 16 x 5 to 4097", 16, 5, 16, 511, 4097, 32, 8, 128, 16, "bf16"),
        # a prompt's first pass, the forward workload's 512 tokens
        _attention("prompt 512", 1, 512, 1, 0, 0, 32, 8, 128, 16, "bf16"),
        # a long prompt: matrix rate (the largest)
        _attention("prompt 8192", 1, 8192, 1, 0, 0, 32, 8, 128, 16, "bf16"),
        # a chunk of a long prompt over what was read so far
        _attention("chunk 513 over 32000", 1, 513, 1, 32000, 32000, 32, 8, 128, 32, "f16"),
        # a serving step: prompts' chunks beside decoding requests, heads of 64 without groups, sliding window
        _attention("mixed 14 + 2 x 333, window", 16, 333, 2, 17, 5000, 12, 12, 64, 16, "f16", window=1000),
        # the fused product's fp32 q, k and v of a decode batch, rotated and stored
        _append("append 64 from f32", 64, 64, 32, 8, 128, 16, "f32", "bf16", 128),
        # a prompt's
        _append("append 8192", 8192, 1, 32, 8, 128, 16, "bf16", "bf16", 128),
        # a decode step's pages and slots
        _plan("plan 64 x 1", 64, 1, 64, 0, 8191, 16),
        # a step with many prompts' chunks
        _plan("plan 300 with 97 x 333", 300, 333, 97, 0, 8191, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    while True:
        kind = rng.random()
        if kind < 0.6:
            kv_heads = rng.choice([1, 2, 4, 8, 8, 8, 12])
            heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 8])
            dim = rng.choice([64, 80, 128, 128, 128, 256])
            page = rng.choice([8, 16, 16, 32, 64, 128])
            dtype = rng.choice(["bf16", "f16"])
            window = rng.choice([0, 0, 0, 128, 1000])
            requests = _log(rng, 1, 64)
            hi = _log(rng, 16, 131071)
            lo = rng.choice([0, 1, hi // 2, hi])
            if rng.random() < 0.5:
                chunk = rng.choice([1, 1, 2, 5])
                chunks = requests
            else:
                chunk = _log(rng, 2, 8192)
                chunks = rng.randint(1, requests)
            case = _attention(None, requests, chunk, chunks, lo, hi, heads, kv_heads, dim, page, dtype, window)
            held, new = _lengths(case)
            longest = max(h + n for h, n in zip(held, new))
            # what the plain form holds: padded scores and padded keys
            if requests * heads * max(new) * longest > 32 * 8192 * 8192:
                continue
            if requests * longest * kv_heads * dim > 64 * 8192 * 8 * 128:
                continue
            if work(case)["flops"] > 2 ** 39 or heads > 64:
                continue
        elif kind < 0.8:
            kv_heads = rng.choice([1, 2, 8, 8, 12])
            dim = rng.choice([64, 80, 128, 128, 256])
            rotary = rng.choice([0, 32, dim // 16 * 16, dim // 16 * 16])
            tokens = _log(rng, 1, 8192)
            case = _append(None, tokens, rng.choice([1, tokens, min(tokens, 7)]), kv_heads * rng.choice([1, 3, 4]),
                           kv_heads, dim, rng.choice([8, 16, 64]), rng.choice(["bf16", "f16", "f32"]),
                           rng.choice(["bf16", "f16"]), rotary, rng.random() < 0.3)
            if work(case)["bytes"] > 256 << 20:
                continue
            if case["source"] != "f32":
                case["source"] = case["dtype"]
        else:
            requests = _log(rng, 1, 512)
            chunk = _log(rng, 1, 1024)
            case = _plan(None, requests, chunk, rng.randint(1, requests), 0, _log(rng, 16, 32768),
                         rng.choice([1, 8, 16, 64]))
            if case["chunk"] * case["chunks"] > 65536 or requests * (case["hi"] + chunk) // case["page"] > 1 << 21:
                continue
        del case["name"]
        return case


def _lengths(case):
    """Tokens held and new tokens of every request, from the case alone."""
    held, new = [], []
    for r in range(case["requests"]):
        u = math.modf((r + 1) * 0.6180339887498949)[0]
        held.append(case["lo"] + int(u * (case["hi"] - case["lo"] + 0.999)))
        # the requests that bring a chunk are spread among the others
        new.append(case["chunk"] if (r * case["chunks"]) % case["requests"] < case["chunks"] else 1)
    return held, new


def _pairs(held, n, window):
    """Unmasked (query, key) pairs of one request."""
    if window <= 0:
        return n * held + n * (n + 1) // 2
    short = max(0, min(n, window - held))  # tokens that still see everything
    return short * held + short * (short + 1) // 2 + (n - short) * window


def work(case):
    if case["op"] == "attention":
        held, new = _lengths(case)
        rows = sum(new)
        w = case["window"]
        keys = sum(h + n if w <= 0 else min(h + n, n + w - 1) for h, n in zip(held, new))
        pairs = sum(_pairs(h, n, w) for h, n in zip(held, new))
        return {"bytes": 2 * 2 * keys * case["kv_heads"] * case["dim"] + 2 * 2 * rows * case["heads"] * case["dim"]
                + 4 * rows * case["heads"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "append":
        n = case["tokens"] * case["dim"] * (case["heads"] + 2 * case["kv_heads"])
        turned = case["tokens"] * case["rotary"] * (case["heads"] + case["kv_heads"])
        return {"bytes": n * (_BYTES[case["source"]] + 2) + case["tokens"] * (12 + 4 * case["rotary"]),
                "flops": 3 * turned}
    held, new = _lengths(case)
    P = case["page"]
    pages = sum(-(-(h + n) // P) - -(-h // P) for h, n in zip(held, new))
    return {"bytes": case["requests"] * (8 + 8 + 4) + 8 * pages + 12 * sum(new), "flops": 10 * sum(new)}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}

    def normal(*shape, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(_TYPES[dtype])

    if case["op"] == "append":
        T, P = case["tokens"], case["page"]
        H, K, D, R = case["heads"], case["kv_heads"], case["dim"], case["rotary"]
        # every request has a run of tokens over scattered pages of its own
        run_len = -(-T // case["requests"])
        run_pages = -(-(run_len + P - 1) // P)
        pages = case["requests"] * run_pages + 1
        state["q"], state["k"], state["v"] = (normal(T, n, D, dtype=case["source"]) for n in (H, K, K))
        state["k_cache"], state["v_cache"] = (torch.zeros(pages, P, K, D, device="cuda", dtype=_TYPES[case["dtype"]])
                                              for _ in range(2))
        start = seed % 1000
        t = torch.arange(T, device="cuda")
        pos = start + t % run_len
        perm = torch.randperm(pages, generator=g, device="cuda")
        at = t // run_len * (run_pages * P) + seed % P + t % run_len
        state["slots"] = perm[at // P] * P + at % P
        state["positions"] = pos.to(torch.int32)
        state["table"] = None
        if R:
            freq = 500000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
            angle = torch.arange(start + run_len, device="cuda", dtype=torch.float64)[:, None] * freq
            state["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return state

    held, new = _lengths(case)
    P, n_req = case["page"], case["requests"]
    total = [h + n for h, n in zip(held, new)]
    state["tokens"] = sum(new)
    state["max_new"] = max(new)
    width = -(-max(total) // P)
    state["width"] = width
    if case["op"] == "plan":
        have = [-(-h // P) for h in held]
        used = sum(have)
        n_pages = used + sum(-(-t // P) for t in total) + 5
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        state["block_table"] = _table(perm[:used], have, width)
        # the free pages stand in a ring that has turned a few times
        free = perm[used:].contiguous()
        head = int(free.numel()) * 3 + seed % int(free.numel())
        state["free_pages"] = free
        state["cursor"] = torch.tensor([head, head + int(free.numel())], dtype=torch.int64, device="cuda")
        state["context_lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        state["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        return state

    need = [-(-t // P) for t in total]
    used = sum(need)
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    state["block_table"] = _table(perm[:used], need, width)
    state["max_len"] = max(total)
    state["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    state["cu_q"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    # the scores' spread grows with the queries' scale, as trained heads' does
    state["q"] = (normal(state["tokens"], case["heads"], case["dim"], dtype="f32") * 1.5).to(_TYPES[case["dtype"]])
    for name in ("k_cache", "v_cache"):
        state[name] = normal(n_pages, P, case["kv_heads"], case["dim"], dtype=case["dtype"])
    # what no token was stored to is memory as it was found
    for name in ("k_cache", "v_cache"):
        state[name][perm[used:].long()] = float("nan")
        last = torch.tensor([n - 1 for n in need], device="cuda")
        page = state["block_table"][torch.arange(n_req, device="cuda"), last].long()
        fill = torch.tensor([(t - 1) % P + 1 for t in total], device="cuda")
        tail = torch.arange(P, device="cuda")[None, :] >= fill[:, None]
        state[name][page] = state[name][page].masked_fill(tail[:, :, None, None], float("nan"))
    return state


def _table(pages, counts, width):
    """Rows of `width` entries holding `counts` pages each, the rest -1."""
    n = torch.tensor(counts, device=pages.device)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=pages.device)
    table[torch.arange(width, device=pages.device)[None, :] < n[:, None]] = pages
    return table


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "plan": _own_plan}[op](state)
    return {"attention": _plain_attention, "append": _plain_append, "plan": _plain_plan}[op](state)


def _own_attention(s):
    import lossless_entropy_coded_dfc_amd as dfc
    out, lse = dfc.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"], s["seq_lens"],
                                   causal=True, window=s["case"]["window"], max_q_len=s["max_new"], lse=True)
    return {"out": out, "lse": lse}


def _own_append(s):
    import lossless_entropy_coded_dfc_amd as dfc
    q = dfc.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"],
                         positions=s["positions"] if s["table"] is not None else None, rotary=s["table"],
                         interleaved=s["case"]["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_plan(s):
    import lossless_entropy_coded_dfc_amd as dfc
    p = dfc.paged_plan(s["context_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["cursor"],
                       page_size=s["case"]["page"], tokens=s["tokens"])
    return {"block_table": s["block_table"], "seq_lens": p.seq_lens, "cu_q": p.cu_q, "slots": p.slots,
            "positions": p.positions, "cursor": p.cursor}


def _plain_attention(s):
    c = s["case"]
    q, table, cu, lens = s["q"], s["block_table"].long(), s["cu_q"].long(), s["seq_lens"].long()
    P, H, K, D, R = c["page"], c["heads"], c["kv_heads"], c["dim"], c["requests"]
    G, M, N = H // K, s["max_new"], s["max_len"]
    new = cu[1:] - cu[:-1]
    key = torch.arange(N, device=q.device)
    there = key[None, :] < lens[:, None]
    slot = torch.where(there, table[:, key // P] * P + key % P, 0)
    empty = ~there[:, :, None, None]
    k = s["k_cache"].view(-1, K, D)[slot].float().masked_fill_(empty, 0.0).permute(0, 2, 3, 1).contiguous()
    v = s["v_cache"].view(-1, K, D)[slot].float().masked_fill_(empty, 0.0).permute(0, 2, 1, 3).contiguous()
    i = torch.arange(M, device=q.device)
    token = torch.clamp(cu[:-1, None] + i, max=q.shape[0] - 1)
    rows = q[token].float().view(R, M, K, G, D).permute(0, 2, 1, 3, 4).reshape(R, K, M * G, D)
    score = torch.matmul(rows, k).mul_(1.0 / math.sqrt(D)).view(R, K, M, G, N)
    at = (lens - new)[:, None] + i
    seen = (key[None, None, :] <= at[:, :, None]) & there[:, None, :]
    if c["window"] > 0:
        seen &= key[None, None, :] > at[:, :, None] - c["window"]
    score.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_(min=-3.0e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, K, M * G, N), v).view(R, K, M, G, D) / total
    lse = (top + total.log()).squeeze(-1)
    t = torch.arange(q.shape[0], device=q.device)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    j = t - cu[r]
    return {"out": o[r, :, j].reshape(-1, H, D).to(q.dtype), "lse": lse[r, :, j].reshape(-1, H)}


def _turn(x, cos, sin, interleaved):
    n = 2 * cos.shape[-1]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., : n // 2], x[..., n // 2: n])
    first, second = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([first, second], -1).flatten(-2) if interleaved else torch.cat([first, second], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_append(s):
    c = s["case"]
    q, k = s["q"].float(), s["k"].float()
    if s["table"] is not None:
        cos, sin = s["table"][s["positions"].long()][:, None, :].chunk(2, -1)
        q, k = _turn(q, cos, sin, c["interleaved"]), _turn(k, cos, sin, c["interleaved"])
    kind = s["k_cache"].dtype
    s["k_cache"].view(-1, *k.shape[1:])[s["slots"]] = k.to(kind)
    s["v_cache"].view(-1, *k.shape[1:])[s["slots"]] = s["v"].to(kind)
    return {"q": q.to(kind), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_plan(s):
    P, T = s["case"]["page"], s["tokens"]
    held, new, table = s["context_lens"].long(), s["new_lens"].long(), s["block_table"]
    head, tail = s["cursor"][0], s["cursor"][1]
    have, need = (held + P - 1) // P, (held + new + P - 1) // P
    more = need - have
    before = more.cumsum(0) - more
    column = torch.arange(table.shape[1], device=table.device)[None, :]
    rank = before[:, None] + column - have[:, None]
    page = s["free_pages"][(head + rank) % s["free_pages"].numel()]
    page = torch.where(rank < tail - head, page, -1)
    table.copy_(torch.where((column >= have[:, None]) & (column < need[:, None]), page, table))
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(T, device=table.device)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = held[r] + t - cu[r]
    at = table[r, pos // P].long()
    return {"block_table": table, "seq_lens": (held + new).int(), "cu_q": cu.int(),
            "slots": torch.where(at >= 0, at * P + pos % P, -1), "positions": pos.int(),
            "cursor": torch.stack([head + torch.minimum(more.sum(), tail - head), tail])}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "append":
        n, R = case["tokens"], case["rotary"]

        def turned(x):
            x = x.double().clone()
            if R:
                half = R // 2
                for j in range(half):
                    i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
                    co = s["table"][s["positions"].long(), j].double()[:, None]
                    si = s["table"][s["positions"].long(), half + j].double()[:, None]
                    x0, x1 = x[:, :, i0].clone(), x[:, :, i1].clone()
                    x[:, :, i0] = x0 * co - x1 * si
                    x[:, :, i1] = x1 * co + x0 * si
            return x

        caches = []
        for name, x in (("k_cache", turned(s["k"])), ("v_cache", s["v"].double())):
            full = s[name].double()
            page, place = s["slots"] // case["page"], s["slots"] % case["page"]
            full[page, place] = x
            caches.append(full)
        assert n == s["slots"].numel()
        return {"q": turned(s["q"]), "k_cache": caches[0], "v_cache": caches[1]}

    held, new = _lengths(case)
    G, P, D, w = case["heads"] // case["kv_heads"], case["page"], case["dim"], case["window"]
    out = torch.zeros(s["tokens"], case["heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], case["heads"], dtype=torch.float64, device="cuda")
    base = 0
    for r in range(case["requests"]):
        n, total = new[r], held[r] + new[r]
        pages = s["block_table"][r, : -(-total // P)].long()
        for h in range(case["kv_heads"]):
            k = s["k_cache"][pages, :, h].reshape(-1, D)[:total].double()
            v = s["v_cache"][pages, :, h].reshape(-1, D)[:total].double()
            step = max(1, (1 << 26) // (G * total))
            for t0 in range(0, n, step):
                t1 = min(n, t0 + step)
                first = held[r] + t0 - w + 1 if w > 0 else 0
                first = max(0, first)
                last = held[r] + t1
                x = s["q"][base + t0: base + t1, h * G: (h + 1) * G].double()
                z = (x.reshape(-1, D) @ k[first:last].t()).view(t1 - t0, G, last - first) / math.sqrt(D)
                key = torch.arange(first, last, device="cuda")
                at = torch.arange(held[r] + t0, last, device="cuda")[:, None]
                hidden = key[None, :] > at
                if w > 0:
                    hidden |= key[None, :] <= at - w
                z = z.masked_fill(hidden[:, None, :], float("-inf"))
                norm = torch.logsumexp(z, -1)
                y = torch.exp(z - norm[..., None]).view(-1, last - first) @ v[first:last]
                out[base + t0: base + t1, h * G: (h + 1) * G] = y.view(t1 - t0, G, D)
                lse[base + t0: base + t1, h * G: (h + 1) * G] = norm
        base += n
    return {"out": out, "lse": lse}
