"""More operators of the serving loop as measured work: the append with norms
of queries and keys, attention with a window and first tokens that stay
visible, the verification of drafted tokens, and the cache's pages given back,
forked and compacted.

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

def _append(name, tokens, requests, heads, kv_heads, dim, page, source, dtype, rotary, interleaved=False, norms="qk"):
    """`tokens` new tokens of `requests` requests; heads of q and k are
    normed (those that `norms` names), then their first `rotary` values
    rotated."""
    return {"op": "append", "name": name, "tokens": tokens, "requests": requests, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "source": source, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved, "norms": norms}


def _attention(name, requests, chunk, chunks, lo, hi, heads, kv_heads, dim, page, dtype, window, sinks):
    """`chunks` of the requests bring `chunk` new tokens, the others one;
    every request holds between lo and hi tokens before the step, and has
    given back the pages that lie wholly between its sinks and its window."""
    return {"op": "attention", "name": name, "requests": requests, "chunk": chunk, "chunks": chunks, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "window": window, "sinks": sinks}


def _verify(name, requests, drafts, ragged, vocab, dtype, drafter):
    """Up to `drafts` drafted tokens a request (from none to all of them
    where `ragged`), with the drafter's logits or without."""
    return {"op": "verify", "name": name, "requests": requests, "drafts": drafts, "ragged": ragged, "vocab": vocab,
            "dtype": dtype, "drafter": drafter}


def _release(name, requests, lo, hi, page, cut, finished, window, sinks, family):
    """Requests that hold lo to hi tokens; `finished` of them give back all,
    the others up to `cut` tokens and what a window has passed since 24 tokens
    ago; `family` neighbours share the first half of their pages."""
    return {"op": "release", "name": name, "requests": requests, "lo": lo, "hi": hi, "page": page, "cut": cut,
            "finished": finished, "window": window, "sinks": sinks, "family": family}


def _fork(name, parents, children, lo, hi, page, layers, kv_heads, dim, dtype):
    """`children` empty requests become copies of `parents` others."""
    return {"op": "fork", "name": name, "parents": parents, "children": children, "lo": lo, "hi": hi, "page": page,
            "layers": layers, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def _compact(name, requests, lo, hi, page, free, layers, kv_heads, dim, dtype):
    """Requests' pages scattered among `free` free ones."""
    return {"op": "compact", "name": name, "requests": requests, "lo": lo, "hi": hi, "page": page, "free": free,
            "layers": layers, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def listed():
    return [
        # a decode batch's fp32 q, k and v from the fused product, Llama-3-8B heads with norms
        _append("append 64 from f32, normed", 64, 64, 32, 8, 128, 16, "f32", "bf16", 128),
        # a prompt's
        _append("append 8192, normed", 8192, 1, 32, 8, 128, 16, "bf16", "bf16", 128),
        # a full decode batch of long conversations that keep a window and their first tokens
        _attention("decode 64 to 8191, window 1000 + 4", 64, 1, 64, 1, 8191, 32, 8, 128, 16, "bf16", 1000, 4),
        # a chunk of a long document under a window
        _attention("chunk 513 over 32000, window 4096 + 64", 1, 513, 1, 32000, 32000, 32, 8, 128, 32, "f16", 4096, 64),
        # one conversation's next token sampled: latency of the smallest call
        _verify("sample 1 of 128256", 1, 0, False, 128256, "f32", False),
        # a batch of requests with five drafts each, checked against the drafter's logits (the largest)
        _verify("verify 64 x 5 of 128256", 64, 5, False, 128256, "f32", True),
        # what a step with rejected drafts gives back
        _release("release 64 after drafts", 64, 1, 8191, 16, 5, 0, 0, 0, 1),
        # requests that end beside others whose window moves on, prefixes shared by four
        _release("release 300, 97 finished, window", 300, 0, 32768, 16, 0, 97, 1000, 4, 4),
        # one prompt answered eight ways
        _fork("fork 1 into 7 over 8191", 1, 7, 8191, 8191, 16, 8, 8, 128, "bf16"),
        # a batch's prompts, each answered several ways
        _fork("fork 16 into 112", 16, 112, 17, 2000, 16, 8, 8, 128, "bf16"),
        # a small cache made dense
        _compact("compact 64 requests", 64, 1, 500, 16, 512, 2, 8, 128, "bf16"),
        # a large one of which half is free
        _compact("compact 300 requests", 300, 0, 900, 16, 8192, 4, 8, 128, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    while True:
        kind = rng.random()
        dtype = rng.choice(["bf16", "f16"])
        page = rng.choice([1, 8, 16, 16, 32, 64, 128])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 12])
        dim = rng.choice([64, 80, 128, 128, 256])
        if kind < 0.2:
            rotary = rng.choice([0, 32, dim // 16 * 16, dim // 16 * 16])
            tokens = _log(rng, 1, 8192)
            source = rng.choice(["f32", dtype])
            case = _append(None, tokens, rng.choice([1, tokens, min(tokens, 7)]), kv_heads * rng.choice([1, 3, 4]),
                           kv_heads, dim, page, source, dtype, rotary, rng.random() < 0.3,
                           rng.choice(["qk", "qk", "k", "q"]))
            if work(case)["bytes"] > 256 << 20:
                continue
        elif kind < 0.45:
            heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 8])
            requests = _log(rng, 1, 64)
            hi = _log(rng, 16, 65536)
            lo = rng.choice([0, 1, hi // 2, hi])
            if rng.random() < 0.5:
                chunk, chunks = rng.choice([1, 1, 2, 5]), requests
            else:
                chunk, chunks = _log(rng, 2, 4096), rng.randint(1, requests)
            case = _attention(None, requests, chunk, chunks, lo, hi, heads, kv_heads, dim, page, dtype,
                              _log(rng, 1, 8192), rng.choice([1, 4, 4, 16, 63, 64, 200]))
            held, new = _lengths(case)
            longest = max(h + n for h, n in zip(held, new))
            # what the plain form holds: padded scores and padded keys
            if requests * heads * max(new) * longest > 32 * 8192 * 4096:
                continue
            if requests * longest * kv_heads * dim > 64 * 8192 * 8 * 128:
                continue
            if requests * longest > page << 17 or work(case)["flops"] > 2 ** 38 or heads > 64:
                continue
        elif kind < 0.65:
            requests, vocab = _log(rng, 1, 64), _log(rng, 200, 131072)
            case = _verify(None, requests, rng.choice([0, 1, 3, 5, 7]), rng.random() < 0.5, vocab,
                           rng.choice(["f32", "f32", "bf16", "f16"]), rng.random() < 0.6)
            if work(case)["bytes"] > 384 << 20:
                continue
        elif kind < 0.8:
            requests = _log(rng, 1, 512)
            window = rng.choice([0, 0, 100, 1000])
            case = _release(None, requests, 0, _log(rng, 16, 32768), page, rng.choice([0, 1, 5]),
                            rng.randint(0, requests), window, rng.choice([0, 4, 64]) if window else 0,
                            rng.choice([1, 1, 4]))
            if requests * case["hi"] // page > 1 << 20:
                continue
        elif kind < 0.9:
            parents = _log(rng, 1, 64)
            case = _fork(None, parents, _log(rng, 1, 256), 1, _log(rng, 16, 8192), page, rng.choice([1, 2, 5]),
                         kv_heads, dim, dtype)
            if (parents * case["hi"] + case["children"] * page) * kv_heads * dim * case["layers"] > 1 << 28:
                continue
        else:
            requests = _log(rng, 1, 300)
            case = _compact(None, requests, 0, _log(rng, 16, 8192), page, _log(rng, 1, 4096), rng.choice([1, 2, 3]),
                            kv_heads, dim, dtype)
            if (requests * case["hi"] + case["free"] * page) * kv_heads * dim * case["layers"] > 1 << 28:
                continue
        del case["name"]
        return case


def _spread(n, lo, hi):
    """n whole numbers from lo to hi."""
    return [lo + int(math.modf((r + 1) * 0.6180339887498949)[0] * (hi - lo + 0.999)) for r in range(n)]


def _lengths(case):
    """Tokens held and new tokens of every request of a step."""
    held = _spread(case["requests"], case["lo"], case["hi"])
    new = [case["chunk"] if (r * case["chunks"]) % case["requests"] < case["chunks"] else 1
           for r in range(case["requests"])]
    return held, new


def _drafts(case):
    """Drafted tokens of every request."""
    if not case["ragged"]:
        return [case["drafts"]] * case["requests"]
    return _spread(case["requests"], 0, case["drafts"])


def _kept(case):
    """Tokens that every request holds and keeps."""
    n = case["requests"]
    held = _spread(n, case["lo"], case["hi"])
    cut = _spread(n, 0, case["cut"]) if case["cut"] else [0] * n
    return held, [0 if (r * case["finished"]) % n < case["finished"] else max(0, h - c)
                  for r, (h, c) in enumerate(zip(held, cut))]


def _hole(keep, page, window, sinks):
    """The pages [first, end) that no token from `keep` on sees again."""
    if window <= 0:
        return 0, 0
    first = -(-sinks // page)
    return first, max(first, max(0, keep - window + 1) // page)


def work(case):
    op = case["op"]
    if op == "append":
        n = case["tokens"] * case["dim"] * (case["heads"] + 2 * case["kv_heads"])
        turned = case["tokens"] * case["rotary"] * (case["heads"] + case["kv_heads"])
        normed = case["tokens"] * case["dim"] * (case["heads"] * ("q" in case["norms"]) +
                                                 case["kv_heads"] * ("k" in case["norms"]))
        return {"bytes": n * (_BYTES[case["source"]] + 2) + case["tokens"] * (12 + 4 * case["rotary"]),
                "flops": 3 * turned + 4 * normed}
    if op == "attention":
        held, new = _lengths(case)
        w, s = case["window"], case["sinks"]
        keys = pairs = 0
        for h, n in zip(held, new):
            begin = max(0, h + 1 - w)
            keys += h + n - begin + min(s, begin)
            p = np.arange(h + 1, h + n + 1, dtype=np.int64)
            pairs += int((np.minimum(p, w) + np.minimum(s, np.maximum(p - w, 0))).sum())
        rows = sum(new)
        return {"bytes": 2 * 2 * keys * case["kv_heads"] * case["dim"] + 2 * 2 * rows * case["heads"] * case["dim"]
                + 4 * rows * case["heads"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if op == "verify":
        drafts = sum(_drafts(case))
        rows = drafts + case["requests"]
        values = (rows + (drafts if case["drafter"] else 0)) * case["vocab"]
        return {"bytes": values * _BYTES[case["dtype"]] + 16 * rows + 16 * case["requests"], "flops": 4 * values}
    P = case["page"]
    if op == "release":
        held, keep = _kept(case)
        entries = 0
        for h, k in zip(held, keep):
            first, end = _hole(k, P, case["window"], case["sinks"])
            entries += -(-h // P) - -(-k // P) + end - first
        # a table entry read and written, a holder's count and a place in the ring
        return {"bytes": 8 * case["requests"] + 16 * entries, "flops": entries}
    one = 2 * 2 * P * case["kv_heads"] * case["dim"] * case["layers"]  # a page of K and V in every layer
    if op == "fork":
        held = _spread(case["parents"], case["lo"], case["hi"])
        child = [held[i % case["parents"]] for i in range(case["children"])]
        copies = sum(h % P != 0 for h in child)
        shared = sum(h // P for h in child)
        return {"bytes": 2 * copies * one + 16 * shared, "flops": shared}
    held = _spread(case["requests"], case["lo"], case["hi"])
    used = sum(-(-h // P) for h in held)
    # of the used pages, as many lie beyond the first `used` as there are free ones before
    moves = used * case["free"] // max(1, used + case["free"])
    return {"bytes": 2 * moves * one + 8 * used + 8 * case["free"], "flops": used + case["free"]}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case, "g": g, "seed": seed}
    {"append": _append_inputs, "attention": _attention_inputs, "verify": _verify_inputs, "release": _release_inputs,
     "fork": _fork_inputs, "compact": _compact_inputs}[case["op"]](state)
    del state["g"]
    return state


def _normal(s, *shape, dtype):
    return torch.randn(shape, generator=s["g"], device="cuda", dtype=torch.float32).to(_TYPES[dtype])


def _append_inputs(s):
    case, seed = s["case"], s["seed"]
    T, P = case["tokens"], case["page"]
    H, K, D, R = case["heads"], case["kv_heads"], case["dim"], case["rotary"]
    # every request has a run of tokens over scattered pages of its own
    run_len = -(-T // case["requests"])
    run_pages = -(-(run_len + P - 1) // P)
    pages = case["requests"] * run_pages + 1
    s["q"], s["k"], s["v"] = (_normal(s, T, n, D, dtype=case["source"]) for n in (H, K, K))
    # a few channels of a trained projection stand out before the norm
    for x in (s["q"], s["k"]):
        x[..., :: 37] *= 8
    s["q_norm"], s["k_norm"] = (1 + 0.2 * _normal(s, D, dtype="f32") if n in case["norms"] else None for n in "qk")
    s["k_cache"], s["v_cache"] = (torch.zeros(pages, P, K, D, device="cuda", dtype=_TYPES[case["dtype"]])
                                  for _ in range(2))
    start = seed % 1000
    t = torch.arange(T, device="cuda")
    perm = torch.randperm(pages, generator=s["g"], device="cuda")
    at = t // run_len * (run_pages * P) + seed % P + t % run_len
    s["slots"] = perm[at // P] * P + at % P
    s["positions"] = (start + t % run_len).to(torch.int32)
    s["table"] = None
    if R:
        freq = 500000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        angle = torch.arange(start + run_len, device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()


def _table(pages, counts, width):
    """Rows of `width` entries holding `counts` pages each, the rest -1."""
    n = torch.tensor(counts, device=pages.device)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=pages.device)
    table[torch.arange(width, device=pages.device)[None, :] < n[:, None]] = pages.to(torch.int32)
    return table


def _attention_inputs(s):
    case = s["case"]
    held, new = _lengths(case)
    P, n_req = case["page"], case["requests"]
    total = [h + n for h, n in zip(held, new)]
    need = [-(-t // P) for t in total]
    used = sum(need)
    n_pages = used + 3
    s["tokens"], s["max_new"], s["max_len"] = sum(new), max(new), max(total)
    perm = torch.randperm(n_pages, generator=s["g"], device="cuda")
    s["block_table"] = _table(perm[:used], need, max(need))
    s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    # the scores' spread grows with the queries' scale, as trained heads' does
    s["q"] = (_normal(s, s["tokens"], case["heads"], case["dim"], dtype="f32") * 1.5).to(_TYPES[case["dtype"]])
    for name in ("k_cache", "v_cache"):
        s[name] = _normal(s, n_pages, P, case["kv_heads"], case["dim"], dtype=case["dtype"])
    # pages wholly between the sinks and the window are others' by now, and
    # what no token was stored to is memory as it was found
    column = torch.arange(max(need), device="cuda")[None, :]
    hole = [_hole(h, P, case["window"], case["sinks"]) for h in held]
    first, end = (torch.tensor(x, device="cuda")[:, None] for x in zip(*hole))
    gone = (column >= first) & (column < end)
    for name in ("k_cache", "v_cache"):
        s[name][s["block_table"][gone].long()] = float("nan")
        s[name][perm[used:]] = float("nan")
        last = torch.tensor([n - 1 for n in need], device="cuda")
        page = s["block_table"][torch.arange(n_req, device="cuda"), last].long()
        fill = torch.tensor([(t - 1) % P + 1 for t in total], device="cuda")
        tail = torch.arange(P, device="cuda")[None, :] >= fill[:, None]
        s[name][page] = s[name][page].masked_fill(tail[:, :, None, None], float("nan"))
    s["block_table"][gone] = -1


def _verify_inputs(s):
    case = s["case"]
    drafts = _drafts(case)
    rows, V = sum(drafts) + case["requests"], case["vocab"]
    # a language model's logits: a few tokens carry most of the weight
    z = _normal(s, rows, V, dtype="f32") * 2.0
    favoured = torch.randint(0, V, (rows, 8), generator=s["g"], device="cuda")
    z.scatter_add_(1, favoured, 6 + 4 * _normal(s, rows, 8, dtype="f32"))
    s["logits"] = z.to(_TYPES[case["dtype"]])
    # a drafter that has learned much of it
    d = (z + _normal(s, rows, V, dtype="f32")).to(_TYPES[case["dtype"]])
    s["draft_logits"] = d if case["drafter"] else None
    s["cu_rows"] = torch.tensor([0] + list(np.cumsum([n + 1 for n in drafts])), dtype=torch.int32, device="cuda")
    # some requests are answered greedily
    t = torch.tensor([0.0 if r % 5 == 3 else 0.6 + 0.1 * (r % 7) for r in range(case["requests"])], device="cuda")
    s["temperature"] = t
    row_t = t.repeat_interleave(torch.tensor([n + 1 for n in drafts], device="cuda"))[:, None]
    noise = -torch.log(-torch.log(torch.rand(rows, V, generator=s["g"], device="cuda").clamp_(1e-30, 1 - 1e-7)))
    s["drafts"] = (d.float() + row_t * noise).argmax(1)
    s["uniforms"] = torch.rand(rows, generator=s["g"], device="cuda")


def _pool(s, table, n_pages, extra=0):
    """A pool's state in one buffer (tables, holders, ring) and as it was."""
    R, W = table.shape
    s["n_pages"], s["shape"] = n_pages, (R, W)
    held = table[table >= 0].long()
    holders = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    holders.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    free = torch.nonzero(holders == 0).flatten()
    free = free[torch.randperm(free.numel(), generator=s["g"], device="cuda")]
    n_ring = n_pages
    head = n_ring * 3 + s["seed"] % n_ring
    ring = torch.zeros(n_ring, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free.numel(), device="cuda")) % n_ring] = free.int()
    s["pool0"] = torch.cat([table.flatten(), (holders - 1).clamp_(min=0), ring])
    s["pool"] = s["pool0"].clone()
    s["block_table"] = s["pool"][:R * W].view(R, W)
    s["shared"] = s["pool"][R * W: R * W + n_pages]
    s["ring"] = s["pool"][R * W + n_pages:]
    s["cursor"] = torch.tensor([head, head + free.numel()], dtype=torch.int64, device="cuda")


def _release_inputs(s):
    case = s["case"]
    P, n, w = case["page"], case["requests"], case["window"]
    held, keep = _kept(case)
    need = [-(-h // P) for h in held]
    width = max(need + [1])
    n_pages = sum(need) + 7
    perm = torch.randperm(n_pages, generator=s["g"], device="cuda")
    table = _table(perm[:sum(need)], need, width)
    # neighbours share the first half of what the shorter of them and the first have filled
    for i in range(1, case["family"]):
        for r in range(i, n, case["family"]):
            m = min(held[r], held[r - i]) // P // 2
            table[r, :m] = table[r - i, :m]
    # the window has been here before
    column = torch.arange(width, device="cuda")[None, :]
    first, end = (torch.tensor(x, device="cuda")[:, None] for x in
                  zip(*(_hole(max(0, h - 24), P, w, case["sinks"]) for h in held)))
    table[(column >= first) & (column < end)] = -1
    _pool(s, table, n_pages)
    s["held_lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    s["keep_lens"] = torch.tensor(keep, dtype=torch.int32, device="cuda")


def _cache(s):
    case = s["case"]
    s["cache"] = _normal(s, case["layers"], 2, s["n_pages"], case["page"], case["kv_heads"], case["dim"],
                         dtype=case["dtype"])


def _fork_inputs(s):
    case = s["case"]
    P, n, c = case["page"], case["parents"], case["children"]
    held = _spread(n, case["lo"], case["hi"])
    need = [-(-h // P) for h in held]
    n_pages = sum(need) + c + 5
    perm = torch.randperm(n_pages, generator=s["g"], device="cuda")
    _pool(s, _table(perm[:sum(need)], need + [0] * c, max(need + [1])), n_pages)
    s["context_lens"] = torch.tensor(held + [0] * c, dtype=torch.int32, device="cuda")
    s["parents"] = torch.tensor([-1] * n + [i % n for i in range(c)], dtype=torch.int32, device="cuda")
    _cache(s)


def _compact_inputs(s):
    case = s["case"]
    P = case["page"]
    held = _spread(case["requests"], case["lo"], case["hi"])
    need = [-(-h // P) for h in held]
    n_pages = sum(need) + case["free"]
    perm = torch.randperm(n_pages, generator=s["g"], device="cuda")
    _pool(s, _table(perm[:sum(need)], need, max(need + [1])), n_pages)
    s["context_lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    _cache(s)


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if "pool" in state:
        # the pool is changed in place: every pass begins with it as it was
        state["pool"].copy_(state["pool0"])
    return (_OWN if own else _PLAIN)[op](state)


def _own_append(s):
    import lossless_entropy_coded_dfc_amd as dfc
    q = dfc.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"],
                         positions=s["positions"] if s["table"] is not None else None, rotary=s["table"],
                         interleaved=s["case"]["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import lossless_entropy_coded_dfc_amd as dfc
    out, lse = dfc.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"], s["seq_lens"],
                                   causal=True, window=s["case"]["window"], sinks=s["case"]["sinks"],
                                   max_q_len=s["max_new"], lse=True)
    return {"out": out, "lse": lse}


def _own_verify(s):
    import lossless_entropy_coded_dfc_amd as dfc
    v = dfc.verify_drafts(s["logits"], s["cu_rows"], s["drafts"], s["uniforms"], draft_logits=s["draft_logits"],
                          temperature=s["temperature"])
    return {"accepted": v.accepted, "tokens": v.tokens}


def _own_release(s):
    import lossless_entropy_coded_dfc_amd as dfc
    case = s["case"]
    cursor = dfc.paged_release(s["held_lens"], s["keep_lens"], s["block_table"], s["ring"], s["cursor"], s["shared"],
                               page_size=case["page"], window=case["window"], sinks=case["sinks"])
    return {"block_table": s["block_table"], "shared": s["shared"], "ring": s["ring"], "cursor": cursor}


def _own_fork(s):
    import lossless_entropy_coded_dfc_amd as dfc
    f = dfc.paged_fork(s["context_lens"], s["parents"], s["block_table"], s["ring"], s["cursor"], s["shared"],
                       page_size=s["case"]["page"])
    dfc.paged_copy([(c[0], c[1]) for c in s["cache"]], f.src, f.dst)
    return {"context_lens": f.context_lens, "block_table": s["block_table"], "shared": s["shared"],
            "cursor": f.cursor, "src": f.src, "dst": f.dst, "cache": s["cache"]}


def _own_compact(s):
    import lossless_entropy_coded_dfc_amd as dfc
    m = dfc.paged_compact(s["context_lens"], s["block_table"], s["ring"], s["cursor"], s["shared"],
                          page_size=s["case"]["page"])
    dfc.paged_copy([(c[0], c[1]) for c in s["cache"]], m.src, m.dst)
    return {"block_table": s["block_table"], "shared": s["shared"], "ring": s["ring"], "src": m.src, "dst": m.dst,
            "cache": s["cache"]}


def _turn(x, cos, sin, interleaved):
    n = 2 * cos.shape[-1]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., : n // 2], x[..., n // 2: n])
    first, second = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([first, second], -1).flatten(-2) if interleaved else torch.cat([first, second], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_append(s):
    q, k = s["q"].float(), s["k"].float()
    if s["q_norm"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["q_norm"]
    if s["k_norm"] is not None:
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["k_norm"]
    if s["table"] is not None:
        cos, sin = s["table"][s["positions"].long()][:, None, :].chunk(2, -1)
        q, k = (_turn(x, cos, sin, s["case"]["interleaved"]) for x in (q, k))
    kind = s["k_cache"].dtype
    s["k_cache"].view(-1, *k.shape[1:])[s["slots"]] = k.to(kind)
    s["v_cache"].view(-1, *k.shape[1:])[s["slots"]] = s["v"].to(kind)
    return {"q": q.to(kind), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    q, table, cu, lens = s["q"], s["block_table"].long(), s["cu_q"].long(), s["seq_lens"].long()
    P, H, K, D, R = c["page"], c["heads"], c["kv_heads"], c["dim"], c["requests"]
    G, M, N = H // K, s["max_new"], s["max_len"]
    new = cu[1:] - cu[:-1]
    key = torch.arange(N, device=q.device)
    page = table[:, key // P]
    i = torch.arange(M, device=q.device)
    at = (lens - new)[:, None] + i
    # what any row of a request sees; the rest may be no page at all
    there = (key[None, :] < lens[:, None]) & (page >= 0)
    there &= (key[None, :] > (lens - new - c["window"])[:, None]) | (key < c["sinks"])
    slot = torch.where(there, page * P + key % P, 0)
    empty = ~there[:, :, None, None]
    k = s["k_cache"].view(-1, K, D)[slot].float().masked_fill_(empty, 0.0).permute(0, 2, 3, 1).contiguous()
    v = s["v_cache"].view(-1, K, D)[slot].float().masked_fill_(empty, 0.0).permute(0, 2, 1, 3).contiguous()
    token = torch.clamp(cu[:-1, None] + i, max=q.shape[0] - 1)
    rows = q[token].float().view(R, M, K, G, D).permute(0, 2, 1, 3, 4).reshape(R, K, M * G, D)
    score = torch.matmul(rows, k).mul_(1.0 / math.sqrt(D)).view(R, K, M, G, N)
    seen = (key[None, None, :] <= at[:, :, None]) & there[:, None, :]
    seen &= (key[None, None, :] > at[:, :, None] - c["window"]) | (key < c["sinks"])
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


def _weights(z, t):
    """Rows' probabilities in 64 bits; t = 0: one at the first of the largest."""
    z = z.double()
    top = z.amax(-1, keepdim=True)
    index = torch.arange(z.shape[1], device=z.device)
    first = torch.where(z == top, index, z.shape[1]).amin(-1, keepdim=True)
    e = torch.exp((z - top) / torch.where(t > 0, t, 1.0))
    return torch.where(t > 0, e / e.sum(-1, keepdim=True), (index == first).double())


def _plain_verify(s):
    cu, x, u = s["cu_rows"].long(), s["drafts"], s["uniforms"].double()
    rows, V = s["logits"].shape
    row = torch.arange(rows, device=x.device)
    r = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    t = s["temperature"].double()[r][:, None]
    p = _weights(s["logits"], t)
    index = torch.arange(V, device=x.device)
    drafted = (index == x[:, None]).double()
    q = drafted if s["draft_logits"] is None else torch.where(t > 0, _weights(s["draft_logits"], t), drafted)
    px, qx = p.gather(1, x[:, None])[:, 0], q.gather(1, x[:, None])[:, 0]
    last = cu[1:] - 1
    holds = (u * qx < px) & (row != last[r])
    # the first row of each request whose draft does not hold, its last row among them
    stop = torch.where(holds, rows, row)
    stop = torch.full_like(last, rows).scatter_reduce(0, r, stop, "amin")
    w = torch.where((stop != last)[:, None], (p[stop] - q[stop]).clamp_(min=0), p[stop])
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p[stop])
    sums = w.cumsum(-1)
    token = torch.searchsorted(sums, u[last][:, None] * sums[:, -1:], right=True)[:, 0]
    return {"accepted": (stop - cu[:-1]).int(), "tokens": token}


def _plain_release(s):
    c = s["case"]
    P, w, n_pages, n_ring = c["page"], c["window"], s["n_pages"], s["ring"].numel()
    table, shared, ring = s["block_table"], s["shared"], s["ring"]
    held, keep = s["held_lens"].long()[:, None], s["keep_lens"].long()[:, None]
    column = torch.arange(table.shape[1], device=table.device)[None, :]
    given = (column >= (keep + P - 1) // P) & (column < (held + P - 1) // P)
    if w > 0:
        given |= (column >= -(-c["sinks"] // P)) & (column < (keep - w + 1).clamp(min=0) // P)
    given &= table >= 0
    holders = shared.long() + 1
    # (entries that stay add nothing, each column in a place of its own)
    times = torch.zeros(n_pages + table.shape[1], dtype=torch.int64, device=table.device)
    times.scatter_add_(0, torch.where(given, table, n_pages + column).flatten(), given.long().flatten())
    left = holders - times[:n_pages]
    freed = left == 0
    shared.copy_((left - 1).clamp(min=0))
    head, tail = s["cursor"][0], s["cursor"][1]
    place = torch.where(freed, (tail + freed.cumsum(0) - 1) % n_ring, n_ring)
    wide = torch.cat([ring, ring[:1]])
    wide[place] = torch.arange(n_pages, dtype=torch.int32, device=table.device)
    ring.copy_(wide[:n_ring])
    table.masked_fill_(given, -1)
    return {"block_table": table, "shared": shared, "ring": ring, "cursor": torch.stack([head, tail + freed.sum()])}


def _copy(cache, src, dst):
    there = src >= 0
    cache[:, :, dst[there].long()] = cache[:, :, src[there].long()]


def _plain_fork(s):
    P, n_pages = s["case"]["page"], s["n_pages"]
    table, shared, ring = s["block_table"], s["shared"], s["ring"]
    parent = s["parents"].long()
    child = parent >= 0
    held = s["context_lens"].long()
    lens = torch.where(child, held[parent.clamp(min=0)], held)
    column = torch.arange(table.shape[1], device=table.device)[None, :]
    theirs = table[parent.clamp(min=0)]
    full = child[:, None] & (column < (lens // P)[:, None])
    times = torch.zeros(n_pages + table.shape[1], dtype=torch.int32, device=table.device)
    times.scatter_add_(0, torch.where(full & (theirs >= 0), theirs, n_pages + column).flatten(), full.int().flatten())
    shared += times[:n_pages]
    part = child & (lens % P != 0)
    head, tail = s["cursor"][0], s["cursor"][1]
    page = ring[(head + part.cumsum(0) - 1) % ring.numel()]
    src = theirs.gather(1, (lens // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    src, dst = torch.where(part, src, -1), torch.where(part, page, -1)
    ends = part[:, None] & (column == (lens // P)[:, None])
    table.copy_(torch.where(full, theirs, torch.where(ends, page[:, None], table)))
    _copy(s["cache"], src, dst)
    return {"context_lens": lens.int(), "block_table": table, "shared": shared,
            "cursor": torch.stack([head + part.sum(), tail]), "src": src, "dst": dst, "cache": s["cache"]}


def _listed(mask, length):
    """The places where mask is set, in order, then -1 up to length."""
    out = torch.full((length + 1,), -1, dtype=torch.int32, device=mask.device)
    out[torch.where(mask, mask.cumsum(0) - 1, length)] = torch.arange(mask.numel(), dtype=torch.int32,
                                                                      device=mask.device)
    return out[:length]


def _plain_compact(s):
    P, n = s["case"]["page"], s["n_pages"]
    table, shared, ring = s["block_table"], s["shared"], s["ring"]
    column = torch.arange(table.shape[1], device=table.device)[None, :]
    used = (column < ((s["context_lens"].long() + P - 1) // P)[:, None]) & (table >= 0)
    held, free = (torch.zeros(n + 1, dtype=torch.bool, device=table.device) for _ in range(2))
    held[torch.where(used, table, n).long()] = True
    held = held[:n]
    head, tail = s["cursor"][0], s["cursor"][1]
    place = torch.arange(ring.numel(), device=table.device)
    free[torch.where((place - head) % ring.numel() < tail - head, ring, n).long()] = True
    free = free[:n]
    rank, count = (held | free).cumsum(0) - 1, held.sum()
    src, dst = _listed(held & (rank >= count), n // 2), _listed(free & (rank < count), n // 2)
    moved = torch.arange(n + 1, dtype=torch.int32, device=table.device)
    moved[torch.where(src >= 0, src, n).long()] = dst
    table.copy_(torch.where(used, moved[table.clamp(min=0).long()], table))
    more = torch.cat([shared, shared[:1]])
    more[torch.where(dst >= 0, dst, n).long()] = more[src.clamp(min=0).long()]
    more[torch.where(src >= 0, src, n).long()] = 0
    shared.copy_(more[:n])
    rest = (held | free) & (rank >= count)
    wide = torch.cat([ring, ring[:1]])
    wide[torch.where(rest, (head + rank - count) % ring.numel(), ring.numel())] = torch.arange(n, dtype=torch.int32,
                                                                                             device=table.device)
    ring.copy_(wide[:-1])
    _copy(s["cache"], src, dst)
    return {"block_table": table, "shared": shared, "ring": ring, "src": src, "dst": dst, "cache": s["cache"]}


_PLAIN = {"append": _plain_append, "attention": _plain_attention, "verify": _plain_verify, "release": _plain_release,
          "fork": _plain_fork, "compact": _plain_compact}
_OWN = {"append": _own_append, "attention": _own_attention, "verify": _own_verify, "release": _own_release,
        "fork": _own_fork, "compact": _own_compact}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    if case["op"] not in ("append", "attention"):
        return None  # whole numbers, and values that are copied
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    case = s["case"]

    def turned(x, weight):
        x = x.double().clone()
        if weight is not None:
            square = torch.zeros_like(x[..., 0])
            for i in range(case["dim"]):
                square += x[..., i] ** 2
            x = x / torch.sqrt(square / case["dim"] + 1e-6)[..., None] * weight.double()
        half = case["rotary"] // 2
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
            co = s["table"][s["positions"].long(), j].double()[:, None]
            si = s["table"][s["positions"].long(), half + j].double()[:, None]
            x0, x1 = x[:, :, i0].clone(), x[:, :, i1].clone()
            x[:, :, i0] = x0 * co - x1 * si
            x[:, :, i1] = x1 * co + x0 * si
        return x

    caches = []
    for name, x in (("k_cache", turned(s["k"], s["k_norm"])), ("v_cache", s["v"].double())):
        full = s[name].double()
        full[s["slots"] // case["page"], s["slots"] % case["page"]] = x
        caches.append(full)
    return {"q": turned(s["q"], s["q_norm"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attention(s):
    case = s["case"]
    held, new = _lengths(case)
    G, P, D, w, first = case["heads"] // case["kv_heads"], case["page"], case["dim"], case["window"], case["sinks"]
    out = torch.zeros(s["tokens"], case["heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], case["heads"], dtype=torch.float64, device="cuda")
    base = 0
    for r in range(case["requests"]):
        n, total = new[r], held[r] + new[r]
        # the keys that some row sees, by their positions
        begin = max(0, held[r] + 1 - w)
        at = torch.cat([torch.arange(min(first, begin), device="cuda"), torch.arange(begin, total, device="cuda")])
        page = s["block_table"][r, at // P].long()
        for h in range(case["kv_heads"]):
            k, v = (s[c][page, at % P, h].double() for c in ("k_cache", "v_cache"))
            step = max(1, (1 << 26) // (G * at.numel()))
            for t0 in range(0, n, step):
                t1 = min(n, t0 + step)
                x = s["q"][base + t0: base + t1, h * G: (h + 1) * G].double()
                z = (x.reshape(-1, D) @ k.t()).view(t1 - t0, G, at.numel()) / math.sqrt(D)
                pos = torch.arange(held[r] + t0, held[r] + t1, device="cuda")[:, None]
                hidden = (at[None, :] > pos) | ((at[None, :] <= pos - w) & (at[None, :] >= first))
                z = z.masked_fill(hidden[:, None, :], float("-inf"))
                norm = torch.logsumexp(z, -1)
                y = torch.exp(z - norm[..., None]).view(-1, at.numel()) @ v
                out[base + t0: base + t1, h * G: (h + 1) * G] = y.view(t1 - t0, G, D)
                lse[base + t0: base + t1, h * G: (h + 1) * G] = norm
        base += n
    return {"out": out, "lse": lse}
