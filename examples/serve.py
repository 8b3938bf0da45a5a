"""A serving loop on compressed weights and a paged key/value cache.

A Llama-shaped decoder whose weights stay entropy-coded in GPU memory: every
product runs fused with its decode (``decode_gemm``, up to 64 tokens a step),
and the memory that the coding frees holds the cache.  Each step brings new
tokens of several requests -- chunks of prompts beside single tokens -- and

* ``paged_plan`` takes their pages off the free ring and numbers their slots,
* per layer, ``paged_append`` rotates q and k (the products' fp32 outputs),
  rounds them and stores k and v,
* ``paged_attention`` attends over everything stored, or over a window and
  the first tokens (``--window``, ``--sinks``).

With ``--drafts`` the answers are speculative: tokens are drafted by looking up
what followed the last one before, a step brings them along, ``verify_drafts``
says which hold and draws the next one, and ``paged_release`` gives back the
pages of the others, of what the window has passed and of requests that end.
``--norms`` norms the heads of q and k, in the append.

Lengths, tables and cursors stay on the GPU from step to step.  Weights are
random (seeded); ``--check`` recomputes every request with resident weights
and plain attention and compares the logits.

    python examples/serve.py --check
    python examples/serve.py --check --drafts 3 --norms --window 40 --sinks 4
    python examples/serve.py --model llama3-8b --layers 4 --steps 64
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import lossless_entropy_coded_dfc_amd as dfc  # noqa: E402
from lossless_entropy_coded_dfc_amd import synth  # noqa: E402

MODELS = {
    # hidden, heads, kv heads, head dim, feed-forward, vocabulary
    "tiny": (512, 8, 2, 64, 1024, 512),
    "llama3-8b": (4096, 32, 8, 128, 14336, 16384),
}


class Weight:
    """A matrix (rows x cols) held as a panel container, and its product."""

    def __init__(self, bits):
        blob = dfc.encode(bits, layout=dfc.LAYOUT_PANEL, panel_k=256)
        self.info = dfc.blob_info(blob)
        self.blob = torch.from_numpy(blob).cuda()
        self.tables = dfc.derive_tables(self.blob, self.info)
        self.bits = bits

    def __call__(self, x):
        """x (tokens, cols) bfloat16 -> (tokens, rows) float32."""
        y = torch.empty(x.shape[0], int(self.info.rows), dtype=torch.float32, device=x.device)
        dfc.decode_gemm(self.blob, self.info, x.contiguous(), y, tables=self.tables)
        return y

    def resident(self):
        return torch.from_numpy(self.bits.view(np.int16)).cuda().view(torch.bfloat16).float()


def norm(x):
    return (x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Server:
    def __init__(self, model="tiny", layers=2, requests=8, pages=256, page_size=16, max_pages=32, norms=False, window=0,
                 sinks=0):
        hidden, self.heads, self.kv_heads, self.dim, ffn, vocab = MODELS[model]
        shapes = [(self.heads * self.dim, hidden), (self.kv_heads * self.dim, hidden), (self.kv_heads * self.dim, hidden),
                  (hidden, self.heads * self.dim), (ffn, hidden), (ffn, hidden), (hidden, ffn)]
        self.layers = [[Weight(synth.gaussian(s, s[1] ** -0.5, (7, i, j))) for j, s in enumerate(shapes)]
                       for i in range(layers)]
        self.head = Weight(synth.gaussian((vocab, hidden), hidden ** -0.5, (8,)))
        self.embedding = torch.from_numpy(synth.gaussian((vocab, hidden), 1.0, (9,)).view(np.int16)).cuda() \
            .view(torch.bfloat16)
        self.page_size = page_size
        cache = (layers, 2, pages, page_size, self.kv_heads, self.dim)
        self.cache = torch.empty(cache, dtype=torch.bfloat16, device="cuda")
        positions = max_pages * page_size
        angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * \
            500000.0 ** (-torch.arange(0, self.dim, 2, dtype=torch.float64, device="cuda") / self.dim)
        self.rotary = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.context = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda").int()
        self.cursor = torch.tensor([0, pages], device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shared = torch.zeros(pages, dtype=torch.int32, device="cuda")  # (no page is: nothing is forked here)
        self.window, self.sinks = window, sinks
        g = torch.Generator(device="cuda").manual_seed(10)
        self.norms = [tuple(1 + 0.2 * torch.randn(self.dim, generator=g, device="cuda") for _ in range(2)) if norms else
                      (None, None) for _ in range(layers)]

    def step(self, counts, tokens):
        """One step: `counts` new tokens of every request (a list), `tokens`
        their ids in order.  Returns the logits of every new token."""
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        plan = dfc.paged_plan(self.context, new, self.table, self.free, self.cursor, self.page_size, len(tokens),
                              status=self.status)
        x = self.embedding[tokens].float()
        n, most = x.shape[0], max(counts)
        for layer, (q_norm, k_norm), (k_cache, v_cache) in zip(self.layers, self.norms, self.cache):
            wq, wk, wv, wo, gate, up, down = layer
            h = norm(x)
            q, k, v = (w(h).view(n, -1, self.dim) for w in (wq, wk, wv))
            q = dfc.paged_append(k, v, k_cache, v_cache, plan.slots, q=q, positions=plan.positions, rotary=self.rotary,
                                 q_norm=q_norm, k_norm=k_norm, status=self.status)
            o = dfc.paged_attention(q, k_cache, v_cache, self.table, plan.cu_q, plan.seq_lens, max_q_len=most,
                                    window=self.window, sinks=self.sinks, status=self.status)
            x = x + wo(o.view(n, -1))
            h = norm(x)
            x = x + down((torch.nn.functional.silu(gate(h)) * up(h)).to(torch.bfloat16))
        self.context, self.cursor = plan.seq_lens, plan.cursor
        return self.head(norm(x))

    def keep(self, lens):
        """Cuts the requests to their first `lens` tokens (a device vector)
        and gives back the pages that they do not need any more."""
        self.cursor = dfc.paged_release(self.context, lens, self.table, self.free, self.cursor, self.shared,
                                        self.page_size, self.window, self.sinks, status=self.status)
        self.context = lens

    def reference(self, tokens):
        """Logits of one request's tokens, all at once: resident weights, plain
        attention in fp32, values rounded where the server rounds them."""
        x = self.embedding[tokens].float()
        n, half = x.shape[0], self.dim // 2
        cos, sin = self.rotary[:n, None, :half], self.rotary[:n, None, half:]

        def turned(t):
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

        def rounded(t):
            return t.to(torch.bfloat16).float()

        def headnorm(t, weight):
            return t if weight is None else t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * weight

        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        if self.window:
            hidden |= torch.ones_like(hidden).tril(-self.window) & (torch.arange(n, device="cuda") >= self.sinks)
        for layer, (q_norm, k_norm) in zip(self.layers, self.norms):
            wq, wk, wv, wo, gate, up, down = (w.resident() for w in layer)
            h = norm(x).float()
            q, k, v = ((h @ w.t()).view(n, -1, self.dim) for w in (wq, wk, wv))
            q, k, v = rounded(turned(headnorm(q, q_norm))), rounded(turned(headnorm(k, k_norm))), rounded(v)
            k, v = (t.repeat_interleave(self.heads // self.kv_heads, 1) for t in (k, v))
            s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) * self.dim ** -0.5
            p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
            o = torch.matmul(p, v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, -1)
            x = x + rounded(o) @ wo.t()
            h = norm(x).float()
            x = x + rounded(torch.nn.functional.silu(h @ gate.t()) * (h @ up.t())) @ down.t()
        return norm(x).float() @ self.head.resident().t()


def serve(server, prompts, steps, chunk=24, budget=dfc.GEMM_MAX_BATCH):
    """Reads the prompts in chunks and answers greedily, at most `budget`
    tokens a step.  Returns the ids of every request and the last logits."""
    ids = [list(p) for p in prompts]
    read = [0] * len(ids)
    last = [None] * len(ids)
    for _ in range(steps):
        counts, room = [], budget
        for r, p in enumerate(ids):
            n = min(chunk, len(p) - read[r], room)
            counts.append(n)
            room -= n
        tokens = [t for r, n in enumerate(counts) for t in ids[r][read[r]: read[r] + n]]
        logits = server.step(counts, tokens)
        at = 0
        for r, n in enumerate(counts):
            at += n
            read[r] += n
            if n and read[r] == len(ids[r]):
                last[r] = logits[at - 1]
                ids[r].append(int(last[r].argmax()))
    return ids, last


def lookup(ids, most):
    """Up to `most` tokens that followed the last one's latest earlier place."""
    for i in range(len(ids) - 2, -1, -1):
        if ids[i] == ids[-1]:
            return ids[i + 1: i + 1 + most]
    return []


def speculate(server, prompts, length, drafts=3, chunk=24, budget=dfc.GEMM_MAX_BATCH, temperature=0.0, seed=0):
    """As `serve`, with up to `drafts` drafted tokens a step for every request
    that answers, until each has answered `length` tokens; then its pages are
    given back.  Returns the ids of every request, how many steps it took and
    how many drafts held."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids, read, done = [list(p) for p in prompts], [0] * len(prompts), [False] * len(prompts)
    steps = held = 0
    t = torch.full((len(ids),), temperature, device="cuda")
    while not all(done):
        counts, brought, rows, room = [], [], [0], budget
        for r, p in enumerate(ids):
            new = [] if done[r] else p[read[r]: read[r] + min(chunk, room)]
            if new and len(new) == len(p) - read[r] == 1:
                new += lookup(p, min(drafts, room - 1, len(prompts[r]) + length - 1 - len(p)))
            counts.append(len(new))
            brought.append(new)
            room -= len(new)
            # an answer is due once a request's last token is among them
            known = min(len(p) - read[r], len(new))
            rows.append(rows[-1] + (len(new) - known + 1 if new and read[r] + known == len(p) else 0))
        at = np.cumsum([0] + counts)
        due = [rows[r + 1] - rows[r] for r in range(len(ids))]
        logits = server.step(counts, [x for new in brought for x in new])
        picked = [i for r, n in enumerate(due) for i in range(at[r + 1] - n, at[r + 1])]
        follow = [x for r, n in enumerate(due) if n for x in brought[r][len(brought[r]) - n + 1:] + [0]]
        got = dfc.verify_drafts(logits[picked], torch.tensor(rows, dtype=torch.int32, device="cuda"),
                                torch.tensor(follow, dtype=torch.int64, device="cuda"),
                                torch.rand(len(picked), generator=g, device="cuda"), temperature=t, status=server.status)
        keep = list(map(int, np.array(read) + counts))
        for r, (n, a, token) in enumerate(zip(due, got.accepted.tolist(), got.tokens.tolist())):
            read[r] = keep[r]
            if not n:
                continue
            known = len(brought[r]) - (n - 1)
            read[r] += known + a - len(brought[r])
            ids[r] += brought[r][known: known + a] + [token]
            held += a
            done[r] = len(ids[r]) >= len(prompts[r]) + length
            keep[r] = 0 if done[r] else read[r]
        steps += 1
        keep = [0 if done[r] else k for r, k in enumerate(keep)]
        server.keep(torch.tensor(keep, dtype=torch.int32, device="cuda"))
    return ids, steps, held


def shortfall(server, prompts, ids):
    """How far greedy answers' logits are below the largest ones of the
    reference, at most, as a share of a row's norm."""
    worst = 0.0
    for p, i in zip(prompts, ids):
        ref = server.reference(i[:-1])[len(p) - 1:]
        got = ref.gather(1, torch.tensor(i[len(p):], device="cuda")[:, None])[:, 0]
        worst = max(worst, float(((ref.amax(1) - got) / ref.norm(dim=1)).max()))
    return worst


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--model", choices=sorted(MODELS), default="tiny")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--check", action="store_true")
    ap.add_argument("--norms", action="store_true")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--drafts", type=int, default=0, help="drafted tokens a step; answers are --steps tokens long then")
    ap.add_argument("--temperature", type=float, default=0.0, help="of answers with drafts")
    args = ap.parse_args()
    server = Server(args.model, args.layers, args.requests, norms=args.norms, window=args.window, sinks=args.sinks)
    rng = np.random.default_rng(0)
    vocab = server.embedding.shape[0]
    prompts = [rng.integers(0, vocab, 5 + 17 * r).tolist() for r in range(args.requests)]
    serve(Server(args.model, 1, args.requests), prompts, 2)  # warm
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    if args.drafts:
        begin.record()
        ids, steps, held = speculate(server, prompts, args.steps, args.drafts, temperature=args.temperature)
        end.record()
        torch.cuda.synchronize()
        print(f"{args.model}, {args.layers} layers, {args.requests} requests: {steps} steps for {args.steps} tokens each, "
              f"{begin.elapsed_time(end) / steps:.3f} ms a step, {held} drafts held, {int(server.context.sum())} tokens in "
              f"the cache, {int(server.cursor[1] - server.cursor[0])} of {server.free.numel()} pages free, status "
              f"{int(server.status.item())}")
        assert int(server.status.item()) == 0
        if args.check:
            print(f"answers short of the largest logit of plain attention on resident weights by at most "
                  f"{shortfall(server, prompts, ids):.4f} of the logits' norm")
        return
    begin.record()
    ids, last = serve(server, prompts, args.steps)
    end.record()
    torch.cuda.synchronize()
    made = sum(len(i) - len(p) for i, p in zip(ids, prompts))
    print(f"{args.model}, {args.layers} layers, {args.requests} requests: {args.steps} steps, "
          f"{begin.elapsed_time(end) / args.steps:.3f} ms a step, {made} tokens answered, "
          f"{int(server.context.sum())} in the cache, status {int(server.status.item())}")
    assert int(server.status.item()) == 0
    if args.check:
        worst = 0.0
        for i, logits in zip(ids, last):
            ref = server.reference(i[:-1])[-1]
            worst = max(worst, float((logits - ref).norm() / ref.norm()))
        print(f"largest relative difference of the last logits from plain attention on resident weights: {worst:.4f}")
        assert worst < 0.03, worst


if __name__ == "__main__":
    main()
