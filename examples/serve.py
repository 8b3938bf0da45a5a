"""A serving loop on compressed weights and a paged key/value cache.

A Llama-shaped decoder whose weights stay entropy-coded in GPU memory: every
product runs fused with its decode (``decode_gemm``, up to 64 tokens a step),
and the memory that the coding frees holds the cache.  Each step brings new
tokens of several requests -- chunks of prompts beside single tokens -- and

* ``paged_plan`` takes their pages off the free ring and numbers their slots,
* per layer, ``paged_append`` rotates q and k (the products' fp32 outputs),
  rounds them and stores k and v,
* ``paged_attention`` attends over everything stored.

Lengths, tables and cursors stay on the GPU from step to step.  Weights are
random (seeded); ``--check`` recomputes every request with resident weights
and plain attention and compares the logits.

    python examples/serve.py --check
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
    def __init__(self, model="tiny", layers=2, requests=8, pages=256, page_size=16, max_pages=32):
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

    def step(self, counts, tokens):
        """One step: `counts` new tokens of every request (a list), `tokens`
        their ids in order.  Returns the logits of every new token."""
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        plan = dfc.paged_plan(self.context, new, self.table, self.free, self.cursor, self.page_size, len(tokens),
                              status=self.status)
        x = self.embedding[tokens].float()
        n, most = x.shape[0], max(counts)
        for layer, (k_cache, v_cache) in zip(self.layers, self.cache):
            wq, wk, wv, wo, gate, up, down = layer
            h = norm(x)
            q, k, v = (w(h).view(n, -1, self.dim) for w in (wq, wk, wv))
            q = dfc.paged_append(k, v, k_cache, v_cache, plan.slots, q=q, positions=plan.positions, rotary=self.rotary,
                                 status=self.status)
            o = dfc.paged_attention(q, k_cache, v_cache, self.table, plan.cu_q, plan.seq_lens, max_q_len=most,
                                    status=self.status)
            x = x + wo(o.view(n, -1))
            h = norm(x)
            x = x + down((torch.nn.functional.silu(gate(h)) * up(h)).to(torch.bfloat16))
        self.context, self.cursor = plan.seq_lens, plan.cursor
        return self.head(norm(x))

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

        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for layer in self.layers:
            wq, wk, wv, wo, gate, up, down = (w.resident() for w in layer)
            h = norm(x).float()
            q, k, v = ((h @ w.t()).view(n, -1, self.dim) for w in (wq, wk, wv))
            q, k, v = rounded(turned(q)), rounded(turned(k)), rounded(v)
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


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--model", choices=sorted(MODELS), default="tiny")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args()
    server = Server(args.model, args.layers, args.requests)
    rng = np.random.default_rng(0)
    vocab = server.embedding.shape[0]
    prompts = [rng.integers(0, vocab, 5 + 17 * r).tolist() for r in range(args.requests)]
    serve(Server(args.model, 1, args.requests), prompts, 2)  # warm
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
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
