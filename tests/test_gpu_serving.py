"""GPU: the serving operators together over many steps, as a program uses them:
plan, normed append, attention with a window and sinks, verification of the
drafts, pages given back, requests that end, begin and are forked, the cache made
dense.  Every step's bookkeeping is compared with the oracle's (equal), and its
attention with the definition over everything a request has stored so far, kept
apart from the cache: whatever loses or mixes up a page shows.  The bound is
test_gpu_paged.py's."""
import sys

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op
from oracle import verify as ov

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def as64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Program:
    """Two layers' caches and a pool of pages; request r's answers are drawn
    from logits that are a fixed function of its attention's output."""

    R, H, K, D, P, V, WIDTH = 9, 4, 2, 64, 8, 300, 40

    def __init__(self, pages, window, sinks, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.window, self.sinks, self.pages = window, sinks, pages
        self.cache = torch.full((2, 2, pages, self.P, self.K, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((self.R, self.WIDTH), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(pages, generator=self.g, device="cuda").int()
        self.cursor = torch.tensor([5 * pages, 6 * pages], device="cuda")
        self.shared = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.context = i32([0] * self.R)
        self.status = i32([0])
        angle = torch.arange(self.WIDTH * self.P, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, self.D, 2, dtype=torch.float64) / self.D)
        self.rotary = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.wq, self.wk = (1 + 0.2 * self.randn(self.D) for _ in range(2))
        self.head = 0.6 * self.randn(self.H * self.D, self.V)
        self.temperature = torch.tensor([0.0, 0.7, 1.0, 1.3, 0.9, 0.0, 0.8, 1.0, 0.6], device="cuda")
        self.given = [[[] for _ in range(self.R)] for _ in range(2)]   # per layer and request: (k, v) of every token

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def books(self):
        return [t.cpu().numpy().copy() for t in (self.table, self.ring, self.cursor, self.shared)]

    def same(self, got, want):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)

    def consistent(self):
        """Every page is held by as many as its count says, or is free."""
        table, ring, (head, tail), shared = self.books()
        holders = np.zeros(self.pages, int)
        for r, c in enumerate(self.context.tolist()):
            for p in table[r, : -(-c // self.P)]:
                if p >= 0:
                    holders[p] += 1
        free = [ring[i % self.pages] for i in range(head, tail)]
        assert len(set(free)) == len(free) and not any(holders[p] for p in free)
        assert len(free) + (holders > 0).sum() == self.pages
        assert np.array_equal(shared, np.maximum(holders - 1, 0))

    def step(self, counts):
        """`counts` tokens of every request, all but the first of them drafts.
        Returns how many tokens each keeps."""
        n, held = sum(counts), self.context.tolist()
        table, ring, cursor, _ = self.books()
        plan = dfc.paged_plan(self.context, i32(counts), self.table, self.ring, self.cursor, self.P, n, status=self.status)
        want = op.plan(held, counts, table, ring, cursor, self.P, n)
        self.same((self.table, plan.seq_lens, plan.cu_q, plan.slots, plan.positions, plan.cursor), want)
        self.cursor = plan.cursor
        for layer, (kc, vc) in enumerate(self.cache):
            q, k, v = (self.randn(n, heads, self.D) for heads in (self.H, self.K, self.K))
            q = dfc.paged_append(k, v, kc, vc, plan.slots, q=q, positions=plan.positions, rotary=self.rotary,
                                 q_norm=self.wq, k_norm=self.wk, status=self.status)
            out, lse = dfc.paged_attention(q, kc, vc, self.table, plan.cu_q, plan.seq_lens, window=self.window,
                                           sinks=self.sinks, lse=True, status=self.status)
            self.remember(layer, counts, plan.slots)
            self.compare(layer, counts, held, q, out)
        logits = out.float().flatten(1) @ self.head
        drafter = logits + 0.5 * self.randn(n, self.V)
        drafts = torch.where(self.randn(n) > 0, drafter.argmax(1), torch.randint(0, self.V, (n,), generator=self.g,
                                                                               device="cuda"))
        u = torch.rand(n, generator=self.g, device="cuda")
        got = dfc.verify_drafts(logits, plan.cu_q, drafts, u, draft_logits=drafter, temperature=self.temperature,
                                status=self.status)
        cu = plan.cu_q.tolist()
        kept = list(held)
        for r, c in enumerate(counts):
            rows = slice(cu[r], cu[r + 1])
            if not c:
                assert (int(got.accepted[r]), int(got.tokens[r])) == (0, -1)
                continue
            a, token, margin = ov.request(as64(logits[rows]), drafts[rows].tolist(), u[rows].tolist(), as64(drafter[rows]),
                                          float(self.temperature[r]))
            assert margin > 1e-10 and (int(got.accepted[r]), int(got.tokens[r])) == (a, token)
            kept[r] = held[r] + 1 + a
        # on the device, as a program does it
        keep = torch.where(i32(counts) > 0, self.context + 1 + got.accepted, self.context)
        assert keep.tolist() == kept
        self.context = plan.seq_lens
        return keep

    def remember(self, layer, counts, slots):
        kk, vv = (as64(c.flatten(0, 1)[slots]) for c in self.cache[layer])
        at = 0
        for r, c in enumerate(counts):
            self.given[layer][r] += [(kk[at + i], vv[at + i]) for i in range(c)]
            at += c

    def compare(self, layer, counts, held, q, out):
        at = 0
        for r, c in enumerate(counts):
            if c:
                assert len(self.given[layer][r]) == held[r] + c
                k, v = (np.stack([t[i] for t in self.given[layer][r]]) for i in range(2))
                ref, _, spread, top, mass = op.attention(as64(q[at: at + c]), k, v, self.D ** -0.5, window=self.window,
                                                         sinks=self.sinks)
                e = 2.0 ** -23 * (self.D * mass + 2 * top + len(k) + 16)[..., None]
                bound = (U + 2 * e) * spread + U * np.abs(ref) + 1e-30
                assert (np.abs(as64(out[at: at + c]) - ref) <= bound).all(), (layer, r)
            at += c

    def release(self, keep):
        want = op.release(self.context.tolist(), keep.tolist(), *self.books(), self.P, self.window, self.sinks)
        self.cursor = dfc.paged_release(self.context, keep, self.table, self.ring, self.cursor, self.shared, self.P,
                                        self.window, self.sinks, status=self.status)
        assert want[4] == []
        self.same((self.table, self.ring, self.cursor, self.shared), want[:4])
        self.context = keep
        for layer in self.given:
            for r, n in enumerate(keep.tolist()):
                del layer[r][n:]
        self.consistent()

    def fork(self, parents, lens=None):
        held = self.context.tolist()
        table, ring, cursor, shared = self.books()
        f = dfc.paged_fork(self.context, i32(parents), self.table, self.ring, self.cursor, self.shared, self.P,
                           fork_lens=None if lens is None else i32(lens), status=self.status)
        dfc.paged_copy([(c[0], c[1]) for c in self.cache], f.src, f.dst, status=self.status)
        context, table, shared, cursor, src, dst = op.fork(held, parents, table, ring, cursor, shared, self.P, lens)
        self.same((f.context_lens, self.table, self.shared, f.cursor, f.src, f.dst),
                  (context, table, shared, cursor, src, dst))
        self.context, self.cursor = f.context_lens, f.cursor
        for layer in self.given:
            for r, p in enumerate(parents):
                if p >= 0:
                    layer[r] = list(layer[p][: int(context[r])])
        self.consistent()

    def compact(self):
        table, ring, cursor, shared = self.books()
        m = dfc.paged_compact(self.context, self.table, self.ring, self.cursor, self.shared, self.P, status=self.status)
        dfc.paged_copy([(c[0], c[1]) for c in self.cache], m.src, m.dst, status=self.status)
        self.same((self.table, self.ring, self.shared, m.src, m.dst),
                  op.compact(self.context.tolist(), table, ring, cursor, shared, self.P))
        self.consistent()
        used = int(m.used)
        assert all(p < used for p in self.table.flatten().tolist() if p >= 0)   # nothing is reserved here
        self.cache[:, :, used:] = float("nan")


@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4), (17, 12), (64, 1)])
def test_a_program_over_many_steps(window, sinks):
    p = Program(pages=340, window=window, sinks=sinks, seed=window + 1)
    rng = np.random.default_rng(window)
    R = p.R
    for turn in range(26):
        held = p.context.tolist()
        busy = [c > 0 for c in held]
        # prompts for empty requests now and then, one token and drafts for the others
        counts = [0 if c > 200 else 1 + int(rng.integers(0, 5)) if c else int(rng.integers(5, 60)) if rng.random() < 0.5
                  else 0 for c in held]
        if not sum(counts):
            counts[held.index(0) if 0 in held else 0] = 1
        say("turn", turn, "window", window, "held", held, "new", counts)
        keep = p.step(counts)
        # a prompt's tokens are given, not drafted: all of them are kept
        keep = torch.where(i32([int(b) for b in busy]) > 0, keep, torch.where(i32(counts) > 0, i32(counts), p.context))
        # some requests end; long ones do for sure
        ends = [int(c > 180 or (turn % 3 == 2 and rng.random() < 0.25)) for c in keep.tolist()]
        p.release(torch.where(i32(ends) > 0, torch.zeros_like(keep), keep))
        held = p.context.tolist()
        if turn % 4 == 1:
            parents = [-1] * R
            full = [r for r, c in enumerate(held) if c]
            for r, c in enumerate(held):
                if not c and full and rng.random() < 0.7:
                    parents[r] = int(rng.choice(full))
            p.fork(parents)
        if turn % 5 == 3:
            p.compact()
    assert int(p.status.item()) == 0
    p.release(torch.zeros_like(p.context))
    assert not p.shared.any() and int(p.cursor[1] - p.cursor[0]) == p.pages


@pytest.mark.parametrize("given", ["another stream", "the default stream"])
def test_what_a_call_allocates_belongs_to_its_stream(given):
    # a given stream does not wait for the current one, whose earlier work may
    # still use memory that torch hands out on the current stream
    from test_gpu_paged import pool_of
    R, P, pages = 3, 8, 40
    lens, keep, parents = i32([50, 23, 0]), i32([44, 0, 0]), i32([-1, -1, 0])
    table = i32([[*range(7)], [*range(10, 13)] + [-1] * 4, [-1] * 7])
    free = torch.tensor([p for p in range(pages) if p > 6 and not 10 <= p < 13], device="cuda").int()
    logits, cu = torch.randn(5, 700, device="cuda"), i32([0, 3, 4, 5])
    u, x = torch.rand(5, device="cuda"), torch.randint(0, 700, (5,), device="cuda")
    cache = torch.randn(2, pages, P, 2, 64, device="cuda").bfloat16()
    k, w = torch.randn(4, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    slots = torch.arange(4, device="cuda")

    def calls(stream):
        t, ring, cursor, shared = table.clone(), free.clone(), torch.tensor([0, free.numel()], device="cuda"), i32([0] * pages)
        ring = torch.cat([ring, i32([0] * 20)])
        c = cache.clone()
        torch.cuda.synchronize()
        end = dfc.paged_release(lens, keep, t, ring, cursor, shared, P, stream=stream)
        f = dfc.paged_fork(keep, parents, t, ring, end, shared, P, stream=stream)
        dfc.paged_copy([(c[0], c[1])], f.src, f.dst, stream=stream)
        m = dfc.paged_compact(f.context_lens, t, ring, f.cursor, shared, P, stream=stream)
        dfc.paged_copy([(c[0], c[1])], m.src, m.dst, stream=stream)
        v = dfc.verify_drafts(logits, cu, x, u, draft_logits=logits.flip(0), stream=stream)
        q = dfc.paged_append(k, k, c[0], c[1], slots, q=k, q_norm=w, k_norm=w, stream=stream)
        torch.cuda.synchronize()
        return [end, *f, *m, *v, q], [t, ring, shared, c]

    plain, kept = calls(None)
    side = torch.cuda.Stream()
    say("allocations", given)
    if given == "another stream":
        handle, (got, left) = side.cuda_stream, calls(side.cuda_stream)
    else:
        with torch.cuda.stream(side):
            handle, (got, left) = 0, calls(0)
    for a, b in zip(plain, got):
        assert pool_of(b) == handle and torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(kept, left))


def test_captured_steps_follow_their_inputs():
    """Plan, append, attention, verification and release captured once, fork and
    copy and compact each once; replays with other lengths between them, with
    eager work between the replays, match the eager calls."""
    R, H, K, D, P, V, T, pages = 4, 4, 2, 64, 8, 1500, 12, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")
    context, new, keep = i32([0] * R), i32([0] * R), i32([0] * R)
    table = torch.full((R, 24), -1, dtype=torch.int32, device="cuda")
    ring, cursor = torch.randperm(pages, generator=g, device="cuda").int(), torch.tensor([0, pages], device="cuda")
    shared, parents = torch.zeros(pages, dtype=torch.int32, device="cuda"), i32([-1] * R)
    caches = torch.zeros(2, 2, pages, P, K, D, dtype=torch.bfloat16, device="cuda")
    q, k, v, u, w = randn(T, H, D), randn(T, K, D), randn(T, K, D), torch.rand(T, device="cuda"), 1 + 0.1 * randn(D)
    rotary, drafts = randn(192, D), torch.zeros(T, dtype=torch.int64, device="cuda")
    logits, drafter = randn(T, V), randn(T, V)
    t, status = torch.tensor([0.0, 1.0, 0.7, 1.2], device="cuda"), i32([0])

    def step():
        plan = dfc.paged_plan(context, new, table, ring, cursor, P, T, status=status)
        outs = []
        for kc, vc in caches:
            x = dfc.paged_append(k, v, kc, vc, plan.slots, q=q, positions=plan.positions, rotary=rotary, q_norm=w,
                                 k_norm=w, status=status)
            outs.append(dfc.paged_attention(x, kc, vc, table, plan.cu_q, plan.seq_lens, window=20, sinks=3,
                                            status=status))
        ver = dfc.verify_drafts(logits, plan.cu_q, drafts, u, draft_logits=drafter, temperature=t, status=status)
        keep.copy_(torch.where(new > 0, context + 1 + ver.accepted, context))
        end = dfc.paged_release(plan.seq_lens, keep, table, ring, plan.cursor, shared, P, 20, 3, status=status)
        cursor.copy_(end)
        context.copy_(keep)
        return (*outs, ver.accepted, ver.tokens, plan.cu_q)

    def split():
        f = dfc.paged_fork(context, parents, table, ring, cursor, shared, P, status=status)
        dfc.paged_copy([(c[0], c[1]) for c in caches], f.src, f.dst, status=status)
        context.copy_(f.context_lens)
        cursor.copy_(f.cursor)
        return f.src, f.dst

    def dense():
        m = dfc.paged_compact(context, table, ring, cursor, shared, P, status=status)
        dfc.paged_copy([(c[0], c[1]) for c in caches], m.src, m.dst, status=status)
        return tuple(m)

    state = (context, keep, table, ring, cursor, shared, caches)
    begin = [x.clone() for x in state]
    graphs = []
    for call in (step, split, dense):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        graphs.append((graph, outs, call))
    for x, y in zip(state, begin):
        x.copy_(y)
    torch.cuda.synchronize()
    rounds = [([5, 4, 0, 3], None, False), ([1, 2, 0, 1], [-1, -1, 0, -1], False), ([3, 1, 4, 4], None, True),
              ([1, 1, 1, 1], None, False), ([6, 0, 2, 4], None, True), ([1, 5, 5, 1], None, False)]
    for i, (counts, fork, compact) in enumerate(rounds):
        for x in (q, k, v, logits, drafter):
            x.normal_()
        u.uniform_()
        drafts.copy_(drafter.argmax(1))
        new.copy_(i32(counts))
        parents.copy_(i32(fork or [-1] * R))
        for (graph, outs, call), on in zip(graphs, (True, fork is not None, compact)):
            if not on:
                continue
            before = [x.clone() for x in state]
            say("replay", i, call.__name__)
            graph.replay()
            torch.cuda.synchronize()
            replayed = [x.clone() for x in (*outs, *state)]
            for x, y in zip(state, before):
                x.copy_(y)
            eager = call()
            torch.cuda.synchronize()
            n = sum(counts)
            for j, (a, b) in enumerate(zip(replayed, (*eager, *state))):
                if call is step and j < 2:   # rows behind the last request are left as they were
                    a, b = a[:n], b[:n]
                assert torch.equal(a, b), (i, call.__name__, j)
    assert int(status.item()) == 0


def test_two_programs_at_once():
    """Steps of two programs on two streams, neither waiting for the other: each
    one's results are those it has alone."""
    R, H, K, D, P, V, T, pages, rounds = 70, 4, 2, 64, 8, 9000, 210, 1024, 6

    def program(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")
        context = torch.randint(0, 60, (R,), generator=g, device="cuda").int()
        new = torch.full((R,), 3, dtype=torch.int32, device="cuda")
        table, ring = i32([[-1] * 20] * R), torch.randperm(pages, generator=g, device="cuda").int()
        cursor, shared, status = torch.tensor([0, pages], device="cuda"), i32([0] * pages), i32([0])
        caches = randn(2, pages, P, K, D).bfloat16()
        q, k, v, u, w = randn(T, H, D), randn(T, K, D), randn(T, K, D), torch.rand(T, generator=g, device="cuda"), randn(D)
        logits, drafter, drafts = randn(T, V), randn(T, V), torch.randint(0, V, (T,), generator=g, device="cuda")
        parents = i32([-1] * (R - 3) + [0, 1, 2])
        torch.cuda.synchronize()
        outs, none = [], torch.zeros_like(context)
        # what they hold at first
        first = dfc.paged_plan(none, context, table, ring, cursor, P, int(R * 60), status=status)
        cursor, keep = first.cursor, context
        for _ in range(rounds):
            plan = dfc.paged_plan(keep, new, table, ring, cursor, P, T, status=status)
            x = dfc.paged_append(k, v, caches[0], caches[1], plan.slots, q=q, q_norm=w, k_norm=w, status=status)
            x = dfc.paged_attention(x, caches[0], caches[1], table, plan.cu_q, plan.seq_lens, window=30, sinks=9,
                                    status=status)
            ver = dfc.verify_drafts(logits, plan.cu_q, drafts, u, draft_logits=drafter, status=status)
            keep = keep + 1 + ver.accepted
            keep[-3:] = 0
            cursor = dfc.paged_release(plan.seq_lens, keep, table, ring, plan.cursor, shared, P, status=status)
            f = dfc.paged_fork(keep, parents, table, ring, cursor, shared, P, status=status)
            dfc.paged_copy([tuple(caches)], f.src, f.dst, status=status)
            m = dfc.paged_compact(f.context_lens, table, ring, f.cursor, shared, P, status=status)
            dfc.paged_copy([tuple(caches)], m.src, m.dst, status=status)
            keep, cursor = f.context_lens, f.cursor
            outs += [x, *ver, *f, *m]
            yield None
        yield [*outs, table, ring, shared, status, caches]

    alone = []
    for seed in (1, 2):
        say("alone", seed)
        *_, got = program(seed)
        torch.cuda.synchronize()
        alone.append(got)
        assert int(got[-2]) == 0
    streams, programs = [torch.cuda.Stream() for _ in range(2)], [program(1), program(2)]
    got = [None, None]
    say("both")
    for _ in range(rounds + 1):
        for i, (stream, p) in enumerate(zip(streams, programs)):
            with torch.cuda.stream(stream):
                got[i] = next(p)
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
