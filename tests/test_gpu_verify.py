"""GPU: verification of drafted tokens (dfc_verify_drafts) against the oracle's
definition in 64 bits.  What comes out is whole numbers, and they are equal
wherever no comparison is within 1e-10 of its border (relative): the kernels'
exponentials and sums are in 64 bits, whose roundings reach some 1e-13 for
logits apart by hundreds.  Such cases are counted: hardly any may be left out."""
import sys

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import verify as ov

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NEAR = 1e-10


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


class Step:
    """Requests with `counts` rows each; drafts drawn from the drafter's
    logits, from the model's favourites where there is no drafter."""

    def __init__(self, counts, vocab, dtype=torch.float32, drafter=True, seed=0, spread=2.0, temperature=None, pad=0):
        g = torch.Generator().manual_seed(seed)
        rows = sum(counts)
        self.counts, self.vocab = counts, vocab
        z = spread * torch.randn(rows, vocab, generator=g)
        if vocab > 4:
            z.scatter_add_(1, torch.randint(0, vocab, (rows, 3), generator=g), 3 * spread + torch.randn(rows, 3, generator=g))
        d = z + 0.7 * spread * torch.randn(rows, vocab, generator=g)
        # rows apart from each other, and the padding something that must not be read
        self.store = torch.full((2, rows, vocab + pad), float("nan")).to(dtype)
        self.store[0, :, :vocab], self.store[1, :, :vocab] = z.to(dtype), d.to(dtype)
        self.z, self.d = self.store[0, :, :vocab], self.store[1, :, :vocab] if drafter else None
        self.cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
        t = torch.tensor([(0.0, 0.5, 1.0, 1.7, 0.9)[(r + seed) % 5] for r in range(len(counts))])
        self.t = t if temperature is None else torch.full((len(counts),), temperature)
        noise = -torch.log(-torch.log(torch.rand(rows, vocab, generator=g).clamp_(1e-30, 1 - 1e-7)))
        row_t = self.t.repeat_interleave(torch.tensor(counts))[:, None] if rows else torch.zeros(0, 1)
        self.x = (self.store[1, :, :vocab].float() + row_t * noise).argmax(1) if rows else torch.zeros(0, dtype=torch.int64)
        self.u = torch.rand(rows, generator=g)

    def run(self, **kw):
        dev = self.store.cuda()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        v = dfc.verify_drafts(dev[0, :, :self.vocab], self.cu.cuda(), self.x.cuda(), self.u.cuda(),
                              draft_logits=None if self.d is None else dev[1, :, :self.vocab],
                              temperature=None if self.t is None else self.t.cuda(), status=st, **kw)
        torch.cuda.synchronize()
        return v.accepted.tolist(), v.tokens.tolist(), int(st.item())

    def want(self, r):
        a, b = int(self.cu[r]), int(self.cu[r + 1])
        if a == b:
            return 0, -1, 1.0
        t = 1.0 if self.t is None else float(self.t[r])
        return ov.request(self.z[a:b].double().numpy(), self.x[a:b].tolist(), self.u[a:b].tolist(),
                          None if self.d is None else self.d[a:b].double().numpy(), t)

    def check(self, got, left_out=0):
        accepted, tokens, _ = got
        near = 0
        for r in range(len(self.counts)):
            a, token, margin = self.want(r)
            if margin <= NEAR:
                near += 1
                continue
            assert (accepted[r], tokens[r]) == (a, token), (r, (accepted[r], tokens[r]), (a, token), margin)
        assert near <= left_out, near


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 65, 1000, 1024, 1025, 4099, 50001])
def test_against_the_definition(vocab, dtype, drafter):
    counts = [1, 3, 6, 0, 2, 9, 1, 4, 5, 17]
    for seed in range(2 if vocab > 5000 else 6):
        s = Step(counts, vocab, dtype, drafter, seed=seed + vocab)
        say("verify", vocab, dtype, drafter, seed)
        got = s.run()
        assert got[2] == 0
        s.check(got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_large_vocabulary(dtype):
    for counts, drafter in (([1], False), ([6, 1, 4], True), ([8, 2], False)):
        s = Step(counts, 128256, dtype, drafter, seed=len(counts))
        say("verify, large vocabulary", counts, dtype)
        s.check(s.run())


def test_rows_apart_and_unaligned():
    for vocab, pad in ((1000, 7), (1001, 1), (2048, 8), (130, 500)):
        for dtype in (torch.float32, torch.float16):
            s = Step([3, 1, 5], vocab, dtype, True, seed=pad, pad=pad)
            say("verify, rows apart", vocab, pad, dtype)
            s.check(s.run())


def test_temperatures():
    for t in (0.0, 1e-3, 0.05, 3.0, 1e4, 1e-30, 3e38):
        s = Step([4] * 8, 3000, seed=5, temperature=t)
        say("verify, temperature", t)
        got = s.run()
        assert got[2] == 0
        s.check(got)
    s = Step([4] * 8, 3000, seed=6)
    s.t = None
    s.check(s.run())


def test_many_requests():
    counts = [1 + (r * 7) % 5 for r in range(1000)]
    s = Step(counts, 300, seed=3)
    say("verify, many requests")
    s.check(s.run(), left_out=1)


def test_ties_go_to_the_lowest_index():
    z = torch.zeros(4, 5000)
    z[0, [4000, 77, 1500]] = 3.0
    z[1] = -1.0
    z[2, 4999] = 1.0
    z[3, [1024, 1023]] = 2.0
    s = Step([1, 1, 1, 1], 5000, drafter=False, temperature=0.0)
    s.store[0, :, :] = z
    assert s.run() == ([0] * 4, [77, 0, 4999, 1023], 0)


def test_masked_logits_have_no_probability():
    s = Step([5, 5, 1], 3000, seed=8)
    open_to = torch.tensor([5, 1999, 2047, 2999])
    keep = torch.zeros(3000, dtype=torch.bool)
    keep[open_to] = True
    s.store[0][:, :3000] = torch.where(keep, s.z, -torch.inf)
    s.z = s.store[0]
    for seed in range(20):
        s.u = torch.rand(11, generator=torch.Generator().manual_seed(seed))
        got = s.run()
        assert got[2] == 0 and all(t in open_to.tolist() for t in got[1])
        s.check(got)
    # a drafter that names what the model never says
    s.x[:] = 17
    got = s.run()
    assert got[0] == [0, 0, 0]
    s.check(got)
    # a drafter whose only tokens are others: what is left is all of p
    s.store[1][:, :3000] = torch.where(keep, -torch.inf, s.store[1])
    s.d = s.store[1]
    got = s.run()
    assert got[0] == [0, 0, 0]
    s.check(got)


def test_random_numbers_at_the_ends():
    for certain in (True, False):
        s = Step([1, 3, 6, 2], 2000, drafter=not certain, seed=9, temperature=0.8)
        for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 7.0, -3.0, float("inf"), float("nan"), 2.0 ** -60):
            s.u[:] = u
            say("verify, random numbers of", u)
            got = s.run()
            for r in range(4):
                a, token, _ = s.want(r)
                assert got[0][r] == a
                if 0 < u < 1:   # (at 0 and past 1 the border is the number itself)
                    assert got[1][r] == token
                assert 0 <= got[1][r] < 2000


def test_random_numbers_that_are_none():
    """Below 0 they count as 0, from 1 on as the largest below it; NaN holds no draft."""
    # p: 0.25, 0.75, 0, 0; all of it on token 1; the drafts have p > 0, p = 0, p = 1 and none
    z = torch.tensor([[0.0, np.log(3.0), -np.inf, -np.inf], [-np.inf, 0.0, -np.inf, -np.inf]],
                     dtype=torch.float32)
    cases = [(0, 0), (0, 2), (1, 1), (0, 7), (0, -3)]
    us = [-1.0, -0.0, float("-inf"), 1.0, 2.0, float("inf"), float("nan")]
    for drafter in (False, True):
        logits = torch.cat([z[[row, 0]] for row, _ in cases for _ in us])
        drafts = torch.tensor([[x, 0] for _, x in cases for _ in us]).flatten()
        u = torch.tensor([[v, 0.5] for _ in cases for v in us]).flatten()
        cu = torch.arange(0, len(u) + 1, 2, dtype=torch.int32)
        q = torch.zeros_like(logits) if drafter else None
        say("verify, random numbers that are none", drafter)
        got = dfc.verify_drafts(logits.cuda(), cu.cuda(), drafts.cuda(), u.cuda(),
                                draft_logits=None if q is None else q.cuda())
        torch.cuda.synchronize()
        for r in range(len(cu) - 1):
            i = slice(2 * r, 2 * r + 2)
            want = ov.request(logits[i].double().numpy(), drafts[i].tolist(), u[i].tolist(),
                              None if q is None else q[i].double().numpy())[:2]
            assert (int(got.accepted[r]), int(got.tokens[r])) == want, (drafter, r)
        if not drafter:
            held = got.accepted.reshape(len(cases), len(us)).tolist()
            assert held[0] == [1, 1, 1, 0, 0, 0, 0] and held[2] == [1] * 6 + [0]
            assert held[1] == held[3] == held[4] == [0] * 7


@pytest.mark.parametrize("vocab", [70, 5000, 300001])
def test_random_numbers_at_the_borders_of_few_tokens(vocab):
    """Most logits -inf, random numbers next to the sums' borders: whatever
    the roundings do there, a token without probability is never drawn."""
    g = torch.Generator().manual_seed(vocab)
    row = torch.full((vocab,), float("-inf"))
    at = torch.randperm(vocab, generator=g)[:20].sort().values
    row[at] = torch.randn(20, generator=g)
    p = ov.softmax(row.numpy(), 1.0)
    sums = np.cumsum(p)[at.numpy()]
    u = torch.tensor(sums, dtype=torch.float32)
    u = torch.cat([u, torch.nextafter(u, torch.zeros(1)), torch.nextafter(u, torch.ones(1))])
    cu = torch.arange(len(u) + 1, dtype=torch.int32)
    say("verify, borders of few tokens", vocab)
    v = dfc.verify_drafts(row.cuda().expand(len(u), vocab).contiguous(), cu.cuda(),
                          torch.zeros(len(u), dtype=torch.int64, device="cuda"), u.cuda())
    tokens = v.tokens.cpu()
    assert torch.isin(tokens, at).all()
    for t, x in zip(tokens.tolist(), u.tolist()):
        j, near = ov.pick(p, x)
        assert near <= NEAR or t == j


def test_the_same_logits_for_drafter_and_model_hold_everything():
    s = Step([6] * 20, 700, seed=10, temperature=1.3)
    s.store[1] = s.store[0]
    s.d = s.store[1]
    s.x = torch.randint(0, 700, (120,))
    got = s.run()
    assert got[0] == [5] * 20 and got[2] == 0
    s.check(got)


def test_what_is_drawn_is_distributed_as_the_logits():
    # 60,000 requests of one row and the same logits, random numbers on an even
    # grid: every token as often as its probability says, to one grid point
    n, vocab = 60000, 40
    z = torch.randn(vocab, generator=torch.Generator().manual_seed(1)) * 1.5
    logits = z.expand(n, vocab).contiguous().cuda()
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().cuda()
    say("distribution")
    v = dfc.verify_drafts(logits, torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                          torch.zeros(n, dtype=torch.int64, device="cuda"), u)
    p = ov.softmax(z.double().numpy(), 1.0)
    counts = np.bincount(v.tokens.cpu().numpy(), minlength=vocab)
    # (a random number in 32 bits is off by up to 2^-25 n grid points)
    assert np.abs(counts - n * p).max() <= 1 + 2 * n * 2.0 ** -25 and not v.accepted.any()


def test_answers_with_drafts_are_distributed_as_the_logits():
    # one draft each, drawn from q on a grid; the first token then follows p
    m, vocab = 244, 6
    g = torch.Generator().manual_seed(2)
    z, d = 1.2 * torch.randn(2, vocab, generator=g), 1.2 * torch.randn(vocab, generator=g)
    p, q = ov.softmax(z[0].double().numpy(), 0.8), ov.softmax(d.double().numpy(), 0.8)
    grid = (np.arange(m) + 0.5) / m
    u0, u1 = (torch.from_numpy(x.ravel()).float() for x in np.meshgrid(grid, grid, indexing="ij"))
    n = m * m
    logits, draft = z.repeat(n, 1).cuda(), d.expand(2 * n, vocab).contiguous().cuda()
    u = torch.stack([u0, u1], 1).flatten().cuda()
    mass = np.zeros(vocab)
    for x in range(vocab):
        say("distribution with a draft", x)
        v = dfc.verify_drafts(logits, torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"),
                              torch.full((2 * n,), x, device="cuda"), u, draft_logits=draft,
                              temperature=torch.full((n,), 0.8, device="cuda"))
        first = torch.where(v.accepted > 0, x, v.tokens).cpu().numpy()
        mass += q[x] * np.bincount(first, minlength=vocab) / n
    assert np.abs(mass - p).max() <= 2.0 / m


def test_rows_without_probabilities():
    for bad in (float("nan"), float("inf"), None):
        s = Step([3, 3, 1, 2], 2500, seed=11, temperature=0.7)
        s.x = s.z.argmax(1)     # drafts that hold for sure with a small random number
        s.u[:] = 1e-6
        row = 1
        if bad is None:
            s.store[0, row, :] = -torch.inf
        else:
            s.store[0, row, 1700] = bad
        say("verify, bad row", bad)
        got = s.run()
        assert got[2] == dfc.ECORRUPT and (got[0][0], got[1][0]) == (1, -1)
        s.z = s.store[0, :, :2500]
        s.check(got)
        # the drafter's, in the first request's second row
        s = Step([3, 3, 1, 2], 2500, seed=11, temperature=0.7)
        s.x = s.z.argmax(1)
        s.u[:] = 1e-6
        s.store[1, row, :] = bad if bad is not None else -torch.inf
        s.d = s.store[1, :, :2500]
        got = s.run()
        assert got[2] == dfc.ECORRUPT and (got[0][0], got[1][0]) == (1, -1)
        s.check(got)
        # of a last row nothing was drafted, and greedy answers ask no drafter
        s.store[1, :, :] = float("nan")
        s.t[:] = 0.0
        got = s.run()
        assert got[2] == 0
        s.check(got)
    # a bad row behind the one that refuses a draft is not looked at
    s = Step([3], 2500, seed=12, temperature=0.0)
    s.x[0] = (int(s.z[0].argmax()) + 1) % 2500
    s.store[0, 1] = float("nan")
    got = s.run()
    assert got == ([0], [int(s.z[0].argmax())], 0)


def test_temperatures_and_drafts_that_make_no_sense():
    s = Step([2, 2, 2, 2], 900, seed=13)
    s.t = torch.tensor([-1.0, float("nan"), float("inf"), 1.0])
    got = s.run()
    assert got[2] == dfc.ECORRUPT and got[0][:3] == [0, 0, 0] and got[1][:3] == [-1, -1, -1]
    s.check(got)
    for drafter in (True, False):
        for t in (0.0, 1.0):
            for x in (-1, 900, 2 ** 40, -2 ** 63):
                s = Step([3, 1], 900, drafter=drafter, seed=14, temperature=t)
                s.x[0] = x
                got = s.run()
                assert got[2] == dfc.ECORRUPT and got[0][0] == 0
                s.check(got)
    # the last row's entry is not read
    s = Step([1, 1], 900, seed=14)
    s.x[:] = 10 ** 9
    assert s.run()[2] == 0


def test_row_ranges_that_make_no_sense():
    for cu in ([0, 5, 3, 8], [-3, 2, 4, 8], [0, 2, 4, 99]):
        s = Step([2, 2, 4], 700, seed=15)
        s.cu = torch.tensor(cu, dtype=torch.int32)
        say("verify, rows", cu)
        assert s.run()[2] == dfc.ECORRUPT
    # rows of no request
    s = Step([2, 2, 4], 700, seed=16)
    s.cu = torch.tensor([1, 3, 3, 7], dtype=torch.int32)
    s.counts = [2, 0, 4]
    got = s.run()
    assert got[2] == 0
    s.check(got)
    s = Step([], 700)
    assert s.run() == ([], [], 0)
    s = Step([0, 0], 700)
    assert s.run() == ([0, 0], [-1, -1], 0)


def test_workspace_results_streams_and_repeats():
    s = Step([6] * 12 + [1, 0], 5000, torch.bfloat16, seed=17)
    first = s.run()
    s.check(first)
    dev = s.store.cuda()
    size = dfc.verify_drafts_workspace(dev[0], s.cu, dev[1])
    i64 = dict(dtype=torch.int64, device="cuda")
    out = dfc.Verified(torch.full((14,), -5, dtype=torch.int32, device="cuda"), torch.full((14,), -5, **i64))
    for fill in (0, 255):
        work = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        versions = [t._version for t in (work, *out)]
        assert s.run(workspace=work, out=out) == first
        assert [t._version for t in (work, *out)] == [v + 1 for v in versions]
    with pytest.raises(dfc.DfcError) as e:
        s.run(workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == dfc.ESIZE
    # two calls at once, each with its own workspace
    other = Step([3] * 20, 4000, seed=18)
    side = torch.cuda.Stream()
    want = other.run()
    args = [(t.store.cuda(), t.cu.cuda(), t.x.cuda(), t.u.cuda(), t.t.cuda()) for t in (s, other)]
    torch.cuda.synchronize()
    for _ in range(5):
        results = []
        for (store, cu, x, u, t), stream in zip(args, (None, side.cuda_stream)):
            results.append(dfc.verify_drafts(store[0], cu, x, u, draft_logits=store[1], temperature=t, stream=stream))
        torch.cuda.synchronize()
        assert [(v.accepted.tolist(), v.tokens.tolist()) for v in results] == [first[:2], want[:2]]


def test_refusals():
    s = Step([3, 1], 900, seed=19)
    z, d, cu, x, u, t = s.store[0].cuda(), s.store[1].cuda(), s.cu.cuda(), s.x.cuda(), s.u.cuda(), s.t.cuda()
    for bad in (lambda: dfc.verify_drafts(z.double(), cu, x, u), lambda: dfc.verify_drafts(z[0], cu, x, u),
                lambda: dfc.verify_drafts(z, cu.long(), x, u), lambda: dfc.verify_drafts(z, cu, x.int(), u),
                lambda: dfc.verify_drafts(z, cu, x, u.double()), lambda: dfc.verify_drafts(z, cu, x.cpu(), u),
                lambda: dfc.verify_drafts(z, cu, x, u, draft_logits=d.half()),
                lambda: dfc.verify_drafts(z, cu, x, u, temperature=t.double()),
                lambda: dfc.verify_drafts(z, cu, x, u, temperature=0.7),
                lambda: dfc.verify_drafts(z, cu[:0], x, u), lambda: dfc.verify_drafts(z, cu, x, u, out=(x,)),
                lambda: dfc.verify_drafts(z, cu, x, u, workspace=torch.empty(9))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dfc.verify_drafts(z, cu, x[:3], u), lambda: dfc.verify_drafts(z, cu, x, u[:3]),
                lambda: dfc.verify_drafts(z, cu, x, u, draft_logits=d[:3]),
                lambda: dfc.verify_drafts(z, cu, x, u, temperature=t[:1]),
                lambda: dfc.verify_drafts(z.t().contiguous().t(), cu, x, u),
                lambda: dfc.verify_drafts(z.clone().requires_grad_(), cu, x, u)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dfc.DfcError) as e:
        dfc.verify_drafts(z[:1].expand(4, 900), cu, x, u)     # rows that overlap
    assert e.value.status == dfc.EINVAL
    with pytest.raises(dfc.DfcError) as e:
        dfc.verify_drafts(z[:, :0], cu, x, u)
    assert e.value.status == dfc.EUNSUPPORTED
