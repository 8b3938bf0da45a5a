"""GPU: pages of the cache given back, shared, made dense and copied
(dfc_paged_release, dfc_paged_fork, dfc_paged_compact, dfc_paged_copy) against
the oracle's loops.  All of it is whole numbers and copied values: equal."""
import sys

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


class Pool:
    """Requests whose rows hold random pages, some of them shared, and a ring
    of the pages that nobody holds."""

    def __init__(self, lens, page, seed=0, share=0.0, spare=9, ring=None, reserve=0, width=None):
        rng = np.random.default_rng(seed)
        self.page, self.lens = page, list(lens)
        need = [-(-n // page) for n in lens]
        width = max(need + [1]) + 2 if width is None else width
        n = max(sum(need) + spare + reserve, 1)
        perm = rng.permutation(n)
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for r, k in enumerate(need):
            self.table[r, :k] = perm[at: at + k]
            at += k
            if r and rng.random() < share:
                p = rng.integers(0, r)
                m = rng.integers(0, min(self.lens[p], self.lens[r]) // page + 1)
                self.table[r, :m] = self.table[p, :m]
        holders = np.zeros(n, np.int64)
        for r, k in enumerate(need):
            for p in self.table[r, :k]:
                holders[p] += 1
        self.shared = np.maximum(holders - 1, 0).astype(np.int32)
        free = [p for p in perm if holders[p] == 0][reserve:]
        size = n + 3 if ring is None else max(ring, len(free))
        head = int(rng.integers(0, 5 * size))
        self.ring = np.full(size, -9, np.int32)
        for i, p in enumerate(free):
            self.ring[(head + i) % size] = p
        self.cursor = np.array([head, head + len(free)], np.int64)

    def on_device(self):
        return dev(self.table), dev(self.ring), dev(self.cursor, torch.int64), dev(self.shared)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def same(got, want):
    for i, (g, w) in enumerate(zip(got, want)):
        assert np.array_equal(g.cpu().numpy(), w), i


# ---------------------------------------------------------------- release

def release(pool, held, keep, window=0, sinks=0, **kw):
    table, ring, cursor, shared = pool.on_device()
    st = status()
    out = dfc.paged_release(dev(held), dev(keep), table, ring, cursor, shared, pool.page, window, sinks, status=st, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(cursor.cpu().numpy(), pool.cursor)
    return (table, ring, out, shared), int(st.item())


@pytest.mark.parametrize("page", [1, 4, 16, 64])
@pytest.mark.parametrize("requests,longest", [(1, 5), (3, 100), (64, 300), (700, 40), (5, 9000)])
@pytest.mark.parametrize("share", [0.0, 0.6])
def test_release(requests, longest, page, share):
    rng = np.random.default_rng(requests + page)
    held = rng.integers(0, longest + 1, requests)
    pool = Pool(held, page, seed=requests, share=share)
    # ended, cut at a page's end or to a length that leaves the shared part, kept
    keep = [h if c == 0 else 0 if c == 1 else max(0, h - int(x)) // page * page if c == 2 else h
            for h, c, x in zip(map(int, held), rng.integers(0, 4, requests), rng.integers(0, 2 * page + 1, requests))]
    for window, sinks in ((0, 0), (7, 0), (50, 5), (20, 64), (1, 1)):
        say("release", requests, longest, page, share, window, sinks)
        got, st = release(pool, held, keep, window, sinks)
        *want, cut = op.release(held, keep, pool.table, pool.ring, pool.cursor, pool.shared, page, window, sinks)
        assert st == 0 and cut == []
        same(got, want)


def test_release_again_and_again():
    # a window that moves on over lengths that grow, then the end
    pool = Pool([200, 90, 33], 8, seed=3)
    table, ring, cursor, shared = pool.on_device()
    want = [pool.table, pool.ring, pool.cursor, pool.shared]
    st = status()
    for cut in (0, 0, 3, 200):
        keep = [max(0, n - cut) for n in pool.lens]
        say("release again", cut)
        cursor = dfc.paged_release(dev(pool.lens), dev(keep), table, ring, cursor, shared, 8, 24, 4, status=st)
        *want, _ = op.release(pool.lens, keep, *want, 8, 24, 4)
        torch.cuda.synchronize()
        same((table, ring, cursor, shared), want)
        pool.lens = keep
    assert int(st.item()) == 0 and int(cursor[1] - cursor[0]) == len(pool.shared)


@pytest.mark.parametrize("n_pages", [1, 1023, 8192, 8193, 100003, 8192 * 1024 + 5])
def test_release_of_scattered_pages_of_large_caches(n_pages):
    rng = np.random.default_rng(n_pages)
    held = np.unique(rng.integers(0, n_pages, min(n_pages, 5000)))
    rng.shuffle(held)
    table = dev(held[None])
    ring = torch.full((n_pages + 2,), -9, dtype=torch.int32, device="cuda")
    shared = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    cursor = torch.tensor([n_pages, n_pages], device="cuda")
    st = status()
    say("release of", n_pages)
    out = dfc.paged_release(dev([len(held) * 4]), dev([0]), table, ring, cursor, shared, 4, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and out.tolist() == [n_pages, n_pages + len(held)]
    assert (table == -1).all() and not shared.any()
    at = (n_pages + np.arange(len(held))) % (n_pages + 2)
    got = ring.cpu().numpy()
    assert np.array_equal(got[at], np.sort(held)) and (np.delete(got, at) == -9).all()


def test_release_of_pages_held_by_all():
    # 300 requests share 40 pages and all give them up at once, or all but one
    table = np.tile(np.arange(40, dtype=np.int32)[::-1], (300, 1))
    pool = Pool([160] * 300, 4, seed=1)
    pool.table, pool.shared = table, np.full(50, 299, np.int32)
    pool.shared[40:] = 0
    pool.ring, pool.cursor = np.full(64, -9, np.int32), np.array([5, 5], np.int64)
    for keep in ([0] * 300, [0] * 299 + [160], [80] * 300):
        got, st = release(pool, [160] * 300, keep)
        *want, _ = op.release([160] * 300, keep, pool.table, pool.ring, pool.cursor, pool.shared, 4)
        assert st == 0
        same(got, want)


@pytest.mark.parametrize("requests,longest,page", [(1, 5000, 1), (64, 1000, 1), (64, 8191, 16), (40, 1600, 1), (65, 900, 2)])
def test_release_of_all_that_few_requests_hold(requests, longest, page):
    # up to 64 requests are one workgroup's work, whose pages are bits in LDS
    rng = np.random.default_rng(requests)
    held = rng.integers(0, longest + 1, requests)
    pool = Pool(held, page, seed=requests, share=0.5)
    for keep in ([0] * requests, [0 if r % 3 else int(h) for r, h in enumerate(held)],
                 [int(h) // page * page // 2 // page * page if r % 2 else int(h) for r, h in enumerate(held)]):
        for window, sinks in ((0, 0), (100, 9)):
            say("release of few", requests, longest, page, window)
            got, st = release(pool, held, keep, window, sinks)
            *want, cut = op.release(held, keep, pool.table, pool.ring, pool.cursor, pool.shared, page, window, sinks)
            assert st == 0 and cut == []
            same(got, want)


def test_release_without_requests():
    e, c = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.tensor([3, 5], device="cuda")
    ring, shared = torch.arange(6, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    out = dfc.paged_release(e, e, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), ring, c, shared, 16)
    assert out.tolist() == [3, 5] and ring.tolist() == [0, 1, 2, 3, 4, 5]


def test_release_inputs_that_make_no_sense():
    pool = Pool([40, 40, 40], 16, seed=5)
    # negative lengths and more than is held: passed over
    for held, keep in (([-1, 40, 40], [0, 40, 40]), ([40, 40, 40], [-2, 40, 40]), ([40, 40, 40], [41, 40, 40])):
        got, st = release(pool, held, keep)
        assert st == dfc.ECORRUPT
        same(got, (pool.table, pool.ring, pool.cursor, pool.shared))
    # more than a row holds: its entries are given up
    got, st = release(pool, [40, 40, 16 * 5 + 1], [40, 40, 0])
    assert st == dfc.ESIZE and (got[0][2] < 0).all()
    # pages that are none
    pool.table[0, 1] = 10 ** 6
    got, st = release(pool, [40, 40, 40], [0, 40, 40])
    assert st == dfc.ECORRUPT and (got[0][0, :3] == -1).all() and int(got[2][1]) == pool.cursor[1] + 2
    pool = Pool([40, 40, 40], 16, seed=5)
    # a page that two requests hold and no count knows of: free once
    pool.table[1, 0] = pool.table[0, 0]
    got, st = release(pool, [40, 40, 40], [0, 0, 40])
    assert st == dfc.ECORRUPT and int(got[2][1]) == pool.cursor[1] + 5 and not got[3].any()
    # a ring without room, and a cursor that does not fit
    for cursor in ([7, 7 + len(pool.ring) - 2], [9, 8], [-1, 3], [0, len(pool.ring) + 1]):
        pool = Pool([40, 40, 40], 16, seed=5)
        pool.cursor = np.array(cursor, np.int64)
        got, st = release(pool, [40, 40, 40], [0, 40, 40])
        assert st == dfc.ECORRUPT and got[2].tolist() == cursor
        same(got[1:2], [pool.ring])
    # cut inside a page that another holds
    pool = Pool([40, 40], 16, seed=6)
    pool.table[1, :2] = pool.table[0, :2]
    pool.shared[pool.table[0, :2]] = 1
    got, st = release(pool, [40, 40], [20, 40])
    assert st == dfc.EUNSUPPORTED
    *want, cut = op.release([40, 40], [20, 40], pool.table, pool.ring, pool.cursor, pool.shared, 16)
    assert cut == [0]
    same(got, want)
    got, st = release(pool, [40, 40], [20, 0])   # the other ends meanwhile
    assert st == 0


def test_release_of_many_requests_that_make_no_sense():
    # the same by several launches: 70 requests more, that hold nothing
    more = [0] * 70

    def go(pool, held, keep):
        return release(pool, held + more, keep + more)

    pool = Pool([40, 40, 40] + more, 16, seed=5)
    for held, keep in (([-1, 40, 40], [0, 40, 40]), ([40, 40, 40], [-2, 40, 40]), ([40, 40, 40], [41, 40, 40])):
        got, st = go(pool, held, keep)
        assert st == dfc.ECORRUPT
        same(got, (pool.table, pool.ring, pool.cursor, pool.shared))
    got, st = go(pool, [40, 40, 16 * 5 + 1], [40, 40, 0])
    assert st == dfc.ESIZE and (got[0][2] < 0).all()
    pool.table[0, 1] = 10 ** 6
    got, st = go(pool, [40, 40, 40], [0, 40, 40])
    assert st == dfc.ECORRUPT and (got[0][0, :3] == -1).all() and int(got[2][1]) == pool.cursor[1] + 2
    pool = Pool([40, 40, 40] + more, 16, seed=5)
    pool.table[1, 0] = pool.table[0, 0]
    got, st = go(pool, [40, 40, 40], [0, 0, 40])
    assert st == dfc.ECORRUPT and int(got[2][1]) == pool.cursor[1] + 5 and not got[3].any()
    for cursor in ([7, 7 + len(pool.ring) - 2], [9, 8], [-1, 3], [0, len(pool.ring) + 1]):
        pool = Pool([40, 40, 40] + more, 16, seed=5)
        pool.cursor = np.array(cursor, np.int64)
        got, st = go(pool, [40, 40, 40], [0, 40, 40])
        assert st == dfc.ECORRUPT and got[2].tolist() == cursor
        same(got[1:2], [pool.ring])
    pool = Pool([40, 40] + more, 16, seed=6)
    pool.table[1, :2] = pool.table[0, :2]
    pool.shared[pool.table[0, :2]] = 1
    got, st = go(pool, [40, 40], [20, 40])
    assert st == dfc.EUNSUPPORTED
    *want, cut = op.release([40, 40] + more, [20, 40] + more, pool.table, pool.ring, pool.cursor, pool.shared, 16)
    assert cut == [0]
    same(got, want)
    got, st = go(pool, [40, 40], [20, 0])
    assert st == 0


def test_release_refusals_and_results():
    pool = Pool([40, 20], 16, seed=7)
    table, ring, cursor, shared = pool.on_device()
    h, k = dev([40, 20]), dev([0, 20])
    with pytest.raises(TypeError):
        dfc.paged_release(h.long(), k, table, ring, cursor, shared, 16)
    with pytest.raises(ValueError):
        dfc.paged_release(h, k[:1], table, ring, cursor, shared, 16)
    with pytest.raises(ValueError):
        dfc.paged_release(h, k, table[:1], ring, cursor, shared, 16)
    with pytest.raises(TypeError):
        dfc.paged_release(h, k, table, ring, cursor.int(), shared, 16)
    with pytest.raises(TypeError):
        dfc.paged_release(h, k, table, ring, cursor, shared.long(), 16)
    with pytest.raises(ValueError):
        dfc.paged_release(h, k, table, ring, cursor, shared, 16, window=-1)
    for kw in (dict(page_size=24), dict(page_size=16, out=cursor), dict(page_size=16, shared=shared[:0])):
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_release(h, k, table, ring, cursor, kw.pop("shared", shared), kw.pop("page_size"), **kw)
        assert e.value.status == dfc.EINVAL
    same((table, ring, cursor, shared), (pool.table, pool.ring, pool.cursor, pool.shared))
    out = torch.zeros(2, dtype=torch.int64, device="cuda")
    versions = [t._version for t in (table, ring, shared, out)]
    assert dfc.paged_release(h, k, table, ring, cursor, shared, 16, out=out) is out
    assert [t._version for t in (table, ring, shared, out)] == [v + 1 for v in versions]
    assert out.tolist() == [pool.cursor[0], pool.cursor[1] + 3]


# ------------------------------------------------------------------- fork

def fork(pool, context, parents, lens=None):
    table, ring, cursor, shared = pool.on_device()
    st = status()
    f = dfc.paged_fork(dev(context), dev(parents), table, ring, cursor, shared, pool.page,
                       fork_lens=None if lens is None else dev(lens), status=st)
    torch.cuda.synchronize()
    assert np.array_equal(cursor.cpu().numpy(), pool.cursor) and np.array_equal(ring.cpu().numpy(), pool.ring)
    return (f.context_lens, table, shared, f.cursor, f.src, f.dst), int(st.item())


@pytest.mark.parametrize("page", [1, 4, 16, 128])
@pytest.mark.parametrize("parents,children,longest", [(1, 1, 1), (1, 7, 300), (3, 40, 90), (16, 700, 33), (300, 5, 60),
                                                      (2, 3, 9000)])
def test_fork(parents, children, longest, page):
    rng = np.random.default_rng(parents * children + page)
    held = rng.integers(1, longest + 1, parents)
    held[0] = longest
    lens = np.concatenate([held, np.zeros(children, int)])
    pool = Pool(lens, page, seed=parents, share=0.4, spare=children + 2)
    who = np.array([-1] * parents + [int(x) for x in rng.integers(-1, parents, children)])
    order = rng.permutation(len(lens))   # children stand among their parents
    place = np.argsort(order)
    pool.table, lens = pool.table[order], lens[order]
    who = np.array([-1 if p < 0 else place[p] for p in who[order]])
    some = np.array([0 if p < 0 else int(rng.integers(0, lens[p] + 1)) for p in who])
    for prefix in (None, some):
        say("fork", parents, children, longest, page, prefix is not None)
        got, st = fork(pool, lens, who, prefix)
        want = op.fork(lens, who, pool.table, pool.ring, pool.cursor, pool.shared, page, prefix)
        assert st == 0
        same(got, want)


def test_fork_of_a_request_behind_a_window():
    pool = Pool([100, 0], 8, seed=2)
    pool.table[0, 1:9] = -1
    got, st = fork(pool, [100, 0], [-1, 0])
    assert st == 0
    same(got, op.fork([100, 0], [-1, 0], pool.table, pool.ring, pool.cursor, pool.shared, 8))
    # a prefix that ends in a page given back cannot be copied
    got, st = fork(pool, [100, 0], [-1, 0], [0, 20])
    assert st == dfc.ECORRUPT and got[0].tolist() == [100, 0]
    same(got[1:4], (pool.table, pool.shared, pool.cursor))


def test_fork_runs_out_of_pages():
    pool = Pool([21, 0, 0, 16, 0, 0], 8, seed=3, spare=2)
    pool.cursor[0] = pool.cursor[1] - 2
    got, st = fork(pool, [21, 0, 0, 16, 0, 0], [-1, 0, 0, -1, 3, 0])
    assert st == dfc.ESIZE and got[0].tolist() == [21, 21, 21, 16, 16, 0]
    assert got[3].tolist() == [pool.cursor[1], pool.cursor[1]]
    want = op.fork([21, 0, 0, 16, 0, 0], [-1, 0, 0, -1, 3, -1], pool.table, pool.ring, pool.cursor, pool.shared, 8)
    same(got, want)


def test_fork_inputs_that_make_no_sense():
    pool = Pool([40, 0, 30, 0], 16, seed=4)
    same_as_before = lambda got: same(got[1:4], (pool.table, pool.shared, pool.cursor))
    for parents, context, lens in (([-1, 4, -1, -1], [40, 0, 30, 0], None), ([-1, -2, -1, -1], [40, 0, 30, 0], None),
                                   ([-1, 1, -1, -1], [40, 0, 30, 0], None), ([2, -1, -1, -1], [40, 0, 30, 0], None),
                                   ([-1, 0, -1, -1], [40, 0, 30, 0], [0, 41, 0, 0]),
                                   ([-1, 0, -1, -1], [40, 0, 30, 0], [0, -1, 0, 0])):
        got, st = fork(pool, context, parents, lens)
        assert st == dfc.ECORRUPT and got[0].tolist() == context
        assert (got[4] == -1).all() and (got[5] == -1).all()
        same_as_before(got)
    # a parent that is forked itself: only the other one is
    got, st = fork(pool, [40, 0, 30, 0], [-1, 0, -1, 1])
    assert st == dfc.ECORRUPT and got[0].tolist() == [40, 40, 30, 0]
    # a cursor that does not fit, a page on the ring that is none
    good = pool.cursor.copy()
    pool.cursor[1] = pool.cursor[0] - 1
    got, st = fork(pool, [40, 0, 30, 0], [-1, 0, -1, -1])
    assert st & 0xFFFFFFFF == (dfc.ECORRUPT | dfc.ESIZE) & 0xFFFFFFFF and got[0].tolist() == [40, 0, 30, 0]
    pool.cursor = good
    pool.ring[good[0] % len(pool.ring)] = 10 ** 6
    got, st = fork(pool, [40, 0, 30, 0], [-1, 0, -1, -1])
    assert st == dfc.ECORRUPT and got[0].tolist() == [40, 0, 30, 0] and (got[5] == -1).all()
    same(got[1:3], (pool.table, pool.shared))
    # more than a row holds
    pool = Pool([40, 0], 16, seed=4, width=3)
    got, st = fork(pool, [49, 0], [-1, 0])
    assert st == dfc.ESIZE and got[0].tolist() == [49, 0]
    # an entry past the cache
    pool.table[0, 0] = 999
    got, st = fork(pool, [40, 0], [-1, 0])
    assert st == dfc.ECORRUPT and got[0].tolist() == [40, 40] and got[1][1, 0] == -1


def test_fork_refusals_and_results():
    pool = Pool([40, 0], 16, seed=7)
    table, ring, cursor, shared = pool.on_device()
    c, p = dev([40, 0]), dev([-1, 0])
    with pytest.raises(TypeError):
        dfc.paged_fork(c, p.long(), table, ring, cursor, shared, 16)
    with pytest.raises(ValueError):
        dfc.paged_fork(c, p[:1], table, ring, cursor, shared, 16)
    with pytest.raises(ValueError):
        dfc.paged_fork(c, p, table, ring, cursor, shared, 16, fork_lens=p[:1])
    with pytest.raises(TypeError):
        dfc.paged_fork(c, p, table, ring, cursor, shared, 16, out=(c, p))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = dfc.PagedFork(torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32),
                        torch.zeros(2, dtype=torch.int64, device="cuda"))
    for bad in (out._replace(cursor=cursor), out._replace(context_lens=c), out._replace(src=p),
                out._replace(dst=out.src)):
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_fork(c, p, table, ring, cursor, shared, 16, out=bad)
        assert e.value.status == dfc.EINVAL
    same((table, ring, cursor, shared), (pool.table, pool.ring, pool.cursor, pool.shared))
    versions = [t._version for t in (table, shared, *out)]
    assert dfc.paged_fork(c, p, table, ring, cursor, shared, 16, out=out) is out
    assert [t._version for t in (table, shared, *out)] == [v + 1 for v in versions]
    same((out.context_lens, table, shared, out.cursor, out.src, out.dst),
         op.fork([40, 0], [-1, 0], pool.table, pool.ring, pool.cursor, pool.shared, 16))
    e = torch.zeros(0, **i32)
    f = dfc.paged_fork(e, e, torch.zeros(0, 4, **i32), ring, cursor, shared, 16)
    assert torch.equal(f.cursor, cursor) and f.src.numel() == 0


# ---------------------------------------------------------------- compact

def compact(pool, context):
    table, ring, cursor, shared = pool.on_device()
    st = status()
    m = dfc.paged_compact(dev(context), table, ring, cursor, shared, pool.page, status=st)
    torch.cuda.synchronize()
    assert np.array_equal(cursor.cpu().numpy(), pool.cursor)
    held = {int(p) for r, c in enumerate(context) for p in pool.table[r, : -(-max(int(c), 0) // pool.page)]
            if 0 <= p < len(pool.shared)}
    assert int(m.used) == len(held)
    return (table, ring, shared, m.src, m.dst), int(st.item())


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("requests,longest,spare,reserve", [(1, 1, 0, 0), (1, 5, 1, 0), (3, 100, 30, 0), (64, 300, 9, 5),
                                                            (64, 30, 5000, 11), (700, 40, 300, 0), (300, 900, 20000, 7),
                                                            (1025, 9, 100, 3), (30, 4000, 500, 0), (2, 8100, 1, 0)])
@pytest.mark.parametrize("share", [0.0, 0.6])
def test_compact(requests, longest, spare, reserve, page, share):
    rng = np.random.default_rng(requests + spare + page)
    lens = rng.integers(0, longest + 1, requests)
    pool = Pool(lens, page, seed=requests, share=share, spare=spare, reserve=reserve)
    pool.table[::3, 1:3] = np.where(pool.table[::3, 1:3] >= 0, -1, pool.table[::3, 1:3])  # given back behind a window
    held = [p for r, n in enumerate(lens) for p in pool.table[r, : -(-int(n) // page)] if p >= 0]
    pool.shared = np.maximum(np.bincount(np.array(held, int), minlength=len(pool.shared)) - 1, 0).astype(np.int32)
    say("compact", requests, longest, spare, reserve, page, share)
    got, st = compact(pool, lens)
    assert st == 0
    same(got, op.compact(lens, pool.table, pool.ring, pool.cursor, pool.shared, page))


def test_compact_without_requests():
    e, cursor = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.tensor([4, 8], device="cuda")
    for width in (0, 5):
        ring, shared = dev([9, 2, 7, -1, 0]), dev([0] * 10)
        m = dfc.paged_compact(e, torch.zeros(0, width, dtype=torch.int32, device="cuda"), ring, cursor, shared, 16)
        # the ring in ascending order from its head on
        assert ring.tolist() == [2, 7, 9, -1, 0]
        assert m.src.tolist() == [-1] * 5 and m.dst.tolist() == [-1] * 5 and m.used.tolist() == [0]


def test_compact_where_nothing_moves():
    for lens, spare in (([0, 0], 20), ([100, 50], 0)):
        pool = Pool(lens, 4, seed=1, spare=spare)
        got, st = compact(pool, lens)
        assert st == 0 and (got[3] == -1).all() and (got[4] == -1).all()
        same(got, op.compact(lens, pool.table, pool.ring, pool.cursor, pool.shared, 4))
    again, st = compact(pool, lens)
    same(again, [g.cpu().numpy() for g in got])


@pytest.mark.parametrize("spare", [30, 20000])  # by one workgroup, by several launches
def test_compact_where_ring_and_tables_contradict(spare):
    lens = [100, 50]
    for spoil in ("twice on the ring", "held and on the ring", "past the cache", "negative", "cursor", "held past"):
        pool = Pool(lens, 4, seed=2, spare=spare)
        n, head = len(pool.ring), int(pool.cursor[0])
        if spoil == "twice on the ring":
            pool.ring[(head + 5) % n] = pool.ring[(head + 2) % n]
        elif spoil == "held and on the ring":
            pool.ring[(head + 5) % n] = pool.table[1, 0]
        elif spoil == "past the cache":
            pool.ring[(head + 5) % n] = len(pool.shared)
        elif spoil == "negative":
            pool.ring[(head + 5) % n] = -1
        elif spoil == "cursor":
            pool.cursor[1] = head + n + 1
        else:
            pool.table[1, 0] = len(pool.shared)
        say("compact,", spoil)
        got, st = compact(pool, lens)
        assert st == dfc.ECORRUPT, spoil
        same(got[:3], (pool.table, pool.ring, pool.shared))
        assert (got[3] == -1).all() and (got[4] == -1).all()
    pool = Pool(lens, 4, seed=2, spare=spare)
    got, st = compact(pool, [100, 4 * pool.table.shape[1] + 1])   # past the row, whose rest is no page
    assert st == dfc.ESIZE
    same(got, op.compact(lens, pool.table, pool.ring, pool.cursor, pool.shared, 4))
    got, st = compact(pool, [100, -5])
    assert st == dfc.ECORRUPT


def test_compact_refusals_and_results():
    pool = Pool([40, 20], 16, seed=7)
    table, ring, cursor, shared = pool.on_device()
    c = dev([40, 20])
    with pytest.raises(TypeError):
        dfc.paged_compact(c.long(), table, ring, cursor, shared, 16)
    with pytest.raises(ValueError):
        dfc.paged_compact(c[:1], table, ring, cursor, shared, 16)
    half = len(pool.shared) // 2
    i32 = dict(dtype=torch.int32, device="cuda")
    out = dfc.PagedMoves(torch.zeros(half, **i32), torch.zeros(half, **i32), torch.zeros(1, **i32))
    with pytest.raises(ValueError):
        dfc.paged_compact(c, table, ring, cursor, shared, 16, out=out._replace(src=out.src[:-1]))
    for kw in (dict(page_size=24), dict(page_size=16, out=out._replace(dst=out.src))):
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_compact(c, table, ring, cursor, shared, **kw)
        assert e.value.status == dfc.EINVAL
    same((table, ring, cursor, shared), (pool.table, pool.ring, pool.cursor, pool.shared))
    versions = [t._version for t in (table, ring, shared, *out)]
    assert dfc.paged_compact(c, table, ring, cursor, shared, 16, out=out) is out
    assert [t._version for t in (table, ring, shared, *out)] == [v + 1 for v in versions]
    same((table, ring, shared, out.src, out.dst),
         op.compact([40, 20], pool.table, pool.ring, pool.cursor, pool.shared, 16))


# ------------------------------------------------------------------- copy

@pytest.mark.parametrize("pages,page,heads,dim,layers,pairs", [(9, 16, 8, 128, 3, 4), (50, 1, 1, 8, 1, 25),
                                                               (40, 4, 3, 24, 70, 17), (3000, 2, 2, 64, 2, 1400),
                                                               (12, 64, 5, 256, 5, 6)])
@pytest.mark.parametrize("order", ["phd", "hpd", "apart"])
def test_copy(pages, page, heads, dim, layers, pairs, order):
    g = torch.Generator(device="cuda").manual_seed(pages)
    shape = {"phd": (layers, 2, pages, page, heads, dim), "hpd": (layers, 2, pages, heads, page, dim),
             "apart": (layers, 2, pages, page, heads, dim + 8)}[order]
    cache = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    view = cache.transpose(3, 4) if order == "hpd" else cache[..., :dim]
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    src, dst = perm[:pairs].clone(), perm[pairs: 2 * pairs].clone()
    src[1::5], dst[3::7] = -1, -1     # pairs that are none
    want = cache.clone()
    there = (src >= 0) & (dst >= 0)
    want.view(torch.int16)[:, :, dst[there].long(), ..., :dim] = cache.view(torch.int16)[:, :, src[there].long(), ..., :dim]
    st = status()
    say("copy", pages, page, heads, dim, layers, pairs, order)
    dfc.paged_copy([(c[0], c[1]) for c in view], src, dst, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(cache.view(torch.int16), want.view(torch.int16))


def test_copy_with_layouts_of_k_and_v_that_differ():
    k = torch.randn(8, 16, 2, 64, device="cuda").half()
    v = torch.randn(8, 2, 16, 64, device="cuda").half().transpose(1, 2)
    want = k.clone(), v.clone()
    for w in want:
        w[5] = w[2]
    dfc.paged_copy([(k, v)], dev([-1, 2]), dev([0, 5]))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_copy_of_a_list_that_is_filled_in_front():
    # as compacting a large cache gives: few pairs of many places
    cache = torch.randn(2, 2, 4000, 1, 1, 8, device="cuda").bfloat16()
    src = torch.full((200000,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[:1500], dst[:1500] = torch.arange(2000, 3500, device="cuda"), torch.arange(1500, device="cuda")
    want = cache.clone()
    want[:, :, :1500] = cache[:, :, 2000:3500]
    say("copy, long list")
    dfc.paged_copy([(c[0], c[1]) for c in cache], src, dst)
    torch.cuda.synchronize()
    assert torch.equal(cache, want)


def test_copy_past_2_to_the_32_bytes():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("too little memory")
    cache = torch.zeros(1100000, 16, 2, 64, dtype=torch.bfloat16, device="cuda")   # 4.5 GB each of K and V
    other = torch.zeros_like(cache)
    cache[1099999], other[1099998] = 3.0, 5.0
    say("copy past 4 GiB")
    dfc.paged_copy([(cache, other)], dev([1099999, 1099998]), dev([1, 1099990]))
    torch.cuda.synchronize()
    assert (cache[1] == 3).all() and (other[1099990] == 5).all() and not cache[2:1099990].any()


def test_copy_where_a_pages_rows_lie_past_2_to_the_36_bytes():
    # tokens of a page outside the pages: 4 x 1.6e6 pages of 14 KB
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("too little memory")
    pages, heads, dim = 1600000, 28, 256
    cache = torch.empty(4, pages, heads, dim, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert cache.stride(1) * 3 // 8 > 2 ** 32 > cache.stride(1) // 8
    for i in range(4):
        cache[pages - 2, i], cache[1, i] = i + 1, -1
    say("copy, rows far apart")
    dfc.paged_copy([(cache, cache)], dev([pages - 2]), dev([1]))
    torch.cuda.synchronize()
    assert all((cache[p, i] == i + 1).all() for p in (1, pages - 2) for i in range(4))
    del cache
    torch.cuda.empty_cache()


def test_copy_inputs_that_make_no_sense_and_refusals():
    k, v = (torch.randn(8, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
    want = k.clone()
    st = status()
    dfc.paged_copy([(k, v)], dev([8, 2, 1]), dev([0, 8, -5]), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == dfc.ECORRUPT and torch.equal(k, want)
    dfc.paged_copy([], dev([1]), dev([2]))
    dfc.paged_copy([(k, v)], dev([]), dev([]))
    for caches in (3, [k], [(k,)], [(k, v, v)], [(k, v.half())], [(k, v.cpu())], [(k, v[:4])], [(k, "v")]):
        with pytest.raises(TypeError):
            dfc.paged_copy(caches, dev([1]), dev([2]))
    with pytest.raises(ValueError):
        dfc.paged_copy([(k, v)], dev([1]), dev([2, 3]))
    with pytest.raises(TypeError):
        dfc.paged_copy([(k, v)], dev([1]).long(), dev([2]))
    with pytest.raises(ValueError, match="gradient"):
        dfc.paged_copy([(k, v.clone().requires_grad_())], dev([1]), dev([2]))
    with pytest.raises(dfc.DfcError):
        dfc.paged_copy([(k, v), (k[:4], v[:4])], dev([1]), dev([2]))
    one = dev([1])
    with pytest.raises(dfc.DfcError):
        dfc.paged_copy([(k, v)], one, one)
    assert torch.equal(k, want)
    versions = k._version, v._version
    dfc.paged_copy([(k, v)], dev([1]), dev([2]))
    assert (k._version, v._version) == (versions[0] + 1, versions[1] + 1)
