"""GPU: the paged key/value cache (dfc_paged_plan, dfc_paged_append,
dfc_paged_attention) against the oracle's definitions in 64 bits.

Every cache starts as NaN, so a value that an operator should not have read
shows.  Bounds on the attention's error come from the formula: weights are
rounded to the cache's type once (relative u = 2^-8 for bfloat16, 2^-11 for
float16) and so is the output, scores accumulate dim products in fp32 and go
through one multiply-add and one exponential; the sums over N keys are in
fp32.  With A the largest sum of |scale q_i k_i| and Z the largest |score| of
a row, a weight and a sum are off by a factor of at most 1 + e,
e = 2^-23 (dim A + 2 Z + N + 16), and
|out - ref| <= (u + 2 e) sum_j w_j |v_j| + u |ref|; float16 weights below
2^-24 of their scaled range lose all bits, N 2^-32 max |v| at most."""
import sys

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def as64(t):
    return t.detach().cpu().double().numpy()


class Step:
    """Requests with `total` tokens of which `new` are the step's, their keys
    and values scattered over the pages of a cache that is NaN elsewhere."""

    def __init__(self, total, new, heads, kv_heads, dim, page, dtype, seed=0, extra_pages=0, order="phd"):
        g = torch.Generator().manual_seed(seed)
        self.total, self.new, self.page = total, new, page
        need = [-(-t // page) for t in total]
        width = max(need + [1]) + extra_pages
        n_pages = sum(need) + 2
        perm = torch.randperm(n_pages, generator=g)
        self.table = torch.full((len(total), width), -1, dtype=torch.int32)
        shape = (n_pages, page, kv_heads, dim)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
        at = 0
        for r, t in enumerate(total):
            self.table[r, : need[r]] = perm[at: at + need[r]].int()
            at += need[r]
            for c in (self.k, self.v):
                rows = torch.randn(t, kv_heads, dim, generator=g).to(dtype)
                for j in range(t):
                    c[self.table[r, j // page], j % page] = rows[j]
        self.q = (1.5 * torch.randn(sum(new), heads, dim, generator=g)).to(dtype)
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.lens = torch.tensor(total, dtype=torch.int32)
        self.order = order

    def cache(self, c):
        """On the device; order "hpd": heads outside the tokens of a page."""
        if self.order == "hpd":
            return c.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
        return c.cuda()

    def run(self, scale=None, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda")
        lse = torch.full(self.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        dfc.paged_attention(self.q.cuda(), self.cache(self.k), self.cache(self.v), self.table.cuda(), self.cu.cuda(),
                            self.lens.cuda(), scale=scale, out=out, lse=lse, status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return out, lse

    def check(self, out, lse, scale=None, causal=True, window=0, rows=None):
        """Every row against the definition, or the first `rows` rows of the
        first request."""
        dim = self.q.shape[2]
        scale = dim ** -0.5 if scale is None else scale
        u = U[self.q.dtype]
        got, got_lse, q = as64(out), as64(lse), as64(self.q)
        for r in range(len(self.total) if rows is None else 1):
            a, b = int(self.cu[r]), int(self.cu[r + 1])
            n = self.total[r]
            if a == b:
                continue
            if rows is not None:
                n -= b - rows
                b = rows
            k, v = (op.gather(as64(c), self.table[r].numpy(), self.page, n) for c in (self.k, self.v))
            ref, ref_lse, spread, top, mass = op.attention(q[a:b], k, v, scale, causal, window)
            e = 2.0 ** -23 * (dim * mass + 2 * top + n + 16)[..., None]
            lost = 2.0 ** -32 * n * np.abs(v).max(initial=0.0)
            bound = (u + 2 * e) * spread + u * np.abs(ref) + lost + 1e-30
            assert np.isfinite(got[a:b]).all(), r
            assert (np.abs(got[a:b] - ref) <= bound).all(), (r, np.abs(got[a:b] - ref).max())
            empty = np.isneginf(ref_lse)
            assert np.isneginf(got_lse[a:b][empty]).all() and (got[a:b][empty] == 0).all()
            diff = np.where(empty, 0, got_lse[a:b]) - np.where(empty, 0, ref_lse)
            assert (np.abs(diff) <= 4 * e[..., 0] + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, ref_lse)))).all(), r


CASES = [
    # total, new, heads, kv_heads, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([700], [1], 32, 8, 128, 16),
    ([1, 2, 31, 32, 33, 64, 65, 127, 300], [1] * 9, 8, 2, 128, 16),
    ([515, 64, 40], [5, 5, 5], 16, 4, 128, 32),
    ([130, 77], [130, 77], 8, 2, 128, 16),
    ([333], [129], 4, 4, 64, 16),
    ([190, 65, 300, 1], [67, 1, 1, 1], 6, 2, 80, 8),
    ([97, 200], [33, 1], 3, 1, 256, 64),
    ([260], [2], 64, 1, 256, 16),
    ([50, 129], [3, 40], 5, 5, 24, 4),
    ([70, 33], [70, 2], 4, 2, 128, 1),
    ([140], [1], 7, 1, 200, 256),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_against_the_definition(case, dtype):
    total, new, heads, kv_heads, dim, page = CASES[case]
    s = Step(total, new, heads, kv_heads, dim, page, dtype, seed=case)
    for hint in (0, max(new)):
        say("attention", case, dtype, "hint", hint)
        s.check(*s.run(max_q_len=hint))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_where_the_tables_are_wide(case):
    # room for far more tokens than there are: tiles may be split, here some
    # hundred tokens later too
    total, new, heads, kv_heads, dim, page = CASES[case]
    for more in (0, 900):
        s = Step([t + more for t in total], new, heads, kv_heads, dim, page, torch.bfloat16, seed=100 + case,
                 extra_pages=8192 // page)
        for hint in (0, max(new)):
            say("wide table", case, more, "hint", hint)
            s.check(*s.run(max_q_len=hint))


def check_rows(s, out, lse, window=0, r=0, rows=None):
    """Rows of request r one at a time against the definition (causal)."""
    a, n, total = int(s.cu[r]), s.new[r], s.total[r]
    k, v = (op.gather(as64(c), s.table[r].numpy(), s.page, total) for c in (s.k, s.v))
    dim, u = s.q.shape[2], U[s.q.dtype]
    q, got, got_lse = as64(s.q[a: a + n]), as64(out[a: a + n]), as64(lse[a: a + n])
    edges = [i for i in (0, 1, 7, 8, 15, 16, 31, 32, 63, 64, 65, n // 2, n - 65, n - 33, n - 2, n - 1) if 0 <= i < n]
    for i in sorted(set(edges if rows is None else rows)):
        m = total - n + i + 1
        lo = max(0, m - window) if window else 0
        ref, ref_lse, spread, top, mass = op.attention(q[i: i + 1], k[lo:m], v[lo:m], dim ** -0.5)
        e = 2.0 ** -23 * (dim * mass + 2 * top + (m - lo) + 16)[..., None]
        bound = (u + 2 * e) * spread + u * np.abs(ref) + 2.0 ** -32 * (m - lo) * np.abs(v).max()
        assert (np.abs(got[i] - ref[0]) <= bound[0]).all(), (i, np.abs(got[i] - ref[0]).max())
        assert (np.abs(got_lse[i] - ref_lse[0]) <= 4 * e[0, :, 0] + 2.0 ** -21 * (1 + np.abs(ref_lse[0]))).all(), i


# Steps large enough for the tallest tiles: a prompt, a chunk whose keys are
# split, chunks beside single tokens under a window, heads narrower than the
# registers' columns, pages smaller than a load's rows.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("total,new,heads,kv_heads,dim,page,window", [
    ([2051], [2051], 32, 8, 128, 16, 0),
    ([2050], [2049], 32, 8, 64, 64, 0),
    ([20000], [333], 16, 2, 128, 32, 0),
    ([4100, 1300, 1, 700], [1900, 1, 1, 500], 36, 12, 64, 16, 777),
    ([3000, 70], [2500, 70], 24, 8, 80, 2, 0),
])
def test_attention_of_large_steps(total, new, heads, kv_heads, dim, page, window, dtype):
    s = Step(total, new, heads, kv_heads, dim, page, dtype, seed=sum(total))
    say("large step", total, new, dtype)
    out, lse = s.run(window=window, max_q_len=max(new))
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for r in range(len(total)):
        check_rows(s, out, lse, window, r)


def test_large_step_without_the_causal_mask():
    s = Step([2100], [2080], 32, 8, 64, 16, torch.bfloat16, seed=20)
    say("large step, not causal")
    out, lse = s.run(causal=False)
    keep, s.new, s.q = s.new, [40], s.q[[*range(8), *range(1000, 1024), *range(2072, 2080)]]
    rows = [*range(8), *range(1000, 1024), *range(2072, 2080)]
    s.cu = torch.tensor([0, 40], dtype=torch.int32)
    s.check(out[rows], lse[rows], causal=False)
    assert keep == [2080]


def test_large_step_with_values_that_are_not_finite_in_masked_places():
    s = Step([2100], [2080], 32, 8, 128, 16, torch.bfloat16, seed=21)
    clean = s.run()
    tok = 1000   # position 1000: row 980
    s.v[s.table[0, tok // 16], tok % 16, 0, 5] = float("inf")
    s.k[s.table[0, tok // 16], tok % 16, 1, 7] = float("nan")
    say("large step, not finite")
    out, lse = s.run()
    assert torch.isfinite(out[:980].float()).all() and torch.isfinite(lse[:980]).all()
    check_rows(s, out, lse, rows=[0, 600, 900, 950, 970, 979])
    assert torch.isposinf(out[980:, :4, 5].float()).all() and torch.isfinite(out[980:, :4, :5].float()).all()
    assert torch.isnan(out[980:, 4:8].float()).all()
    assert torch.equal(out[:, 8:], clean[0][:, 8:])


def test_layouts_of_k_and_v_that_differ():
    s = Step([1900], [1900], 32, 8, 64, 16, torch.bfloat16, seed=22)
    v = s.v.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    out, lse = (torch.empty(s.q.shape, dtype=s.q.dtype, device="cuda"), torch.empty(s.q.shape[:2], device="cuda"))
    say("K and V of different layouts")
    dfc.paged_attention(s.q.cuda(), s.k.cuda(), v, s.table.cuda(), s.cu.cuda(), s.lens.cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    check_rows(s, out, lse)


@pytest.mark.parametrize("dim", [64, 256])
def test_one_workspace_for_every_window_and_layout(dim):
    # the bytes paged_attention_workspace gives, in a workspace that is NaN
    s = Step([1900, 300], [1900, 30], 32, 8, dim, 16, torch.bfloat16, seed=23)
    q, k, v, table, cu, lens = s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    other = s.v.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    size = dfc.paged_attention_workspace(q, k, v, table, cu, lens)
    for window in (0, 3, 500):
        for values in (v, other):
            say("workspace", dim, window, values.stride())
            out, lse = dfc.paged_attention(q, k, values, table, cu, lens, window=window, lse=True,
                                           workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
            torch.cuda.synchronize()
            check_rows(s, out, lse, window)
            check_rows(s, out, lse, window, r=1)


def test_many_requests():
    # more requests than a wavefront has lanes, and than a workgroup has threads
    for n in (65, 300, 700):
        total = [(37 * r) % 90 + 1 for r in range(n)]
        new = [min(t, 1 + r % 3) for r, t in enumerate(total)]
        total[n // 2] += 1500
        s = Step(total, new, 4, 2, 64, 16, torch.bfloat16, seed=n)
        for hint in (3, 0):
            say("many requests", n, hint)
            s.check(*s.run(max_q_len=hint))


@pytest.mark.parametrize("window", [1, 7, 64, 100, 2 ** 31 - 1])
def test_attention_window(window):
    s = Step([300, 90, 64], [70, 1, 64], 8, 2, 128, 16, torch.bfloat16, seed=window % 1000)
    say("window", window)
    s.check(*s.run(window=window), window=window)
    say("window, not causal", window)
    s.check(*s.run(window=window, causal=False), window=window, causal=False)


def test_attention_without_the_causal_mask():
    s = Step([300, 90, 64], [70, 1, 64], 8, 2, 64, 16, torch.float16, seed=3)
    say("not causal")
    s.check(*s.run(causal=False), causal=False)


def test_rows_that_see_nothing():
    # no tokens at all, more rows than tokens, a request without rows
    s = Step([0, 3, 40, 17], [1, 5, 0, 1], 4, 2, 128, 16, torch.bfloat16, seed=4)
    for hint in (0, 5, 1):
        say("rows that see nothing, hint", hint)
        s.check(*s.run(max_q_len=hint))


def test_attention_splits_and_joins_long_keys():
    # enough keys for several pieces of a tile, in each tile height
    for new, heads, kv_heads in ((1, 4, 2), (9, 8, 2), (40, 4, 1)):
        s = Step([9000], [new], heads, kv_heads, 64, 64, torch.float16, seed=new)
        say("split", new)
        s.check(*s.run(max_q_len=new))


def test_extreme_scores():
    # scores of tens of thousands: one key has all the weight; and a constant
    # score, where every key has the same
    s = Step([200, 70], [20, 1], 4, 2, 128, 16, torch.bfloat16, seed=6)
    say("scale 300")
    s.check(*s.run(scale=300.0), scale=300.0)
    say("scale 1e-30")
    s.check(*s.run(scale=1e-30), scale=1e-30)


def test_float16_small_weights_add_up():
    # one key far above 60,000 equal ones, whose weights are 2^-20 of its own
    n = 60000
    s = Step([8], [1], 1, 1, 64, 8, torch.float16, seed=7)
    pages = n // 8
    s.k, s.v = torch.zeros(pages, 8, 1, 64, dtype=torch.float16), torch.ones(pages, 8, 1, 64, dtype=torch.float16)
    s.table = torch.arange(pages, dtype=torch.int32)[None]
    s.total, s.lens = [n], torch.tensor([n], dtype=torch.int32)
    s.q.zero_()
    s.q[0, 0, 0] = 16.0
    s.k[3, 5, 0, 0] = 20 * np.log(2.0) / 2   # its score: 0.125 x 16 x this
    s.v[3, 5] = 0.0
    scale = 0.125
    say("float16 small weights")
    out, lse = s.run(scale=scale)
    z = scale * 16.0 * float(s.k[3, 5, 0, 0])
    share = (n - 1) / (n - 1 + np.exp(z))
    # a weight of 2^-20 is held above 2^-14, with all its bits: one rounding
    # of the weights, one of the output, and sums of n fp32 terms
    assert np.abs(as64(out) - share).max() <= share * (2 * 2.0 ** -11 + n * 2.0 ** -24)
    assert abs(float(lse[0, 0]) - np.log(n - 1 + np.exp(z))) <= n * 2.0 ** -24


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite_in_masked_places(bad):
    # tokens 60 and 100 of 130 new ones: rows before them must not notice
    for dtype in (torch.bfloat16, torch.float16):
        s = Step([150, 40], [130, 1], 4, 2, 128, 16, dtype, seed=8)
        clean = s.run()
        for tok in (80, 120):
            p, j = s.table[0, tok // 16], tok % 16
            s.v[p, j, 0, 5] = bad
            s.k[p, j, 1, 7] = bad
        say("not finite", bad, dtype)
        out, lse = s.run()
        # token i stands at 20 + i: those before 80 see neither key
        i = 60
        s.check(out, lse, rows=i)
        assert torch.isfinite(out[130:].float()).all() and torch.equal(out[130:], clean[0][130:])
        # those that see it: their weight is above 0, so the value is theirs
        seen = out[i:130, :2, 5].float().cpu()
        want = float("nan") if bad != bad else bad
        first = seen[:40]  # rows 60..99 see one of the two
        assert torch.isnan(first).all() if want != want else (first == want).all()
        others = out[i:130, :2, :5].float()
        assert torch.isfinite(others).all()
        # head group 1 has the key: a score of inf or NaN makes NaN, -inf nothing
        assert torch.isfinite(lse[:i]).all()


def test_strides_and_streams():
    s = Step([140, 33], [67, 33], 8, 2, 128, 16, torch.bfloat16, seed=9, order="hpd", extra_pages=3)
    say("cache with heads outside the page")
    s.check(*s.run())
    # q and out inside wider rows, on a stream that is not the current one
    wide = torch.zeros(s.q.shape[0], 3, 8, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = s.q.cuda()
    out = torch.full_like(wide, float("nan"))
    lse = torch.full(s.q.shape[:2], float("nan"), device="cuda")
    k, v, table, cu, lens = s.cache(s.k), s.cache(s.v), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("strided rows, side stream")
    dfc.paged_attention(wide[:, 1], k, v, table, cu, lens, out=out[:, 1], lse=lse, stream=side.cuda_stream)
    side.synchronize()
    s.check(out[:, 1], lse)
    assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, 2]).all()


def test_page_offsets_past_32_bits():
    # 40,000 pages of 128 x 8 x 128: K is 10.5 GB, and the pages used lie at its end
    n, page, kv_heads, dim = 40000, 128, 8, 128
    s = Step([700, 129], [3, 129], 16, kv_heads, dim, page, torch.bfloat16, seed=10)
    k, v = (torch.empty(n, page, kv_heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    used = s.k.shape[0]
    k[n - used:], v[n - used:] = s.k.cuda(), s.v.cuda()
    table = torch.where(s.table >= 0, s.table + (n - used), s.table).cuda()
    out, lse = torch.empty(s.q.shape, dtype=s.q.dtype, device="cuda"), torch.empty(s.q.shape[:2], device="cuda")
    say("offsets past 32 bits")
    dfc.paged_attention(s.q.cuda(), k, v, table, s.cu.cuda(), s.lens.cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    s.check(out, lse)
    # and the append's
    slots = torch.tensor([(n - 1) * page + 127, (n - 2) * page], device="cuda")
    x = torch.randn(2, kv_heads, dim, device="cuda").bfloat16()
    dfc.paged_append(x, -x, k, v, slots)
    torch.cuda.synchronize()
    assert torch.equal(k[n - 1, 127], x[0]) and torch.equal(v[n - 2, 0], -x[1])


def test_same_bits_again_and_no_stale_workspace():
    s = Step([2500, 800, 90], [5, 1, 90], 8, 2, 128, 16, torch.bfloat16, seed=11)
    need = dfc.paged_attention_workspace(s.q.cuda(), s.cache(s.k), s.cache(s.v), s.table.cuda(), s.cu.cuda(),
                                         s.lens.cuda())
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0xFF, 0x00, 0x5A):
        ws.fill_(fill)
        say("workspace fill", fill)
        got = s.run(workspace=ws)
        assert first is None or (torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]))
        first = got


def test_lengths_and_pages_that_make_no_sense():
    s = Step([300, 90], [2, 1], 4, 2, 128, 16, torch.bfloat16, seed=12)
    args = [s.q.cuda(), s.k.cuda(), s.v.cuda()]
    for name, table, cu, lens in (
            ("page past the cache", s.table.clone().index_fill_(1, torch.tensor([2]), 10 ** 6), s.cu, s.lens),
            ("missing page", s.table.clone().index_fill_(1, torch.tensor([1]), -1), s.cu, s.lens),
            ("length past the table", s.table, s.cu, torch.tensor([10 ** 9, 90], dtype=torch.int32)),
            ("negative length", s.table, s.cu, torch.tensor([-5, 90], dtype=torch.int32)),
            ("rows past q", s.table, torch.tensor([0, 2, 900], dtype=torch.int32), s.lens),
            ("descending rows", s.table, torch.tensor([0, 3, 1], dtype=torch.int32), s.lens),
            ("negative rows", s.table, torch.tensor([-7, 2, 3], dtype=torch.int32), s.lens)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        say(name)
        dfc.paged_attention(*args, table.cuda(), cu.cuda(), lens.cuda(), status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == dfc.ECORRUPT, name


def test_attention_refusals():
    s = Step([30], [2], 4, 2, 128, 16, torch.bfloat16, seed=13)
    q, k, v, t, cu, lens = (s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda())
    go = dfc.paged_attention
    with pytest.raises(TypeError):
        go(q.half(), k, v, t, cu, lens)
    with pytest.raises(TypeError):
        go(q.float(), k.float(), v.float(), t, cu, lens)
    with pytest.raises(TypeError):
        go(q.cpu(), k, v, t, cu, lens)
    with pytest.raises(TypeError):
        go(q, k, v, t.long(), cu, lens)
    with pytest.raises(TypeError):
        go(q, k, v, t, cu.long(), lens)
    with pytest.raises(ValueError):
        go(q[:, :3].contiguous(), k, v, t, cu, lens)
    with pytest.raises(ValueError):
        go(q, k, v, t, cu[:1], lens)
    with pytest.raises(ValueError):
        go(q, k, v, t, cu, lens, window=-1)
    with pytest.raises(ValueError):
        go(q, k, v, t, cu, lens, out=torch.empty(1, 4, 128, dtype=q.dtype, device="cuda"))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(dfc.DfcError) as e:
            go(q, k, v, t, cu, lens, scale=scale)
        assert e.value.status == dfc.EINVAL
    with pytest.raises(dfc.DfcError) as e:
        go(q, k, v, t, cu, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == dfc.ESIZE
    with pytest.raises(dfc.DfcError) as e:   # pages of 15 tokens
        go(q, k[:, :15], v[:, :15], t, cu, lens)
    assert e.value.status == dfc.EINVAL
    with pytest.raises(dfc.DfcError) as e:   # head dim not a multiple of 8
        go(q[..., :60], k[..., :60], v[..., :60], t, cu, lens)
    assert e.value.status == dfc.EINVAL
    with pytest.raises(dfc.DfcError) as e:   # rows at odd addresses
        go(q[..., 4:124], k[..., :120], v[..., :120], t, cu, lens)
    assert e.value.status == dfc.EINVAL
    # nothing to do
    none = torch.empty(0, 4, 128, dtype=q.dtype, device="cuda")
    assert go(none, k, v, t[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), lens[:0]).shape == (0, 4, 128)


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("source,dtype", [(torch.float32, torch.bfloat16), (torch.float32, torch.float16),
                                          (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16)])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,rot,page", [(1, 4, 1, 64, 64, 16), (13, 6, 3, 80, 32, 4),
                                                              (70, 8, 2, 128, 128, 16), (5, 3, 1, 8, 0, 1),
                                                              (9, 2, 2, 256, 256, 128)])
def test_append(tokens, heads, kv_heads, dim, rot, page, source, dtype, interleaved):
    g = torch.Generator().manual_seed(tokens + dim)
    q, k, v = (torch.randn(tokens, n, dim, generator=g).to(source) for n in (heads, kv_heads, kv_heads))
    pages = 2 * tokens // page + 2
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 4:
        slots[tokens // 2] = -1
    pos = torch.randint(0, 400, (tokens,), generator=g).int()
    angle = torch.arange(400)[:, None] * 10000.0 ** (-torch.arange(0, max(rot, 2), 2) / max(rot, 2))
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    kc, vc = (torch.full((pages, page, kv_heads, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("append", tokens, heads, dim, rot, source, dtype, interleaved)
    got = dfc.paged_append(k.cuda(), v.cuda(), kc, vc, slots.cuda(), q=q.cuda(), positions=pos.cuda(),
                           rotary=table.cuda() if rot else None, interleaved=interleaved, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref = [as64(x) for x in (q, k)]
    if rot:
        ref = [op.rotate(x, pos.tolist(), table.numpy(), interleaved) for x in ref]
    size = [np.abs(as64(x)).max(-1, keepdims=True) for x in (q, k)]
    # two products and a sum in fp32, then one rounding
    u = U[dtype]
    small = 2.0 ** -24 if dtype == torch.float16 else 0.0
    stored = slots >= 0
    assert (np.abs(as64(got) - ref[0]) <= u * np.abs(ref[0]) + 2.0 ** -21 * size[0] + small).all()
    flat_k, flat_v = as64(kc).reshape(-1, kv_heads, dim), as64(vc).reshape(-1, kv_heads, dim)
    at = slots[stored].numpy()
    kept = stored.numpy()
    assert (np.abs(flat_k[at] - ref[1][kept]) <= u * np.abs(ref[1][kept]) + 2.0 ** -21 * size[1][kept] + small).all()
    assert np.array_equal(flat_v[at], as64(v.to(dtype))[kept])
    rest = np.setdiff1d(np.arange(pages * page), at)
    assert np.isnan(flat_k[rest]).all() and np.isnan(flat_v[rest]).all()


def test_append_strides_and_a_quarter_turn():
    # cos 0, sin 1: the pair (a, b) becomes (-b, a) exactly
    x = torch.arange(2 * 6 * 32, dtype=torch.float32, device="cuda").view(2, 6, 32)   # k, v, q side by side
    kc, vc = (torch.zeros(4, 2, 8, 32, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)[:, :, :2]
              for _ in range(2))
    table = torch.cat([torch.zeros(1, 16), torch.ones(1, 16)], 1).cuda()
    q_out = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")[:, 1:3, :32]
    slots = torch.tensor([9, 30], device="cuda")
    dfc.paged_append(x[:, :2], x[:, 2:4], kc, vc, slots, q=x[:, 4:], q_out=q_out,
                     positions=torch.zeros(2, dtype=torch.int32, device="cuda"), rotary=table)
    torch.cuda.synchronize()
    turned = torch.cat([-x[..., 16:], x[..., :16]], -1).bfloat16()
    for t, (p, j) in enumerate(((1, 1), (3, 6))):
        assert torch.equal(kc[p, j], turned[t, :2]) and torch.equal(vc[p, j], x[t, 2:4].bfloat16())
    assert torch.equal(q_out, turned[:, 4:])
    assert int((kc != 0).any(-1).sum()) == 4


def test_append_slots_and_positions_that_make_no_sense():
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.ones(4, 64, device="cuda")
    for slots, pos in (([0, 10 ** 12, 1], [0, 1, 2]), ([0, 32, 1], [0, 1, 2]), ([0, 2, 1], [0, 4, 2]),
                       ([0, 2, 1], [0, -1, 2])):
        kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        say(slots, pos)
        dfc.paged_append(x, x, kc, vc, torch.tensor(slots, device="cuda"),
                         positions=torch.tensor(pos, dtype=torch.int32, device="cuda"), rotary=table, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == dfc.ECORRUPT
        assert torch.equal(vc[0, 0], x[0]) and torch.equal(vc[0, 1], x[2])


def test_append_refusals():
    x = torch.ones(3, 2, 64, device="cuda")
    kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        dfc.paged_append(x.half(), x.half(), kc, vc, slots)
    with pytest.raises(TypeError):
        dfc.paged_append(x, x, kc, vc, slots.int())
    with pytest.raises(ValueError):
        dfc.paged_append(x, x, kc, vc, slots[:2])
    with pytest.raises(ValueError):
        dfc.paged_append(x, x[:, :1], kc, vc, slots)
    with pytest.raises(ValueError):
        dfc.paged_append(x, x, kc, vc, slots, rotary=torch.ones(4, 64, device="cuda"))
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for width in (24, 80):   # not a multiple of 16; more than a head
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_append(x, x, kc, vc, slots, positions=pos, rotary=torch.ones(4, width, device="cuda"))
        assert e.value.status == dfc.EINVAL
    b = x.bfloat16()
    with pytest.raises(dfc.DfcError) as e:   # rotated in place
        dfc.paged_append(b, b, kc, vc, slots, q=b, q_out=b, positions=pos, rotary=torch.ones(4, 64, device="cuda"))
    assert e.value.status == dfc.EINVAL
    dfc.paged_append(x[:0], x[:0], kc, vc, slots[:0])


# --------------------------------------------------------------------- plan

def run_plan(context, new, page, ring, head, tail, tokens=None, width=None, holes=0, seed=0):
    rng = np.random.default_rng(seed)
    have = [-(-c // page) for c in context]
    need = [-(-(c + n) // page) for c, n in zip(context, new)]
    width = max(need + [1]) + 2 if width is None else width
    table = np.full((len(context), width), -7, np.int32)
    used = rng.permutation(100000)
    for r, h in enumerate(have):
        table[r, :h] = used[:h]
        used = used[h:]
    free = used[:ring].astype(np.int32)
    tokens = sum(new) + 5 if tokens is None else tokens
    want = op.plan(context, new, table, free, (head, tail), page, tokens)
    dev = torch.from_numpy(table).cuda()
    cursor = torch.tensor([head, tail], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dfc.paged_plan(torch.tensor(context, dtype=torch.int32, device="cuda"),
                         torch.tensor(new, dtype=torch.int32, device="cuda"), dev, torch.from_numpy(free).cuda(),
                         cursor, page, tokens, status=status)
    torch.cuda.synchronize()
    assert torch.equal(cursor.cpu(), torch.tensor([head, tail]))
    return want, (dev, got.seq_lens, got.cu_q, got.slots, got.positions, got.cursor), int(status.item())


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("requests,longest", [(1, 1), (3, 50), (64, 1), (1000, 7), (1024, 3), (1025, 2), (2600, 9)])
def test_plan(requests, longest, page):
    rng = np.random.default_rng(requests + page)
    context = rng.integers(0, 60, requests).tolist()
    new = rng.integers(0 if requests > 1 else 1, longest + 1, requests).tolist()
    say("plan", requests, longest, page)
    ring = sum(new) + 3
    want, got, status = run_plan(context, new, page, ring, 10 * ring + 2, 10 * ring + 2 + ring)
    assert status == 0
    for w, x in zip(want, got):
        assert np.array_equal(w, x.cpu().numpy())


def test_plan_of_long_prompts():
    want, got, status = run_plan([0, 5, 0, 4000], [9000, 1, 0, 5000], 16, 1000, 0, 900)
    assert status == 0
    for w, x in zip(want, got):
        assert np.array_equal(w, x.cpu().numpy())


def test_plan_runs_out_of_pages():
    want, got, status = run_plan([3, 16, 0, 31], [14, 40, 20, 1], 16, 10, 7, 11)
    assert status == dfc.ESIZE and (want[3] == -1).sum() > 5
    for w, x in zip(want, got):
        assert np.array_equal(w, x.cpu().numpy())


def test_plan_without_requests():
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    free, cursor = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([1, 3], device="cuda")
    p = dfc.paged_plan(e, e, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), free, cursor, 16, 2)
    assert p.cu_q.tolist() == [0] and p.slots.tolist() == [-1, -1] and p.cursor.tolist() == [1, 3]


def test_plan_inputs_that_make_no_sense():
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((2, 4), -7, **i32)
    free = torch.arange(10, 30, **i32)

    def go(context, new, cursor, tokens=40, t=table):
        status = torch.zeros(1, **i32)
        t = t.clone()
        p = dfc.paged_plan(torch.tensor(context, **i32), torch.tensor(new, **i32), t, free,
                           torch.tensor(cursor, device="cuda"), 16, tokens, status=status)
        torch.cuda.synchronize()
        return p, t, int(status.item())

    p, t, status = go([0, -4], [3, -2], [0, 20])
    assert status == dfc.ECORRUPT and p.cu_q.tolist() == [0, 3, 3] and p.slots.tolist() == [160, 161, 162] + [-1] * 37
    p, t, status = go([0, 0], [3, 2], [5, 26])          # more free pages than the ring has
    assert status & 0xFFFFFFFF == (dfc.ECORRUPT | dfc.ESIZE) & 0xFFFFFFFF and (p.slots == -1).all()
    p, t, status = go([0, 0], [3, 90], [0, 20], tokens=100)   # more pages than a row holds
    assert status == dfc.ESIZE and p.slots[3 + 64:93].eq(-1).all() and p.slots[3:67].ge(0).all()
    p, t, status = go([0, 0], [3, 5], [0, 20], tokens=4)      # more tokens than fit
    assert status == dfc.ESIZE and p.cu_q.tolist() == [0, 3, 4] and p.slots.tolist() == [160, 161, 162, 176]
    p, t, status = go([17, 0], [3, 1], [0, 20])               # the page it holds is missing
    assert status == dfc.ECORRUPT and p.slots.tolist()[:4] == [-1, -1, -1, 160]


def test_plan_refusals():
    i32 = dict(dtype=torch.int32, device="cuda")
    c, n, t = torch.zeros(2, **i32), torch.ones(2, **i32), torch.zeros(2, 4, **i32)
    free, cursor = torch.arange(10, **i32), torch.tensor([0, 10], device="cuda")
    with pytest.raises(TypeError):
        dfc.paged_plan(c.long(), n, t, free, cursor, 16, 2)
    with pytest.raises(TypeError):
        dfc.paged_plan(c, n, t, free, cursor.int(), 16, 2)
    with pytest.raises(ValueError):
        dfc.paged_plan(c, n[:1], t, free, cursor, 16, 2)
    with pytest.raises(ValueError):
        dfc.paged_plan(c, n, t[:1], free, cursor, 16, 2)
    for kw in (dict(page_size=0), dict(page_size=24), dict(page_size=16, free=free[:0])):
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_plan(c, n, t, kw.get("free", free), cursor, kw["page_size"], 2)
        assert e.value.status == dfc.EINVAL
    p = dfc.paged_plan(c, n, t, free, cursor, 16, 2)
    for out in (p._replace(cursor=cursor), p._replace(seq_lens=c)):
        with pytest.raises(dfc.DfcError) as e:
            dfc.paged_plan(c, n, t, free, cursor, 16, 2, out=out)
        assert e.value.status == dfc.EINVAL


# ---------------------------------------------------------------- one step

def test_a_captured_step_follows_the_lengths():
    """Plan, append and attention captured once; replays with other lengths
    between them match the eager calls."""
    H, K, D, P, R, T = 8, 2, 64, 16, 3, 6
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.zeros(R, **i32), torch.zeros(R, **i32)
    table = torch.full((R, 20), -1, **i32)
    free = torch.randperm(60, device="cuda").int()
    cursor = torch.tensor([0, 60], device="cuda")
    kc, vc = (torch.zeros(60, P, K, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.zeros(T, n, D, device="cuda") for n in (H, K, K))
    angle = torch.arange(320, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    rotary = torch.cat([angle.cos(), angle.sin()], 1).float()
    plan = dfc.paged_plan(ctx, new, table, free, cursor, P, T)
    q16 = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q16)
    ws = torch.empty(dfc.paged_attention_workspace(q16, kc, vc, table, plan.cu_q, plan.seq_lens), dtype=torch.uint8,
                     device="cuda")

    def step():
        dfc.paged_plan(ctx, new, table, free, cursor, P, T, out=plan)
        dfc.paged_append(k, v, kc, vc, plan.slots, q=q, q_out=q16, positions=plan.positions, rotary=rotary)
        dfc.paged_attention(q16, kc, vc, table, plan.cu_q, plan.seq_lens, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [[], [], []]
    for i, counts in enumerate(([2, 3, 1], [1, 1, 1], [1, 0, 4], [0, 5, 1], [1, 1, 1])):
        new.copy_(torch.tensor(counts))
        for t in (q, k, v):
            t.normal_()
        say("replay", i, counts)
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        kept = (table.clone(), kc.clone(), vc.clone())
        step()
        torch.cuda.synchronize()
        n = sum(counts)
        assert torch.equal(replayed[:n], out[:n])
        assert all(torch.equal(a, b) for a, b in zip(kept, (table, kc, vc)))
        # the whole history from scratch
        at = 0
        for r, c in enumerate(counts):
            pos = plan.positions[at: at + c].tolist()
            assert pos == list(range(len(held[r]), len(held[r]) + c))
            kr = torch.from_numpy(op.rotate(as64(k[at: at + c]), pos, rotary.cpu().numpy(), False))
            held[r] += [(kr[j], v[at + j].double().cpu()) for j in range(c)]
            if c:
                kk = torch.stack([x[0] for x in held[r]]).numpy()
                vv = torch.stack([x[1] for x in held[r]]).numpy()
                qq = op.rotate(as64(q[at: at + c]), pos, rotary.cpu().numpy(), False)
                ref, _, spread, _, mass = op.attention(qq, kk, vv, D ** -0.5)
                # q, k and v are rounded to 8 bits: a score moves by 2 u mass,
                # a weight by e^(2 of that); then v, the weights, the output
                u = 2.0 ** -8
                bound = (np.expm1(2 * 2.02 * u * mass)[..., None] + 3 * u) * spread + u * np.abs(ref) + 1e-5
                assert (np.abs(as64(out[at: at + c]) - ref) <= bound).all()
            at += c
        ctx.copy_(plan.seq_lens)
        cursor.copy_(plan.cursor)


# ------------------------------------------------------- scores far apart

# Tables so wide that a step of 130 tokens of 8 heads over 2 takes each tile
# height (the keys a table has room for choose it); heads wider than 128 take
# two of them.
HEIGHTS = [(16, 128), (16384, 128), (65536, 128), (262144, 128), (16384, 64), (262144, 64), (65536, 80), (16, 200),
           (262144, 256)]


def far_apart(s, seed):
    """Small whole numbers for q and k: scores before the scale are whole, exact
    in fp32, and with a scale of 1024 those that are not a row's largest weigh
    nothing.  Returns the largest score, how many keys have it, and the mean of
    their values and of their magnitudes, by integers."""
    rng = np.random.default_rng(seed)
    q = rng.integers(-2, 3, s.q.shape)
    s.q = torch.from_numpy(q).to(s.q.dtype)
    tops, counts, means, spreads = [], [], [], []
    for r, n in enumerate(s.total):
        heads, kv_heads, dim = s.q.shape[1], s.k.shape[2], s.k.shape[3]
        k = rng.integers(-2, 3, (n, kv_heads, dim))
        k[n // 3] = k[n // 2]  # two keys of one score
        for j in range(n):
            s.k[s.table[r, j // s.page], j % s.page] = torch.from_numpy(k[j]).to(s.k.dtype)
        v = op.gather(as64(s.v), s.table[r].numpy(), s.page, n)
        for i in range(s.new[r]):
            seen = n - s.new[r] + i + 1
            for h in range(heads):
                z = k[:seen, h * kv_heads // heads] @ q[int(s.cu[r]) + i, h]
                best = v[:seen, h * kv_heads // heads][z == z.max()]
                tops.append(z.max())
                counts.append(len(best))
                means.append(best.mean(0))
                spreads.append(np.abs(best).mean(0))
    shape = s.q.shape[:2]
    return (*(np.array(x).reshape(shape) for x in (tops, counts)),
            *(np.array(x).reshape(s.q.shape) for x in (means, spreads)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("keys,dim", HEIGHTS)
def test_scores_of_tens_of_thousands(keys, dim, dtype):
    s = Step([300, 90], [130, 1], 8, 2, dim, 16, dtype, seed=60 + dim, extra_pages=keys // 16)
    top, count, mean, spread = far_apart(s, dim)
    scale = 1024.0
    assert np.abs(top).max() * scale > 30000
    say("scores of tens of thousands", keys, dim, dtype)
    out, lse = s.run(scale=scale)
    # one rounding of the weights and one of the output, u each, and sums in
    # fp32; a weight's exponent is rounded to 2^-24 of the score, but all
    # weights that are not 0 are equal, so that it leaves the mean
    bound = (2 * U[dtype] + 2.0 ** -15) * spread + 2.0 ** -24
    assert (np.abs(as64(out) - mean) <= bound).all(), np.abs(as64(out) - mean).max()
    assert (np.abs(mean) > 4 * bound).mean() > 0.9  # the bound tells a wrong row
    ref = scale * top + np.log(count)
    assert (np.abs(as64(lse) - ref) <= 2.0 ** -22 * scale * np.abs(top) + 2.0 ** -20).all()


# ---------------------------------------------- pages that are not there

def run_with_pages(s, holes, window=0, last=50.0):
    """The step with the table entries `holes` ((request, place): page) in
    place of its own, over a cache whose last page nobody owns and holds
    `last`.  Returns out, lse, the status."""
    page = torch.full((1,) + tuple(s.k.shape[1:]), last, dtype=s.k.dtype)
    k, v = (torch.cat([c, page]).cuda() for c in (s.k, s.v))
    table = s.table.clone()
    for (r, i), p in holes.items():
        table[r, i] = p
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = dfc.paged_attention(s.q.cuda(), k, v, table.cuda(), s.cu.cuda(), s.lens.cuda(), window=window, lse=True,
                                   status=status)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


@pytest.mark.parametrize("last", [50.0, float("nan")], ids=["finite", "nan"])
@pytest.mark.parametrize("keys,dim", HEIGHTS)
def test_pages_that_are_not_there_count_as_zeros(keys, dim, last):
    s = Step([300, 90], [130, 1], 8, 2, dim, 16, torch.bfloat16, seed=30 + dim, extra_pages=keys // 16)
    for absent in (-1, s.k.shape[0] + 1, 10 ** 6, -2 ** 31):
        holes = {(0, 2): absent, (0, 11): absent, (0, 18): absent, (1, 5): absent}
        say("absent pages", keys, dim, absent, last)
        out, lse, status = run_with_pages(s, holes, last=last)
        assert status == dfc.ECORRUPT
        # the definition over a cache with a page of zeros there
        z = Step.__new__(Step)
        z.__dict__.update(s.__dict__)
        zeros = torch.zeros((1,) + tuple(s.k.shape[1:]), dtype=s.k.dtype)
        z.k, z.v, z.table = torch.cat([s.k, zeros]), torch.cat([s.v, zeros]), s.table.clone()
        for r, i in holes:
            z.table[r, i] = s.k.shape[0]
        z.check(out, lse)


@pytest.mark.parametrize("absent", [-1, 10 ** 6])
@pytest.mark.parametrize("keys,dim", HEIGHTS)
def test_pages_behind_the_window_may_be_gone(keys, dim, absent):
    # pages that no row of the step sees: neither the result nor the status
    # knows of them, wherever the window begins in a tile of keys
    for window in (1, 20, 41, 100, 170):
        s = Step([431, 290], [130, 1], 8, 2, dim, 16, torch.bfloat16, seed=50 + window, extra_pages=keys // 16)
        holes = {}
        for r, (t, n) in enumerate(zip(s.total, s.new)):
            gone = max(0, t - n + 1 - window) // 16
            assert gone > 0
            holes.update({(r, i): absent for i in range(gone)})
        say("behind the window", keys, dim, absent, window)
        out, lse, status = run_with_pages(s, holes, window, last=float("nan"))
        assert status == 0, window
        s.check(out, lse, window=window)
        # one page further some row sees a key
        holes[(1, max(0, s.total[1] - window) // 16)] = absent
        assert run_with_pages(s, holes, window)[2] == dfc.ECORRUPT


# ------------------------------------------------- streams and allocations

def pool_of(t):
    """The stream (handle) from whose memory torch took a tensor."""
    at = t.untyped_storage().data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not torch's memory")


def reserved(handle):
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == handle)


def a_step(s, free, cursor, stream, current):
    """Plan, append and attention with results that the calls allocate, their
    work on `stream` (a handle or None)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    t, (n, heads, dim), kv_heads = s.table.cuda(), s.q.shape, s.k.shape[2]
    q, k, v = (torch.randn(n, h, dim, generator=g, device="cuda") for h in (heads, kv_heads, kv_heads))
    angle = torch.randn(2048, dim, generator=g, device="cuda")
    held = (s.lens - torch.tensor(s.new, dtype=torch.int32)).cuda()
    new, kc, vc = torch.tensor(s.new, dtype=torch.int32, device="cuda"), *(torch.cat([c, c]).cuda()
                                                                                  for c in (s.k, s.v))
    torch.cuda.synchronize()
    p = dfc.paged_plan(held, new, t, free, cursor, s.page, n, stream=stream)
    r = dfc.paged_append(k, v, kc, vc, p.slots, q=q, positions=p.positions, rotary=angle, stream=stream)
    torch.cuda.empty_cache()
    before = reserved(current)
    out, lse = dfc.paged_attention(r, kc, vc, t, p.cu_q, p.seq_lens, lse=True, stream=stream)
    # neither the results nor the workspace come from elsewhere
    if stream is not None and stream != current:
        assert reserved(current) == before
    torch.cuda.synchronize()
    return [*p, r, out, lse]


@pytest.mark.parametrize("given", ["another stream", "the default stream", "the current stream"])
def test_what_a_call_allocates_belongs_to_its_stream(given):
    # a given stream does not wait for the current one, whose earlier work may
    # still use memory that torch hands out on the current stream
    s = Step([900, 20, 300], [700, 1, 33], 32, 8, 128, 16, torch.bfloat16, seed=40, extra_pages=60)
    n = s.k.shape[0]
    free, cursor = torch.arange(n, 2 * n, dtype=torch.int32, device="cuda"), torch.tensor([0, n], device="cuda")
    say("allocations", given)
    torch.cuda.empty_cache()
    plain = a_step(s, free, cursor, None, 0)
    side = torch.cuda.Stream()
    assert side.cuda_stream != 0 == torch.cuda.default_stream().cuda_stream
    if given == "another stream":
        got, handle = a_step(s, free, cursor, side.cuda_stream, 0), side.cuda_stream
    elif given == "the default stream":
        with torch.cuda.stream(side):
            got, handle = a_step(s, free, cursor, 0, side.cuda_stream), 0
    else:
        with torch.cuda.stream(side):
            got, handle = a_step(s, free, cursor, side.cuda_stream, side.cuda_stream), side.cuda_stream
    assert torch.cuda.current_stream().cuda_stream == 0
    for a, b in zip(plain, got):
        assert pool_of(b) == handle
        assert torch.equal(a.nan_to_num(), b.nan_to_num())


def test_results_given_by_the_caller_stay_the_callers():
    s = Step([140, 33], [67, 33], 8, 2, 128, 16, torch.bfloat16, seed=9)
    q, k, v, table, cu, lens = s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("results given, side stream")
    r = dfc.paged_attention(q, k, v, table, cu, lens, out=out, lse=lse, stream=side.cuda_stream)
    side.synchronize()
    assert r[0] is out and r[1] is lse
    s.check(out, lse)


# ------------------------------------------------------------------ autograd

def test_gradients_are_refused_and_writes_are_told():
    s = Step([30, 7], [2, 1], 4, 2, 64, 16, torch.bfloat16, seed=70)
    q, k, v, table, cu, lens = s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    x, slots = torch.randn(3, 2, 64, device="cuda").bfloat16(), torch.arange(3, device="cuda")
    angle, pos = torch.randn(4, 64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def attention(**other):
        a = dict(dict(q=q, k_cache=k, v_cache=v), **other)
        return dfc.paged_attention(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), table, cu, lens, **a)

    def append(**other):
        a = dict(dict(k=x, v=x, k_cache=k.clone(), v_cache=v.clone(), q=q, rotary=angle), **other)
        return dfc.paged_append(a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), slots, positions=pos, **a)

    say("gradients")
    for call, names in ((attention, dict(q=q, k_cache=k, v_cache=v, out=q, lse=torch.empty(3, 4, device="cuda"))),
                        (append, dict(k=x, v=x, k_cache=k, v_cache=v, q=q, q_out=q, rotary=angle))):
        for name, t in names.items():
            with pytest.raises(ValueError, match="gradient"):
                call(**{name: t.clone().requires_grad_()})
            with torch.no_grad():
                got = call(**{name: t.clone().requires_grad_()})
            assert not (got[0] if isinstance(got, tuple) else got).requires_grad or name in ("out", "q_out")
    torch.cuda.synchronize()
    # what a call writes in place: its version moves, what it reads does not
    out, lse = torch.empty_like(q), torch.empty(3, 4, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = {n: t._version for n, t in dict(q=q, k=k, v=v, table=table, lens=lens).items()}
    seen = [t._version for t in (out, lse, status)]
    attention(out=out, lse=lse, status=status)
    assert [t._version for t in (out, lse, status)] == [n + 1 for n in seen]
    assert before == {n: t._version for n, t in dict(q=q, k=k, v=v, table=table, lens=lens).items()}
    kept = (k.float() * 1.0).bfloat16().requires_grad_()
    held = k.clone()
    loss = (kept * held).sum()      # held is saved for the backward pass
    append(k_cache=held, v_cache=v.clone())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        frozen = k.clone()
    append(k_cache=frozen, v_cache=v.clone())   # outside the mode too
    new = torch.ones(2, dtype=torch.int32, device="cuda")
    free, cursor = torch.arange(10, dtype=torch.int32, device="cuda"), torch.tensor([0, 10], device="cuda")
    at = table._version
    p = dfc.paged_plan(lens, new, table, free, cursor, 16, 2)
    assert table._version == at + 1
    versions = [t._version for t in p]
    dfc.paged_plan(lens, new, table, free, cursor, 16, 2, out=p)
    assert [t._version for t in p] == [n + 1 for n in versions]
    torch.cuda.synchronize()
