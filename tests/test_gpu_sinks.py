"""GPU: attention with a window and first tokens that stay visible
(dfc_paged_attention_sinks) against the oracle's definition in 64 bits, inside
the bounds that test_gpu_paged.py derives from the formula (with N the keys of
a row's request)."""
import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged import Step, U, as64, say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(s, out, lse, window, sinks, causal=True, rows=None):
    """Rows (all, or some of the first request's) against the definition."""
    dim, u = s.q.shape[2], U[s.q.dtype]
    got, got_lse, q = as64(out), as64(lse), as64(s.q)
    for r in range(len(s.total) if rows is None else 1):
        a, n, total = int(s.cu[r]), s.new[r], s.total[r]
        if not n:
            continue
        k, v = (op.gather(as64(c), s.table[r].clamp(min=0).numpy(), s.page, total) for c in (s.k, s.v))
        for i in range(n) if rows is None else rows:
            # the definition of one row: what it sees of the first `end` keys
            end = total - n + i + 1 if causal else total
            lo = max(0, total - n + i + 1 - window) if window else 0
            seen = [j for j in range(max(end, 0)) if j >= lo or j < sinks]
            ref, ref_lse, spread, top, mass = op.attention(q[a + i: a + i + 1], k[seen], v[seen], dim ** -0.5,
                                                           causal=False)
            e = 2.0 ** -23 * (dim * mass + 2 * top + len(seen) + 16)[..., None]
            lost = 2.0 ** -32 * len(seen) * np.abs(v[seen]).max(initial=0.0)
            bound = (u + 2 * e) * spread + u * np.abs(ref) + lost + 1e-30
            assert (np.abs(got[a + i] - ref[0]) <= bound[0]).all(), (r, i, np.abs(got[a + i] - ref[0]).max())
            if not seen:
                assert np.isneginf(got_lse[a + i]).all() and (got[a + i] == 0).all()
                continue
            diff = np.abs(got_lse[a + i] - ref_lse[0])
            assert (diff <= 4 * e[0, :, 0] + 2.0 ** -21 * (1 + np.abs(ref_lse[0]))).all(), (r, i)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("sinks", [1, 4, 32, 33, 100])
@pytest.mark.parametrize("window", [1, 20, 64, 150])
def test_against_the_definition(window, sinks, dtype):
    s = Step([330, 190, 64, 1, 402], [70, 1, 64, 1, 5], 8, 2, 128, 16, dtype, seed=window + sinks)
    for hint in (0, 70):
        say("sinks", window, sinks, dtype, hint)
        check(s, *s.run(window=window, sinks=sinks, max_q_len=hint), window, sinks)


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 4, 64, 1), (6, 2, 80, 8), (3, 1, 256, 64), (5, 5, 24, 4),
                                                     (16, 1, 200, 128)])
def test_heads_and_pages(heads, kv_heads, dim, page):
    s = Step([300, 77, 260], [33, 1, 2], heads, kv_heads, dim, page, torch.bfloat16, seed=dim)
    for window, sinks in ((50, 3), (7, 40), (200, 65)):
        say("sinks, heads of", dim, window, sinks)
        check(s, *s.run(window=window, sinks=sinks), window, sinks)


def test_without_the_causal_mask():
    s = Step([300, 90, 64], [70, 1, 64], 8, 2, 64, 16, torch.float16, seed=3)
    for window, sinks in ((20, 5), (100, 33)):
        say("sinks, not causal", window, sinks)
        check(s, *s.run(causal=False, window=window, sinks=sinks), window, sinks, causal=False)


# (tokens, window) of steps whose work takes each tile height for heads of 128
# and 64: 32, 64, 128 and 256 rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("total,new,heads,kv_heads,dim,window,sinks", [
    (1500, 8, 32, 8, 128, 500, 4),
    (1500, 600, 32, 8, 128, 200, 70),
    (2500, 1200, 32, 8, 128, 400, 4),
    (4200, 2500, 32, 8, 128, 777, 130),
    (4200, 2500, 32, 8, 64, 777, 4),
    (4200, 2500, 8, 8, 128, 300, 64),
    (2600, 1100, 16, 4, 256, 600, 33),
])
def test_every_tile_height(total, new, heads, kv_heads, dim, window, sinks, dtype):
    s = Step([total], [new], heads, kv_heads, dim, 16, dtype, seed=new)
    say("sinks, step of", new, "over", total, "window", window, dtype)
    out, lse = s.run(window=window, sinks=sinks, max_q_len=new)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    rows = sorted({i for i in (0, 1, 7, 31, 32, 63, 64, 65, 255, 256, 257, new // 2, new - 66, new - 2, new - 1)
                   if 0 <= i < new})
    check(s, out, lse, window, sinks, rows=rows)


def test_long_windows_are_split_and_repeat():
    for new, heads, kv_heads in ((1, 4, 2), (9, 8, 2), (40, 4, 1), (300, 8, 1)):
        s = Step([9000], [new], heads, kv_heads, 64, 64, torch.float16, seed=new)
        say("sinks, split", new)
        first = s.run(max_q_len=new, window=6000, sinks=70)
        check(s, *first, 6000, 70, rows=sorted({0, new // 2, new - 1}))
        again = s.run(max_q_len=new, window=6000, sinks=70)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_many_requests():
    for n in (65, 300):
        total = [(37 * r) % 90 + 1 for r in range(n)]
        new = [min(t, 1 + r % 3) for r, t in enumerate(total)]
        total[n // 2] += 1500
        s = Step(total, new, 4, 2, 64, 16, torch.bfloat16, seed=n)
        say("sinks, many requests", n)
        check(s, *s.run(max_q_len=3, window=21, sinks=4), 21, 4)


def test_rows_that_see_nothing():
    s = Step([0, 3, 40, 17], [1, 5, 0, 1], 4, 2, 128, 16, torch.bfloat16, seed=4)
    say("sinks, rows that see nothing")
    check(s, *s.run(window=2, sinks=1), 2, 1)


def test_where_sinks_change_nothing():
    s = Step([330, 190, 64], [70, 1, 64], 8, 2, 128, 16, torch.bfloat16, seed=5)
    say("sinks that change nothing")
    plain, narrow = s.run(), s.run(window=50)
    for a, b in ((plain, s.run(sinks=9)), (narrow, s.run(window=50, sinks=0))):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for sinks in (330, 2 ** 31 - 1):  # every token is one
        check(s, *s.run(window=50, sinks=sinks), 0, 0)


def gone(s, window, sinks):
    """Table entries of the pages that no row sees: wholly behind the first
    row's window, and behind the sinks."""
    return [(r, i) for r, (t, n) in enumerate(zip(s.total, s.new))
            for i in range(-(-sinks // s.page), max(0, t - n + 1 - window) // s.page)]


@pytest.mark.parametrize("absent", [-1, 10 ** 6])
@pytest.mark.parametrize("dim,heads,new", [(128, 8, 130), (64, 8, 1), (256, 8, 40), (128, 32, 1900)])
def test_pages_between_sinks_and_window_may_be_gone(dim, heads, new, absent):
    for window, sinks in ((20, 1), (41, 33), (100, 64)):
        s = Step([300 + new, 290], [new, 1], heads, 2, dim, 16, torch.bfloat16, seed=50 + window)
        want = s.run(window=window, sinks=sinks)
        holes = gone(s, window, sinks)
        assert len(holes) > 10
        say("behind the sinks", dim, new, absent, window, sinks)
        table = s.table
        s.table = table.clone()
        for r, i in holes:
            s.table[r, i] = absent
        got = s.run(window=window, sinks=sinks)       # (asserts that the status stays 0)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        # the sinks' own pages, and the window's, are missed
        for r, i in ((0, 0), (1, (sinks - 1) // 16), (1, (290 - window) // 16)):
            s.table = table.clone()
            s.table[r, i] = absent
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            dfc.paged_attention(s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda(),
                                window=window, sinks=sinks, status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == dfc.ECORRUPT, (r, i)
        s.table = table


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dim,new", [(128, 130), (64, 1), (128, 1900)])
def test_values_that_are_not_finite_where_no_row_looks(dim, new, bad):
    # behind the sinks in their own tile of keys, in the gap, and right before
    # the window
    window, sinks = 50, 5
    s = Step([300 + new], [new], 32, 8, dim, 16, torch.bfloat16, seed=9)
    want = s.run(window=window, sinks=sinks)
    first = 300 + 1 - window  # the first row's window
    for tok in (5, 20, 31, 100, first - 1):
        for c in (s.k, s.v):
            c[s.table[0, tok // 16], tok % 16] = bad
    say("sinks, not finite", dim, new, bad)
    out, lse = s.run(window=window, sinks=sinks)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    rows = sorted({i for i in (0, 1, 20, 49, 50, 120, new - 1) if i < new})
    check(s, out, lse, window, sinks, rows=rows)
    far = [i for i in (80, 129) if i < new]   # rows whose tiles meet none of them but the sinks'
    assert all(torch.allclose(out[i].float(), want[0][i].float(), atol=0.05) for i in far)


def test_a_sink_that_is_not_finite_is_seen():
    s = Step([400], [3], 4, 2, 64, 16, torch.bfloat16, seed=10)
    s.v[s.table[0, 0], 2, 0, 5] = float("inf")
    say("sink not finite")
    out, _ = s.run(window=20, sinks=3)
    assert torch.isposinf(out[:, :2, 5].float()).all() and torch.isfinite(out[:, 2:].float()).all()
    out, _ = s.run(window=20, sinks=2)
    assert torch.isfinite(out.float()).all()


def test_layouts_workspace_and_refusals():
    s = Step([900, 300], [500, 30], 32, 8, 64, 16, torch.bfloat16, seed=23)
    q, k, v, table, cu, lens = s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    other = s.v.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    size = dfc.paged_attention_workspace(q, k, v, table, cu, lens)
    for window, sinks in ((3, 500), (500, 3), (100, 100)):
        for values in (v, other):
            say("sinks, workspace", window, sinks)
            out, lse = dfc.paged_attention(q, k, values, table, cu, lens, window=window, sinks=sinks, lse=True,
                                           workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
            torch.cuda.synchronize()
            check(s, out, lse, window, sinks, rows=[0, 250, 499])
    for sinks in (-1, 1 << 31):
        with pytest.raises(ValueError):
            dfc.paged_attention(q, k, v, table, cu, lens, window=3, sinks=sinks)
    with pytest.raises(TypeError):
        dfc.paged_attention(q, k, v, table, cu, lens, window=3, sinks=2.5)


@pytest.mark.parametrize("total,new,heads,kv_heads,dim,window,sinks", [
    ([8200], [513], 32, 8, 128, 2048, 16),     # tiles of 128 rows, split
    ([9000], [1000], 32, 8, 128, 4096, 64),    # of 256, split
    ([9000], [700], 16, 4, 64, 5000, 3),
    ([1024], [1024], 32, 8, 128, 1000, 4),     # a table as short as the window
    ([1100, 5000], [600, 100], 32, 8, 128, 1000, 4),
    ([3000] * 6, [128] * 6, 32, 8, 128, 1500, 40),
    ([4000], [500], 8, 2, 256, 2500, 10),
])
def test_tall_tiles_stay_in_the_workspace(total, new, heads, kv_heads, dim, window, sinks):
    s = Step(total, new, heads, kv_heads, dim, 16, torch.bfloat16, seed=sum(new))
    q, k, v, table, cu, lens = s.q.cuda(), s.k.cuda(), s.v.cuda(), s.table.cuda(), s.cu.cuda(), s.lens.cuda()
    for most in (0, max(new)):
        size = dfc.paged_attention_workspace(q, k, v, table, cu, lens, most)
        store = torch.full((size + 4096,), 170, dtype=torch.uint8, device="cuda")
        say("sinks, tall tiles", total[:2], new[:2], window, most)
        first = [t.clone() for t in dfc.paged_attention(q, k, v, table, cu, lens, window=window, sinks=sinks, lse=True,
                                                        max_q_len=most, workspace=store[:size])]
        again = dfc.paged_attention(q, k, v, table, cu, lens, window=window, sinks=sinks, lse=True, max_q_len=most)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert (store[size:] == 170).all()
        assert torch.isfinite(first[0].float()).all() and torch.isfinite(first[1]).all()
        rows = sorted({i for i in (0, 31, 32, 63, 64, new[0] // 2, new[0] - 2, new[0] - 1) if 0 <= i < new[0]})
        check(s, *first, window, sinks, rows=rows)
