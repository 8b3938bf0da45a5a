"""GPU: the append with norms of queries and keys (dfc_paged_append_normed)
against the oracle's definition in 64 bits.

The square sum and the root are in 64 bits, so a normed value carries the
root's rounding to 32 bits, one of x by it and one of the product with its
weight, 2^-24 each.  A rotation adds three roundings of 2^-24 of |a cos| + |b sin|, the store
one rounding u to the cache's type (2^-8 for bfloat16, 2^-11 for float16, below
their normal ranges half the smallest step, 2^-134 and 2^-25).  All in all
|got - ref| <= u |ref| + 6 2^-24 (|a cos| + |b sin|) (1 + u) + that."""
import sys

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def as64(t):
    return t.detach().cpu().double().numpy()


def table_of(positions, dim):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, dim, 2, dtype=torch.float64) / max(dim, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Case:
    def __init__(self, tokens, heads, kv_heads, dim, page, source, dtype, rot, weights=torch.float32, seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.dtype = page, dtype
        self.q, self.k, self.v = ((spread * torch.randn(tokens, n, dim, generator=g)).to(source)
                                  for n in (heads, kv_heads, kv_heads))
        self.wq, self.wk = ((1 + 0.3 * torch.randn(dim, generator=g)).to(weights) for _ in range(2))
        pages = -(-tokens // page) + 2
        self.slots = torch.randperm(pages * page, generator=g)[:tokens]
        self.positions = torch.randint(0, 500, (tokens,), generator=g).int()
        self.table = table_of(500, rot) if rot else None
        self.shape = (pages, page, kv_heads, dim)

    def run(self, norms="qk", eps=1e-6, interleaved=False, q=None, **kw):
        kc, vc = (torch.full(self.shape, float("nan"), dtype=self.dtype, device="cuda") for _ in range(2))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = dfc.paged_append(self.k.cuda(), self.v.cuda(), kc, vc, self.slots.cuda(),
                               q=self.q.cuda() if q is None else q,
                               positions=self.positions.cuda() if self.table is not None else None,
                               rotary=None if self.table is None else self.table.cuda(), interleaved=interleaved,
                               q_norm=self.wq.cuda() if "q" in norms else None,
                               k_norm=self.wk.cuda() if "k" in norms else None, eps=eps, status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return out, kc, vc

    def check(self, got, norms="qk", eps=1e-6, interleaved=False):
        out, kc, vc = got
        stored = self.slots >= 0
        flat = lambda c: c.reshape(-1, *self.shape[2:])[self.slots[stored].cuda()]
        assert torch.equal(flat(vc).cpu(), self.v.to(self.dtype)[stored])
        for got, x, w, name in ((out, self.q, self.wq, "q"), (flat(kc), self.k, self.wk, "k")):
            x = as64(x)
            if name in norms:
                x = op.norm(x, as64(w), eps)
            reach = np.abs(x)
            if self.table is not None:
                t = self.table.numpy()
                ref, size = op.rotate(x, self.positions.tolist(), t, interleaved), np.abs(x)
                half = t.shape[1] // 2
                for i in range(half):
                    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                    p = self.positions.numpy()
                    c, s = np.abs(t[p, i])[:, None], np.abs(t[p, half + i])[:, None]
                    reach[:, :, a], reach[:, :, b] = (size[:, :, a] * c + size[:, :, b] * s,
                                                      size[:, :, b] * c + size[:, :, a] * s)
            else:
                ref = x
            if name == "k":
                ref, reach = ref[stored.numpy()], reach[stored.numpy()]
            u = U[self.dtype]
            bound = u * np.abs(ref) + 6 * 2.0 ** -24 * reach * (1 + u) + TINY[self.dtype]
            assert (np.abs(as64(got) - ref) <= bound).all(), (name, np.abs(as64(got) - ref).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("source", ["f32", "cache"])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,page,rot", [
    (1, 32, 8, 128, 16, 128), (64, 32, 8, 128, 16, 128), (7, 3, 1, 80, 8, 80), (5, 4, 4, 256, 64, 64), (9, 2, 2, 8, 1, 0),
    (33, 6, 2, 24, 4, 16), (11, 5, 5, 200, 32, 192), (3, 8, 2, 64, 16, 32), (600, 12, 12, 64, 16, 64), (40, 1, 1, 40, 2, 32)])
def test_against_the_definition(tokens, heads, kv_heads, dim, page, rot, source, dtype):
    c = Case(tokens, heads, kv_heads, dim, page, torch.float32 if source == "f32" else dtype, dtype, rot, seed=tokens + dim)
    for interleaved in (False, True):
        for norms in ("qk", "q", "k"):
            say("norms", tokens, dim, rot, source, dtype, interleaved, norms)
            c.check(c.run(norms, interleaved=interleaved), norms, interleaved=interleaved)


def test_weights_of_the_caches_type():
    for dtype in U:
        c = Case(20, 8, 2, 128, 16, torch.float32, dtype, 64, weights=dtype, seed=1)
        say("norm weights of", dtype)
        c.check(c.run())


def test_what_is_not_normed_is_as_without_norms():
    c = Case(70, 8, 2, 128, 16, torch.float32, torch.bfloat16, 128, seed=2)
    plain = c.run("")
    say("norms of one")
    q_only, k_only = c.run("q"), c.run("k")
    same = lambda a, b: torch.equal(a.nan_to_num(), b.nan_to_num())
    assert same(plain[1], q_only[1]) and same(plain[0], k_only[0]) and same(plain[2], k_only[2])
    assert not same(plain[0], q_only[0]) and not same(plain[1], k_only[1])
    # and the plain call is the one without the arguments
    kc, vc = (torch.full(c.shape, float("nan"), dtype=c.dtype, device="cuda") for _ in range(2))
    out = dfc.paged_append(c.k.cuda(), c.v.cuda(), kc, vc, c.slots.cuda(), q=c.q.cuda(), positions=c.positions.cuda(),
                           rotary=c.table.cuda())
    assert same(out, plain[0]) and same(kc, plain[1]) and same(vc, plain[2])


@pytest.mark.parametrize("spread", [0.0, 1e-30, 1e-12, 1e18, 3e37])
def test_sizes_at_the_ends_of_32_bits(spread):
    # squares of 1e37 leave 32 bits, those of 1e-30 vanish beside eps
    c = Case(12, 4, 2, 64, 16, torch.float32, torch.bfloat16, 64, seed=3, spread=spread)
    c.v.clamp_(-1e30, 1e30)
    for eps in (1e-6, 1e-20):
        say("norms of size", spread, eps)
        c.check(c.run(eps=eps), eps=eps)


def test_tokens_without_a_slot_and_strides():
    c = Case(50, 8, 2, 128, 16, torch.bfloat16, torch.bfloat16, 128, seed=4)
    c.slots[::3] = -1
    say("norms, no slots")
    c.check(c.run())
    # q, k and v as slices of one product's rows
    rows = torch.cat([c.q.flatten(1), c.k.flatten(1), c.v.flatten(1)], 1).cuda()
    q, k, v = rows[:, :1024].view(50, 8, 128), rows[:, 1024:1280].view(50, 2, 128), rows[:, 1280:].view(50, 2, 128)
    kc, vc = (torch.full(c.shape, float("nan"), dtype=c.dtype, device="cuda") for _ in range(2))
    say("norms, strided")
    out = dfc.paged_append(k, v, kc, vc, c.slots.cuda(), q=q, positions=c.positions.cuda(), rotary=c.table.cuda(),
                           q_norm=c.wq.cuda(), k_norm=c.wk.cuda())
    c.check((out, kc, vc))


def test_values_that_are_not_finite_stay_in_their_head():
    c = Case(9, 4, 2, 80, 16, torch.float32, torch.bfloat16, 80, seed=5)
    want = c.run()
    c.q[3, 1, 7] = float("nan")
    c.q[4, 2, 0] = float("inf")
    say("norms, not finite")
    got = c.run()
    for t, h in ((3, 1), (4, 2)):
        assert not torch.isfinite(got[0][t, h].float()).all()
        got[0][t, h] = want[0][t, h]
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(want, got))


def test_large_appends():
    # past the size from which stores pass the caches by
    c = Case(3000, 32, 8, 128, 16, torch.bfloat16, torch.bfloat16, 128, seed=6)
    say("norms, large")
    got = c.run()
    some = [*range(0, 3000, 271), 2999]
    assert torch.isfinite(got[0].float()).all()
    c.q, c.k, c.v, c.slots, c.positions = c.q[some], c.k[some], c.v[some], c.slots[some], c.positions[some]
    c.check((got[0][some], got[1], got[2]))


def test_refusals():
    c = Case(3, 4, 2, 64, 16, torch.bfloat16, torch.bfloat16, 64, seed=7)
    k, v, q, slots, wq, pos, table = (t.cuda() for t in (c.k, c.v, c.q, c.slots, c.wq, c.positions, c.table))
    kc, vc = (torch.zeros(c.shape, dtype=c.dtype, device="cuda") for _ in range(2))

    def go(q=q, **kw):
        return dfc.paged_append(k, v, kc, vc, slots, q=q, **kw)

    with pytest.raises(ValueError):
        go(q_norm=wq[:32])
    with pytest.raises(TypeError):
        go(q_norm=wq.double())
    with pytest.raises(TypeError):
        go(k_norm=wq.half())
    with pytest.raises(TypeError):
        go(q_norm=wq, k_norm=wq.bfloat16())
    with pytest.raises(TypeError):
        go(k_norm=wq.cpu())
    with pytest.raises(TypeError):
        go(k_norm=wq[None])
    with pytest.raises(TypeError):
        go(k_norm=[1.0] * 64)
    with pytest.raises(ValueError):
        go(q=None, q_norm=wq)
    with pytest.raises(ValueError, match="gradient"):
        go(k_norm=wq.clone().requires_grad_())
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-60):
        with pytest.raises(dfc.DfcError) as e:
            go(k_norm=wq, eps=eps)
        assert e.value.status == dfc.EINVAL
    with pytest.raises(dfc.DfcError):
        go(k_norm=torch.zeros(65, device="cuda")[1:])     # not 16-byte aligned
    with pytest.raises(dfc.DfcError):
        go(q_norm=wq, q_out=q)
    assert not kc.any() and not vc.any()
