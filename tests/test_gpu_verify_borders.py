"""GPU: verification of drafted tokens where little decides (dfc_verify_drafts):
drafts whose random number lies next to the border to within a few roundings of
64 bits, what is left of rows that nearly agree, and vocabularies beyond the
262,144 values whose sums are kept."""
import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
import test_gpu_verify as gv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

REAL = np.longdouble  # 64 bits of mantissa: the definition's side


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def next_to_the_border():
    """Logits z of float32, as many as there are in (-16, -2], for which the
    probability p = e^z / (1 + e^z) lies next to a number u of float32: by 5e-15
    to 3e-14 of itself."""
    z = np.arange(np.float32(2).view(np.uint32), np.float32(16).view(np.uint32), dtype=np.uint32).view(np.float32)
    found = []
    for some in np.array_split(z, 64):
        p = 1 / (1 + np.exp(some.astype(REAL)))
        u = p.astype(np.float32)
        far = np.abs(u.astype(REAL) / p - 1)
        keep = (far > 5e-15) & (far < 3e-14)
        found += [(-a, b, b < c) for a, b, c in zip(some[keep], u[keep], p[keep])]
    return found


def test_drafts_next_to_the_border():
    """Errors of a probability here, of itself: 2^t 6.3e-16 and Horner's
    roundings 1.2e-16; t = z log2(e), |t| < 24, is off by half a unit, 2^-49, and
    by 24 2^-53 of the constant's, together 4.4e-15, times ln 2: 3.1e-15; sum,
    quotient and product 3 2^-53.  5e-15 covers them: 4.2e-15."""
    cases = next_to_the_border()
    assert len(cases) >= 10 and 0 < sum(h for _, _, h in cases) < len(cases)
    n = len(cases)
    logits = torch.zeros(2 * n, 2)
    logits[::2, 1] = torch.tensor([float(z) for z, _, _ in cases])
    u = torch.full((2 * n,), 0.5)
    u[::2] = torch.tensor([float(x) for _, x, _ in cases])
    drafts = torch.tensor([1, 0] * n)
    gv.say("verify, drafts next to the border", n)
    got = dfc.verify_drafts(logits.cuda(), torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"), drafts.cuda(),
                            u.cuda())
    assert got.accepted.tolist() == [int(h) for _, _, h in cases]


def probabilities(z):
    e = np.exp(z.numpy().astype(REAL) - z.max().numpy().astype(REAL))
    return e / e.sum()


@pytest.mark.parametrize("vocab", [50, 3000, 128256])
@pytest.mark.parametrize("apart", ["masked 8e-8", "masked 3e-11", "an ulp"])
def test_rows_that_nearly_agree(vocab, apart):
    """A draft refused against a drafter that is the model but for one token.
    What is left sums to that little, and the token drawn is the definition's to
    within 5e-14 of a probability: a probability's errors (6.3e-16 and 1.2e-16, and
    3.1e-16 |t| of four roundings in t = (z - top) / T log2(e)) come to 3.1e-16 times
    the mean of |t|, below 24.5, and 7.5e-16, over a row 8.4e-15; twice that, for the
    sum's, and 3.3e-15 of 30 additions make 2e-14, of two rows 4e-14."""
    g = torch.Generator().manual_seed(vocab)
    z = 2 * torch.randn(vocab, generator=g)
    x = vocab // 3
    model, drafter = z.clone(), z.clone()
    n = 40
    u = torch.rand(2 * n, generator=g)
    if apart == "an ulp":
        model[x] = drafter[x] = 4.5
        drafter[x] = torch.nextafter(drafter[x], torch.tensor(20.0))
        u[::2] = 1 - 2.0 ** -24
    else:
        model[x] = -torch.inf
        others = probabilities(model[torch.arange(vocab) != x])
        top = model.max()
        drafter[x] = float(top - np.log(float(others.max())) + np.log(float(apart.split()[1])))
    p, q = probabilities(model), probabilities(drafter)
    left = np.maximum(p - q, 0)
    sums = np.concatenate([[REAL(0)], np.cumsum(left)])
    assert 0 < sums[-1] < 1e-6
    rows = torch.stack([model, z]).repeat(n, 1)
    drafts = torch.full((2 * n,), x)
    gv.say("verify, rows that nearly agree", vocab, apart, float(sums[-1]))
    got = dfc.verify_drafts(rows.cuda(), torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"), drafts.cuda(),
                            u.cuda(), draft_logits=torch.stack([drafter, z]).repeat(n, 1).cuda())
    assert not got.accepted.any()
    for token, v in zip(got.tokens.tolist(), u[1::2].tolist()):
        share = REAL(v) * sums[-1]
        assert token != x and sums[token] - 5e-14 <= share <= sums[token + 1] + 5e-14


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("vocab", [262145, 300001])
def test_vocabularies_past_the_sums_that_are_kept(vocab, drafter, dtype):
    """A row of more than 256 pieces of 1,024 values: those past them are added
    up again for each token."""
    for spread, seed in ((2.0, 0), (0.01, 1)):
        s = gv.Step([3, 1, 2, 2], vocab, dtype, drafter, seed=seed, spread=spread, temperature=0.9)
        # the last request's draft lies in the last piece; where it is certain it
        # has a good part of the weight and is refused
        s.x[6] = vocab - 1
        s.z[6, vocab - 1] = s.z[6].max() + 8 * spread
        if drafter:
            s.d[6, vocab - 1] = s.z[6, vocab - 1] + 4 * spread
        gv.say("verify, large vocabulary", vocab, drafter, dtype, spread)
        for u in (0.3, 0.9, 0.99, 1 - 2.0 ** -13, 1 - 2.0 ** -24):
            s.u[:] = u
            s.u[6] = 1 - 2.0 ** -20
            got = s.run()
            assert got[2] == 0 and got[0][3] == 0
            s.check(got)
