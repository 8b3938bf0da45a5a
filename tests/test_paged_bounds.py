"""The error bounds that the GPU's attention is held to
(tests/test_gpu_paged.py) reject an output of zeros, without a GPU: a bound as
wide as the result would pass anything."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as gpu  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(gpu.CASES)))
def test_zeros_are_rejected(case, dtype):
    s = gpu.Step(*gpu.CASES[case], dtype, seed=case)
    lse = np.concatenate([gpu.op.attention(
        gpu.as64(s.q)[int(s.cu[r]): int(s.cu[r + 1])],
        *(gpu.op.gather(gpu.as64(c), s.table[r].numpy(), s.page, n) for c in (s.k, s.v)), s.q.shape[2] ** -0.5)[1]
        for r, n in enumerate(s.total)])
    with pytest.raises(AssertionError):
        s.check(torch.zeros_like(s.q), torch.from_numpy(lse))


def test_scores_far_apart_by_integers():
    # the inputs of the test of large scores, against the definition in 64 bits
    s = gpu.Step([40, 9], [12, 1], 4, 2, 24, 4, torch.bfloat16, seed=1)
    top, count, mean, spread = gpu.far_apart(s, 0)
    for r, n in enumerate(s.total):
        a, b = int(s.cu[r]), int(s.cu[r + 1])
        k, v = (gpu.op.gather(gpu.as64(c), s.table[r].numpy(), s.page, n) for c in (s.k, s.v))
        out, lse, wide, _, _ = gpu.op.attention(gpu.as64(s.q)[a:b], k, v, 1024.0)
        assert np.allclose(out, mean[a:b], rtol=0, atol=1e-12) and np.allclose(wide, spread[a:b], rtol=0, atol=1e-12)
        assert np.allclose(lse, 1024.0 * top[a:b] + np.log(count[a:b]), rtol=0, atol=1e-9)
