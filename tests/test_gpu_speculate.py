"""GPU: the serving example's answers with drafts (examples/serve.py): normed
heads, a window with sinks, verification and pages given back, together over many
steps.  Greedy answers are compared with every request recomputed at once: each
token's logit has to be the largest but for what roundings move, as in
test_gpu_serve.py (2^-8 a value, a dozen on a token's way through two layers, of
the row's norm, for each of the two logits compared)."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("speculate_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("norms,window,sinks", [(False, 0, 0), (True, 0, 0), (True, 24, 4)])
def test_greedy_answers_with_drafts(example, norms, window, sinks):
    server = example.Server(layers=2, requests=5, pages=40, max_pages=12, norms=norms, window=window, sinks=sinks)
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, 512, n).tolist() for n in (1, 16, 17, 40, 90)]
    prompts[3] = prompts[3][:20] * 2   # something to look up
    ids, steps, held = example.speculate(server, prompts, 14)
    torch.cuda.synchronize()
    assert int(server.status.item()) == 0
    assert all(i[: len(p)] == p and len(i) == len(p) + 14 for i, p in zip(ids, prompts))
    # all have ended: every page is on the ring again, once
    head, tail = server.cursor.tolist()
    assert tail - head == 40 and not server.context.any() and not server.shared.any()
    assert sorted(server.free.tolist()) == list(range(40)) and (server.table == -1).all()
    assert example.shortfall(server, prompts, ids) <= 2 * 12 * 2.0 ** -8
    # each step answers a token and what held
    assert steps >= 14 - held


def test_a_window_holds_few_pages(example):
    # 150 tokens in pages of 16 under a window of 24: 3 pages and the sinks', not 10
    server = example.Server(layers=1, requests=1, pages=10, max_pages=12, window=24, sinks=4)
    seen = []
    keep = server.keep
    server.keep = lambda lens: (keep(lens), seen.append(10 - int(server.cursor[1] - server.cursor[0])))
    ids, *_ = example.speculate(server, [list(range(60))], 90)
    assert int(server.status.item()) == 0 and len(ids[0]) == 150
    assert max(seen[8:-1]) <= 4 and seen[-1] == 0


def test_drawn_answers_repeat(example):
    server = example.Server(layers=1, requests=3, pages=40, max_pages=12, norms=True)
    prompts = [[5, 9, 5, 9], [7], list(range(30))]
    first = example.speculate(server, prompts, 10, temperature=0.9, seed=4)
    assert example.speculate(server, prompts, 10, temperature=0.9, seed=4) == first
    assert example.speculate(server, prompts, 10, temperature=0.9, seed=5) != first
    assert int(server.status.item()) == 0
