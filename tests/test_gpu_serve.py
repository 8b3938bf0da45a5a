"""GPU: the serving example (examples/serve.py): products on compressed
weights, the plan, the append and the attention together over many steps,
against every request recomputed at once with resident weights and plain
attention in fp32.  The logits differ by roundings to bfloat16 that fall
differently (2^-8 a value, a dozen on a token's way through two layers)."""
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
    spec = importlib.util.spec_from_file_location("serve_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_prompts_in_chunks_and_answers_match_the_whole(example):
    server = example.Server(layers=2, requests=5, pages=40, max_pages=12)
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, 512, n).tolist() for n in (1, 16, 17, 40, 90)]
    ids, last = example.serve(server, prompts, 12)
    torch.cuda.synchronize()
    assert int(server.status.item()) == 0
    held = [len(i) - 1 for i in ids]
    assert server.context.tolist() == held
    # every page taken off the ring stands once in the table
    taken = int(server.cursor[0])
    assert taken == sum(-(-n // 16) for n in held)
    pages = server.table[server.table >= 0].tolist()
    assert sorted(pages) == sorted(server.free[:taken].tolist())
    for i, logits in zip(ids, last):
        ref = server.reference(i[:-1])[-1]
        assert float((logits - ref).norm() / ref.norm()) <= 12 * 2.0 ** -8


def test_running_out_of_pages_is_told(example):
    server = example.Server(layers=1, requests=2, pages=3, max_pages=4)
    example.serve(server, [list(range(40)), list(range(30))], 4)
    torch.cuda.synchronize()
    assert int(server.status.item()) != 0
