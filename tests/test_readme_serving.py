"""README's step with drafts, a window and requests that end, run as it is
written: the calls answered by the oracle, without a GPU.  Requests that read
their prompt or bring nothing keep what they hold."""
import os
import re
from types import SimpleNamespace

import numpy as np
import pytest

import lossless_entropy_coded_dfc_amd as dfc
from oracle import paged as op
from oracle import verify as ov

torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def snippet():
    """The lines from the verification on."""
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = (b for b in blocks if "verify_drafts" in b)
    return block[block.index("verified ="):]


def verify_drafts(logits, cu_rows, drafts, uniforms, temperature=None):
    cu, got = cu_rows.tolist(), []
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        got.append(ov.request(logits[a:b].double().numpy(), drafts[a:b].tolist(), uniforms[a:b].tolist(), None,
                              float(temperature[r]))[:2] if b > a else (0, -1))
    accepted, tokens = zip(*got)
    return dfc.Verified(torch.tensor(accepted, dtype=torch.int32), torch.tensor(tokens))


def paged_release(held, keep, table, ring, cursor, shared, page_size, window=0, sinks=0):
    assert ((0 <= keep) & (keep <= held)).all(), (keep, held)     # or the request is passed over
    got = op.release(held.tolist(), keep.tolist(), table.numpy(), ring.numpy(), cursor.numpy(), shared.numpy(), page_size,
                     window, sinks)
    for t, x in zip((table, ring, shared), (got[0], got[1], got[3])):
        t.copy_(torch.from_numpy(x))
    return torch.from_numpy(got[2])


def test_lengths_and_pages():
    i32 = dict(dtype=torch.int32)
    page_size, width, pages = 16, 8, 40
    # held before; brought: a token and three drafts, a token and two, a token, a prompt's chunk, nothing, a token that ends it
    context = torch.tensor([30, 46, 20, 32, 47, 40], **i32)
    new = torch.tensor([4, 3, 1, 20, 0, 1], **i32)
    drafted = torch.tensor([3, 2, 0, 0, 0, 0], **i32)
    answers = [True, True, True, False, False, True]
    finished = torch.tensor([False] * 5 + [True])
    vocab, total = 50, int(new.sum())
    ring, shared = torch.arange(pages, **i32), torch.zeros(pages, **i32)
    table, cursor = torch.full((6, width), -1, **i32), np.array([0, pages])
    for n in (context, new):   # what is held, then the step
        before = torch.zeros_like(context) if n is context else context
        t, lens, cu, _, _, cursor = op.plan(before, n, table, ring, cursor, page_size, int(n.sum()))
        table = torch.from_numpy(t)
    plan = SimpleNamespace(seq_lens=torch.from_numpy(lens), cu_q=torch.from_numpy(cu), cursor=torch.from_numpy(cursor))
    rows = torch.tensor([i for r in range(6) if answers[r] for i in range(int(cu[r]), int(cu[r + 1]))])
    cu_rows = torch.tensor([0] + list(np.cumsum([int(n) if a else 0 for n, a in zip(new, answers)])), **i32)
    logits = torch.full((total, vocab), -10.0)
    logits[torch.arange(total), torch.arange(total) % vocab] = 10.0     # row i says token i
    drafts = rows % vocab
    drafts[[2, 4, 5]] = torch.tensor([49, 7, 8])   # the first request's third and the second's do not hold
    names = dict(dfc=SimpleNamespace(verify_drafts=verify_drafts, paged_release=paged_release), torch=torch, plan=plan,
                 context_lens=context, new_lens=new, logits=logits, rows=rows, cu_rows=cu_rows, drafts=drafts,
                 drafted=drafted, uniforms=torch.full((len(rows),), 0.5), temperature=torch.zeros(6), finished=finished,
                 block_table=table, free_pages=ring, shared=shared, page_size=page_size)
    exec(snippet(), names)
    kept = [30 + 1 + 2, 46 + 1, 20 + 1, 32 + 20, 47, 0]
    assert names["verified"].accepted.tolist() == [2, 0, 0, 0, 0, 0]
    assert names["context_lens"].tolist() == kept
    held = [int((row >= 0).sum()) for row in table]
    assert held == [-(-n // page_size) for n in kept]
    assert int(names["cursor"][1] - names["cursor"][0]) == pages - sum(held)
