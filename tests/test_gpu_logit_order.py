"""Which column a row's argmax is when CTAs, slices and warps find their best in any order, and the paths of aligned and
unaligned histories and biases."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_logit_rules import BF, F32, Job, check, dfv, run  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(kind, rows, V, g):
    """Values that both types hold exactly."""
    c = torch.arange(V)
    if kind == "rising":  # each best is in a later slice, 128 columns share it
        x = (c // 128 % 256).float().expand(rows, V)
    elif kind == "falling":
        x = -(c // 128 % 256).float().expand(rows, V)
    elif kind == "flat":
        x = torch.full((rows, V), -1.5)
    elif kind == "zeros":  # +0 and -0 are equal
        x = torch.where(c % 2 == 0, -0.0, 0.0).expand(rows, V)
    elif kind == "twice":  # two equal peaks anywhere
        x = torch.randint(-9, 9, (rows, V), generator=g).float()
        for r in range(rows):
            x[r, torch.randint(0, V, (2,), generator=g)] = 20.0
    else:  # one column that is not -inf
        x = torch.full((rows, V), -torch.inf)
        for r in range(rows):
            if r % 3:
                x[r, torch.randint(0, V, (1,), generator=g)] = -2.0 ** 100
    return x.contiguous()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [20488, 20483])
@pytest.mark.parametrize("nodes", [[1], [2, 64, 5], [16] * 40])
@pytest.mark.parametrize("kind", ["rising", "falling", "flat", "zeros", "twice", "one"])
def test_argmax_is_the_first_of_equals(dfv, dtype, V, nodes, kind):  # noqa: F811
    rows, off = sum(nodes), [0]
    for n in nodes:
        off.append(off[-1] + n)
    x = rows_of(kind, rows, V, torch.Generator().manual_seed(V)).to(dtype)
    tree = dfv.TreeBatch(torch.tensor(off, dtype=torch.int32).cuda(), rows, max(nodes))
    ws = dfv.alloc_workspace(dfv.logits_workspace_size(rows))
    want = np.argmax(x.float().numpy(), axis=1)
    # penalties that change nothing: the listed columns are found apart from the others
    same = dict(hist=torch.randint(0, V, (len(nodes), 100), dtype=torch.int32).cuda(),
                hist_len=torch.full((len(nodes),), 100, dtype=torch.int32).cuda(), presence=torch.zeros(len(nodes)).cuda())
    tokens = torch.randint(0, V, (rows,), dtype=torch.int32).cuda()
    for rules in ({}, same):
        for _ in range(3):
            out, best = dfv.logits_process(x.cuda(), tree, tokens, dfv.LogitRules(**rules), ws)
            assert np.array_equal(best.cpu().numpy(), want)
            assert torch.equal(out.cpu(), x)
    assert not bool(ws.any())


@pytest.mark.parametrize("hist", [2, 3, 5, 6, 7, 2047, 2050, 4099])
def test_widths_of_a_history(dfv, hist):  # noqa: F811
    """Rows of a history that start anywhere within 16 bytes, counted from quads and single tokens."""
    job = Job(8200, [3, 2, 4, 1, 2], BF, seed=hist, hist=hist, few=900)
    check(job, *run(dfv, job))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [8200, 8201])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_bias_at_any_word(dfv, dtype, V, shift):  # noqa: F811
    """Rows of a bias that start at any multiple of four bytes."""
    job = Job(V, [3, 2, 1], dtype, seed=shift, bias=3, allowed=6, few=900)
    tree, rules, x, tokens = job.gpu(dfv)
    room = torch.zeros(3 * V + 8, device="cuda")
    at = (-room.data_ptr() // 4 + shift) % 4
    view = room[at:at + 3 * V].view(3, V)
    view.copy_(job.bias)
    rules = dfv.LogitRules(hist=job.hist.cuda(), hist_len=job.hist_len.cuda(), prompt_len=job.prompt_len.cuda(), bias=view,
                           allowed=job.allowed.cuda(), **{k: v.cuda() for k, v in job.pen.items()})
    ws = dfv.alloc_workspace(dfv.logits_workspace_size(job.rows))
    out, best = dfv.logits_process(x, tree, tokens, rules, ws)
    check(job, out, best)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [32008, 32003])
@pytest.mark.parametrize("hist", [None, 30, 6000])
def test_many_single_rows(dfv, dtype, V, hist):  # noqa: F811
    """One row a sequence, more slices of them than CTAs run at once."""
    job = Job(V, [1] * 45, dtype, seed=V + (hist or 0), hist=hist, bias=45, allowed=45, few=700)
    check(job, *run(dfv, job))
