"""Penalties, bias and grammar mask on the logits: the steps in fp32 bit for bit, the values against 64 bits, and the
argmax."""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

from tests._tree_util import HALF_STEP, chain_mask, signed, tree_masks

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


class Job:
    def __init__(self, V, nodes, dtype, seed=0, hist=40, rules=("repetition", "frequency", "presence"), bias=None,
                 allowed=None, prompt=True, chain=False, few=None):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        S = len(nodes)
        self.V, self.nodes, self.S, self.dtype = V, nodes, S, dtype
        self.off = [0]
        for n in nodes:
            self.off.append(self.off[-1] + n)
        self.rows = self.off[-1]
        self.x = (torch.randn(self.rows, V, generator=g) * 3).to(dtype)
        self.masks = None if chain else [m for n in nodes for m in tree_masks(n, rng)]
        few = few or V  # tokens from the first `few`: repeats
        self.tokens = torch.randint(0, few, (self.rows,), generator=g, dtype=torch.int32)
        self.hist = torch.randint(0, few, (S, hist), generator=g, dtype=torch.int32) if hist is not None else None
        if hist:
            self.hist[:, ::7] = self.tokens[torch.randint(0, self.rows, (S, 1), generator=g)]
            self.hist[0, 0], self.hist[-1, -1] = -1, V  # ids outside the vocabulary
        self.hist_len = None if hist is None else torch.tensor([rng.randint(0, hist) if s else hist for s in range(S)], dtype=torch.int32)
        self.prompt_len = self.hist_len // 2 if prompt and hist is not None else None
        self.pen = {k: (1 + torch.rand(S, generator=g) if k == "repetition" else torch.randn(S, generator=g)) for k in rules}
        self.bias = None if bias is None else torch.randn(bias, V, generator=g)
        W = (V + 31) // 32
        self.allowed = None if allowed is None else torch.randint(-2 ** 31, 2 ** 31, (allowed, W), generator=g, dtype=torch.int64).to(torch.int32)

    def gpu(self, dfv):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        m = None if self.masks is None else torch.tensor([signed(x) for x in self.masks], dtype=torch.int64).cuda()
        tree = dfv.TreeBatch(torch.tensor(self.off, dtype=torch.int32).cuda(), self.rows, max(max(self.nodes), 1), mask=m)
        rules = dfv.LogitRules(hist=c(self.hist), hist_len=c(self.hist_len), prompt_len=c(self.prompt_len), bias=c(self.bias),
                               allowed=c(self.allowed), **{k: c(v) for k, v in self.pen.items()})
        return tree, rules, c(self.x), c(self.tokens)

    def steps(self, wide):
        """The values in `wide` arithmetic (numpy rounds each operation), and the sum of the magnitudes met."""
        out = np.zeros((self.rows, self.V), wide)
        mag = np.zeros((self.rows, self.V))
        for s in range(self.S):
            gen, seen = np.zeros(self.V, np.int64), np.zeros(self.V, bool)
            if self.hist is not None:
                P = 0 if self.prompt_len is None else int(self.prompt_len[s])
                for i, t in enumerate(self.hist[s, :int(self.hist_len[s])].tolist()):
                    if 0 <= t < self.V:
                        seen[t] = True
                        gen[t] += i >= P
            for i in range(self.nodes[s]):
                r = self.off[s] + i
                m = chain_mask(i) if self.masks is None else self.masks[r]
                c, met = gen.copy(), seen.copy()
                for j in range(self.nodes[s]):
                    if m >> j & 1:
                        c[int(self.tokens[self.off[s] + j])] += 1
                        met[int(self.tokens[self.off[s] + j])] = True
                x = self.x[r].float().numpy().astype(wide)
                a = np.abs(x).astype(np.float64)
                if "repetition" in self.pen:
                    k = wide(self.pen["repetition"][s].item())
                    x = np.where(met, np.where(x > 0, x / k, x * k), x)
                    a += np.abs(x)
                if "frequency" in self.pen:
                    y = wide(self.pen["frequency"][s].item()) * c.astype(wide)
                    x = x - y
                    a += np.abs(y)
                if "presence" in self.pen:
                    k = wide(self.pen["presence"][s].item())
                    x = np.where(c > 0, x - k, x)
                    a += abs(float(k))
                if self.bias is not None:
                    b = self.bias[s if self.bias.shape[0] > 1 else 0].numpy().astype(wide)
                    x = x + b
                    a += np.abs(b)
                if self.allowed is not None:
                    w = self.allowed[r if self.allowed.shape[0] > 1 else 0].numpy().view(np.uint32)
                    ok = (w[np.arange(self.V) // 32] >> (np.arange(self.V) % 32).astype(np.uint32)) & 1
                    x = np.where(ok == 1, x, wide(-np.inf))
                out[r], mag[r] = x, a
        return out, mag


def check(job: Job, out, best):
    x32 = torch.from_numpy(job.steps(np.float32)[0]).to(job.dtype)
    assert torch.equal(out.cpu(), x32)
    x64, mag = job.steps(np.float64)
    fin = np.isfinite(x64)
    half = HALF_STEP[job.dtype]
    tol = half * np.abs(np.where(fin, x64, 0)) * (1 + 1e-6) + 5 * 2.0 ** -24 * mag
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), fin)
    assert (np.abs(got - np.where(fin, x64, 0))[fin] <= tol[fin]).all()
    want = np.argmax(x32.float().numpy(), axis=1)  # first of equals
    assert np.array_equal(best.cpu().numpy(), want)


def run(dfv, job, **kw):
    tree, rules, x, tokens = job.gpu(dfv)
    ws = dfv.alloc_workspace(dfv.logits_workspace_size(job.rows))
    out, best = dfv.logits_process(x, tree, tokens, rules, ws, **kw)
    torch.cuda.synchronize()
    assert not bool(ws.any())  # ready for the next call
    return out, best


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 1000, 1024, 4097, 32003, 50280])
def test_vocabulary_sizes(dfv, dtype, V):
    job = Job(V, [5, 1, 9], dtype, seed=V, bias=3, allowed=15, few=max(1, V // 3))
    check(job, *run(dfv, job))


@pytest.mark.parametrize("rules", [(), ("repetition",), ("frequency",), ("presence",), ("repetition", "frequency", "presence")])
@pytest.mark.parametrize("bias,allowed", [(None, None), (1, None), (None, 1), (2, 7)])
def test_each_rule(dfv, rules, bias, allowed):
    job = Job(2049, [3, 4], BF, seed=11, rules=rules, bias=bias, allowed=allowed, few=200)
    check(job, *run(dfv, job))


@pytest.mark.parametrize("nodes", [[1], [64], [16] * 8, [0, 3, 0, 64, 1], [2] * 50])
@pytest.mark.parametrize("chain", [False, True])
def test_trees(dfv, nodes, chain):
    job = Job(3000, nodes, F32, seed=12, chain=chain, few=20)
    check(job, *run(dfv, job))


@pytest.mark.parametrize("hist", [None, 0, 1, 5000])
def test_histories(dfv, hist):
    job = Job(640, [4, 2], BF, seed=13, hist=hist, prompt=hist != 1, few=300)
    check(job, *run(dfv, job))


def test_whole_vocabulary(dfv):
    job = Job(151936, [4, 3], BF, seed=14, hist=3000, bias=2, allowed=7, few=2000)
    check(job, *run(dfv, job))


def test_ties_go_to_the_lowest_index_and_nothing_allowed_gives_zero(dfv):
    job = Job(9000, [4], BF, seed=15, rules=(), allowed=4)
    job.x[:] = 0.25
    job.x[1, ::2] = -0.0
    job.allowed[0] = -1
    job.allowed[1] = -1
    job.allowed[2] = 0
    job.allowed[3] = 0
    job.allowed[3, 200] = 1 << 5
    out, best = run(dfv, job)
    check(job, out, best)
    assert best.tolist()[2:] == [0, 6405]
    assert bool((out[2] == -math.inf).all())


def test_infinite_logits(dfv):
    job = Job(500, [3], F32, seed=16, rules=("repetition",), few=500)
    job.x[0, 3], job.x[1, 4], job.x[2] = math.inf, -math.inf, -math.inf
    job.x[2, 77] = torch.finfo(F32).min
    check(job, *run(dfv, job))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_strides_and_argmax_only(dfv, dtype):
    for V, pad, shift in ((1000, 8, 0), (1001, 0, 0), (997, 3, 1), (4000, 1, 3)):
        job = Job(V, [6, 2], dtype, seed=V, bias=2, allowed=8, few=50)
        tree, rules, x, tokens = job.gpu(dfv)
        ws = dfv.alloc_workspace(dfv.logits_workspace_size(job.rows))
        wide = torch.full((job.rows, V + pad + shift), 9.0, dtype=dtype, device="cuda")
        view = wide[:, shift:shift + V]
        view.copy_(x)
        none, best = dfv.logits_process(view, tree, tokens, rules, ws, store=False)
        assert none is None
        out, again = dfv.logits_process(view, tree, tokens, rules, ws)
        check(job, out, best)
        assert torch.equal(best, again)
        # another alignment of the output than of the input
        other = torch.full((job.rows, V + 13), 9.0, dtype=dtype, device="cuda")
        got, third = dfv.logits_process(view, tree, tokens, rules, ws, out=other[:, 5:5 + V])
        check(job, got, third)
        assert bool((other[:, :5] == 9).all()) and bool((other[:, 5 + V:] == 9).all())
        same, best = dfv.logits_process(view, tree, tokens, rules, ws, out=view)
        check(job, same, best)
        assert bool((wide[:, :shift] == 9).all()) and bool((wide[:, shift + V:] == 9).all())


def test_repeatable_in_a_graph(dfv):
    job = Job(5000, [16, 16], BF, seed=17, few=40)
    tree, rules, x, tokens = job.gpu(dfv)
    ws = dfv.alloc_workspace(dfv.logits_workspace_size(job.rows))
    out, best = dfv.logits_process(x, tree, tokens, rules, ws)
    o2, b2 = torch.empty_like(out), torch.empty_like(best)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfv.logits_process(x, tree, tokens, rules, ws, out=o2, argmax=b2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(best, b2)


def test_a_chain_feeds_greedy_acceptance(dfv):
    """argmax and the acceptance of a chain agree with dfv_accept_greedy on the stored logits."""
    job = Job(2000, [9], BF, seed=18, chain=True, few=100)
    out, best = run(dfv, job)
    draft = best[:-1].clone()
    draft[5] = (draft[5] + 1) % 2000
    aws = dfv.alloc_workspace(dfv.accept_workspace_size(16, 2000))
    tau, com = dfv.accept_greedy(out, draft, aws)
    tree = dfv.TreeBatch(torch.tensor([0, 9], dtype=torch.int32).cuda(), 9, 9)
    tokens = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), draft])
    path, t2 = dfv.accept_tree(tree, tokens, best)
    torch.cuda.synchronize()
    assert int(tau) == int(t2[0]) == 6
    assert path[0].tolist() == [0, 1, 2, 3, 4, 5, -1, -1, -1]
    assert com[:6].tolist() == best[path[0, :6].long()].tolist()
