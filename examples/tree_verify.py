"""A verify loop over drafted trees, end to end on the GPU: a small target with attention and MoE layers, a paged cache,
and a drafter that proposes a tree of tokens for each of several requests.

The prompts go in by chunks of some rows per request, all requests' rows packed:
  1. pages for the chunk's rows                        pages_reserve
  2. per layer: norm, one projection to q, k and v     (torch)
                norms per head, rotary positions,
                rows into the cache                    norm_rope_append
                the cached rows (later chunks)         cache_read
                causal attention of the rows           prompt_attention
                output projection, MoE block           (as below)

One step, in the order a serving loop runs it:
  1. pages for the trees' nodes                        pages_reserve
  2. per layer: norm, one projection to q, k and v     (torch)
                norms per head, rotary positions,
                rows into the cache                    norm_rope_append
                attention of the nodes                 tree_attention
                output projection, residual            (torch)
                MoE block                              moe_stack_forward
  3. logits under penalties, and their argmax          logits_process
  4. greedy walk of each tree                          accept_tree
  5. accepted rows together in every layer             cache_commit
Nothing in a step copies to the host: the lengths, page tables, counts and paths stay on the device.

Speculation must not change the text: the committed tokens are those that decoding one token at a time gives.  `main`
runs both and compares; the drafter here knows the plain decode's text and mixes wrong tokens in, so that paths of every
length occur.  With --codes the cache holds e4m3 codes with a power of two per token and head, half the bytes.

    python examples/tree_verify.py [--steps 12] [--requests 4] [--nodes 12] [--chunk 24] [--codes]
"""
from __future__ import annotations

import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_moe_gb300 import dfv, inputs  # noqa: E402

D_MODEL, HEADS, KV_HEADS, HEAD_DIM, LAYERS, VOCAB, PAGE = 512, 8, 2, 64, 2, 2048, 16


class Target:
    """Random weights of a small pre-norm model: attention (q and k normed per head) and MoE blocks in turn."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *shape, std=0.05: torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
        self.embed = w(VOCAB, D_MODEL, std=1.0)
        self.qkv = [w(D_MODEL, (HEADS + 2 * KV_HEADS) * HEAD_DIM) for _ in range(LAYERS)]
        self.proj = [w(HEADS * HEAD_DIM, D_MODEL) for _ in range(LAYERS)]
        shape = inputs.LayerShape(d=D_MODEL, n_experts=16, top_k=4, d_ff=128)
        self.moe = [dfv.Layer(inputs.make_layer(shape, seed + 1 + i, device="cuda")) for i in range(LAYERS)]
        self.moe_ws = dfv.alloc_workspace(dfv.workspace_size(self.moe[0], 16))
        self.rope = dfv.Rope(HEAD_DIM, theta=1e4)
        self.gains = [[1 + w(HEAD_DIM) for _ in range(2)] for _ in range(LAYERS)]

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def layers(self, cache, rows, tokens, positions, attention):
        """The residual stream behind the last layer [rows, D_MODEL]; the rows' keys and values are in the cache afterwards.
        attention(layer, q, k, v): over the rows just stored and what was there before."""
        x = self.embed[tokens.long()]
        n = x.shape[0]
        for i in range(LAYERS):
            qkv = (self.norm(x) @ self.qkv[i]).view(n, HEADS + 2 * KV_HEADS, HEAD_DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            q = dfv.norm_rope_append(cache, i, rows, self.rope, q, k, v, positions, q_gain=self.gains[i][0],
                                     k_gain=self.gains[i][1], k_out=k)
            o = attention(i, q, k, v)
            x = (x.float() + (o.view(n, -1) @ self.proj[i]).float()).to(torch.bfloat16)
            for r in range(0, n, 16):  # the residual stack takes blocks of 16 rows
                x[r:r + 16] = dfv.moe_stack_forward([self.moe[i]], x[r:r + 16].clone(), self.moe_ws)
        return x

    def verify(self, cache, tree, tokens, positions, ws):
        """Logits of every node [rows, VOCAB]."""
        rows = dfv.RowBatch(tree.row_off, tree.n_rows, tree.max_nodes)
        x = self.layers(cache, rows, tokens, positions, lambda i, q, k, v: dfv.tree_attention(cache, i, tree, q, ws))
        return (self.norm(x) @ self.embed.t()).float() * 0.05

    def prefill(self, cache, rows, keys, tokens, positions, ws):
        """A chunk of the prompts; keys: all cached rows with the chunk's, None while nothing was cached before."""
        def attention(i, q, k, v):
            if keys is not None:
                k, v = dfv.cache_read(cache, i, keys)
            return dfv.prompt_attention(rows, q, k, v, ws, keys=keys)
        self.layers(cache, rows, tokens, positions, attention)


class Server:
    """Requests with their own sequences of one cache."""

    def __init__(self, target, prompts, tokens_per_request, max_nodes, chunk=24, dtype=torch.bfloat16):
        self.t, self.S, self.N = target, len(prompts), max_nodes
        room = max(len(p) for p in prompts) + tokens_per_request + max_nodes
        width = -(-room // PAGE)
        self.cache = dfv.KVCache.empty(LAYERS, self.S * width + 1, PAGE, KV_HEADS, HEAD_DIM, self.S, width, dtype=dtype)
        self.pages_ws = dfv.alloc_workspace(dfv.cache_workspace_size(self.cache))
        self.attn_ws = None
        self.all = torch.arange(self.S, dtype=torch.int32, device="cuda")
        self.hist = torch.zeros(self.S, room + 1, dtype=torch.int32, device="cuda")
        self.hist_len = torch.zeros(self.S, dtype=torch.int32, device="cuda")
        self.prompt_len = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        pen = torch.full((self.S,), 1.2, device="cuda")
        self.rules = dfv.LogitRules(hist=self.hist, hist_len=self.hist_len, prompt_len=self.prompt_len, repetition=pen,
                                    frequency=torch.full((self.S,), 0.1, device="cuda"))
        self.logits_ws = dfv.alloc_workspace(dfv.logits_workspace_size(self.S * max(max_nodes, 64)))
        # prompts but for their last token, which is the first root
        done = [0] * self.S
        for start in range(0, max(len(p) for p in prompts) - 1, chunk):
            parts = [p[start:min(start + chunk, len(p) - 1)] for p in prompts]
            self.prefill(parts, done)
            done = [d + len(p) for d, p in zip(done, parts)]

    def space(self, nbytes):
        """One workspace for all attention calls, of chunks and of trees, made again only for a call that needs a larger one."""
        if self.attn_ws is None or self.attn_ws.numel() < nbytes:
            self.attn_ws = dfv.alloc_workspace(nbytes)
        return self.attn_ws

    @staticmethod
    def rows(counts):
        off = [0]
        for n in counts:
            off.append(off[-1] + n)
        return dfv.RowBatch(torch.tensor(off, dtype=torch.int32, device="cuda"), off[-1], max(counts))

    def prefill(self, parts, done):
        """Rows of prompts behind the first done[s] of each, which are in the cache."""
        dev = dict(dtype=torch.int32, device="cuda")
        rows = self.rows([len(p) for p in parts])
        keys = self.rows([d + len(p) for d, p in zip(done, parts)]) if any(done) else None
        toks = torch.tensor([x for p in parts for x in p], **dev)
        pos = torch.tensor([d + i for d, p in zip(done, parts) for i in range(len(p))], **dev)
        taken = torch.tensor([len(p) for p in parts], **dev)
        dfv.pages_reserve(self.cache, self.all, taken, self.pages_ws)
        ws = self.space(dfv.prompt_attention_workspace_size(rows, HEADS, KV_HEADS, HEAD_DIM))
        self.t.prefill(self.cache, rows, keys, toks, pos, ws)
        self.cache.lens += taken
        for s, (d, p) in enumerate(zip(done, parts)):
            self.hist[s, d:d + len(p)] = torch.tensor(p, **dev)
        self.hist_len += taken

    def batch(self, tokens, masks):
        """Tree descriptor, tokens and rotary positions of one call (trees built on the host, as a drafter would)."""
        off = [0]
        for t in tokens:
            off.append(off[-1] + len(t))
        dev = dict(dtype=torch.int32, device="cuda")
        flat = [m - (1 << 64) if m >> 63 else m for s in masks for m in s]
        tree = dfv.TreeBatch(torch.tensor(off, **dev), off[-1], max(len(t) for t in tokens),
                             mask=torch.tensor(flat, dtype=torch.int64, device="cuda"))
        depth = torch.tensor([bin(m).count("1") - 1 for s in masks for m in s], **dev)
        seq = torch.tensor([s for s, t in enumerate(tokens) for _ in t], device="cuda")
        return tree, torch.tensor([x for t in tokens for x in t], **dev), self.cache.lens[seq] + depth

    def reserve(self, n):
        dfv.pages_reserve(self.cache, self.all, torch.full_like(self.all, n), self.pages_ws)

    def run(self, tree, tokens, positions):
        ws = self.space(dfv.tree_attention_workspace_size(self.cache, tree, HEADS))
        return self.t.verify(self.cache, tree, tokens, positions, ws)

    def keep(self, tree, tokens, path, tau):
        """The accepted nodes' rows stay in the cache, their tokens join the history."""
        j = torch.arange(tree.max_nodes, device="cuda")
        on = j[None, :] < tau[:, None]
        row = (tree.row_off[:-1, None] + path.clamp_min(0)).long().clamp_max(tree.n_rows - 1)
        at = torch.where(on, self.hist_len[:, None] + j, self.hist.shape[1] - 1).long()
        self.hist.scatter_(1, at, torch.where(on, tokens[row], 0))
        self.hist_len += tau
        dfv.cache_commit(self.cache, tree, path, tau, self.pages_ws)

    def step(self, tokens, masks):
        """One verify step; (paths, tau, the target's tokens at every node)."""
        tree, toks, pos = self.batch(tokens, masks)
        self.reserve(tree.max_nodes)
        logits = self.run(tree, toks, pos)
        _, best = dfv.logits_process(logits, tree, toks, self.rules, self.logits_ws, store=False)
        path, tau = dfv.accept_tree(tree, toks, best)
        self.keep(tree, toks, path, tau)
        return path, tau, best, tree


def drafted_tree(root, right, n, rng):
    """A tree of n nodes under `root`: a backbone of tokens that are right until the drafter errs, and wrong branches."""
    tokens, masks, depth_of_right = [root], [1], {0: 0}
    tip, d = 0, 0
    while len(tokens) < n:
        i = len(tokens)
        if d < len(right) and rng.random() < 0.6:  # the next right token, now and then a wrong one in its place
            parent, tok = tip, right[d] if rng.random() < 0.85 else (right[d] + 1) % VOCAB
            tip, d = i, d + 1
        else:
            parent, tok = rng.randrange(i), rng.randrange(VOCAB)
        tokens.append(tok)
        masks.append(masks[parent] | 1 << i)
    return tokens, masks


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--nodes", type=int, default=12)
    ap.add_argument("--chunk", type=int, default=24, help="rows of a prompt per call")
    ap.add_argument("--codes", action="store_true", help="cache in e4m3 codes")
    a = ap.parse_args(argv)
    rng = random.Random(7)
    target = Target()
    prompts = [[rng.randrange(VOCAB) for _ in range(rng.randint(2, 40))] for _ in range(a.requests)]
    total = a.steps * a.nodes
    how = dict(chunk=a.chunk, dtype=torch.float8_e4m3fn if a.codes else torch.bfloat16)

    # one token at a time
    plain = Server(target, prompts, total, 1, **how)
    text = [[] for _ in prompts]
    roots = [p[-1] for p in prompts]
    for _ in range(total):
        _, _, best, _ = plain.step([[r] for r in roots], [[1]] * a.requests)
        roots = best.tolist()
        for t, r in zip(text, roots):
            t.append(r)

    # trees
    spec = Server(target, prompts, total, a.nodes, **how)
    got = [[] for _ in prompts]
    roots = [p[-1] for p in prompts]
    for _ in range(a.steps):
        trees = [drafted_tree(r, text[s][len(got[s]):], a.nodes, rng) for s, r in enumerate(roots)]
        path, tau, best, tree = spec.step([t for t, _ in trees], [m for _, m in trees])
        off, best = tree.row_off.tolist(), best.tolist()
        for s, (p, n) in enumerate(zip(path.tolist(), tau.tolist())):
            got[s] += [best[off[s] + i] for i in p[:n]]
            roots[s] = got[s][-1]
    assert spec.cache.errors() == 0 and plain.cache.errors() == 0
    same = sum(g == t[:len(g)] for g, t in zip(got, text))
    mean = sum(map(len, got)) / (a.steps * a.requests)
    print("%d of %d requests match plain decoding; %.2f tokens committed per step" % (same, a.requests, mean))
    dfv.pages_free(spec.cache, spec.all)
    return same, a.requests, mean


if __name__ == "__main__":
    main()
