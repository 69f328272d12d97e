"""Operators of a tree-verify step around the MoE layers: the cases that are measured and their plain forms.

The verify step of speculative decoding with a TREE of drafted tokens: the rows of all trees get their rotary positions and
enter the paged cache (rope), attend to the cache and to their own ancestors (attention), their logits get penalties, biases
and grammar masks (logits), the greedy walk picks the accepted path whose cache rows are compacted in every layer (commit),
and sequences are dropped and forked (fork).

`own` false: elementary torch operations, in 32 bits (64 for angles), rounded once.  `own` true: the framework's calls.
Nodes of a tree are numbered parents first; bit j of a node's mask is set for its ancestors and itself.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request: the step between two drafts, latency only
        dict(name="rope decode", op="rope", seqs=1, nodes=1, ctx=4097, heads=32, kv=4, dim=128, rot=128, inter=False,
             theta=1e6, scaling="none", factor=1.0, page=16, dtype="bf16"),
        # 32 requests with trees of up to 64 nodes, half of the head rotated, positions stretched by bands
        dict(name="rope batch bands", op="rope", seqs=32, nodes=64, ctx=2039, heads=32, kv=4, dim=128, rot=64, inter=True,
             theta=1e4, scaling="bands", factor=8.0, page=16, dtype="f16"),
        # one token of one request over a short cache
        dict(name="attn decode", op="attn", seqs=1, nodes=1, ctx=1021, heads=32, kv=4, dim=128, page=16, dtype="bf16", chain=True),
        # the same over a long document, narrow heads, larger pages
        dict(name="attn long decode", op="attn", seqs=1, nodes=1, ctx=131071, heads=32, kv=8, dim=64, page=64, dtype="f16", chain=True),
        # a verify block of 16 positions of one request, ordinary chat
        dict(name="attn block", op="attn", seqs=1, nodes=16, ctx=8191, heads=32, kv=4, dim=128, page=16, dtype="bf16", chain=True),
        # 32 requests with 16-node trees and ragged lengths
        dict(name="attn batch", op="attn", seqs=32, nodes=16, ctx=8191, heads=32, kv=4, dim=128, page=16, dtype="bf16", chain=False),
        # 8 requests with trees of 64 nodes over long caches: the largest
        dict(name="attn wide trees", op="attn", seqs=8, nodes=64, ctx=32749, heads=32, kv=4, dim=128, page=32, dtype="bf16", chain=False),
        # the logits of one token with penalties over a short history
        dict(name="logits decode", op="logits", seqs=1, nodes=1, vocab=151936, hist=509, dtype="bf16", rep=True, bias=False,
             grammar=False),
        # every row of 32 requests with 16 nodes, all steps on
        dict(name="logits batch", op="logits", seqs=32, nodes=16, vocab=151936, hist=4093, dtype="bf16", rep=True, bias=True,
             grammar=True),
        # one request accepts part of its 16-node tree; a small model's cache
        dict(name="commit one", op="commit", seqs=1, nodes=16, ctx=1021, accept=5, layers=8, kv=4, dim=128, page=16, dtype="bf16"),
        # 32 requests with 64-node trees commit their paths in all of 40 layers
        dict(name="commit batch", op="commit", seqs=32, nodes=64, ctx=47, accept=9, layers=40, kv=4, dim=128, page=16, dtype="bf16"),
        # beams: 12 losing sequences are dropped, the 4 winners are forked into their places
        dict(name="fork beams", op="fork", seqs=4, forks=12, ctx=509, layers=40, kv=4, dim=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "logits", "commit", "fork"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    if op == "rope":
        seqs, nodes = _log(rng, 1, 32), _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, nodes=nodes, ctx=_log(rng, 1, min(131072, 65536 // seqs)), heads=kv * rng.randint(1, 32 // kv),
                    kv=min(kv, 4), dim=dim, rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5, theta=rng.choice([1e4, 1e6]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands"]), factor=float(rng.randint(2, 16)), page=page,
                    dtype=rng.choice(["bf16", "f16"])) if kv <= 4 else draw(rng)
    if op == "attn":
        seqs, nodes = _log(rng, 1, 32), _log(rng, 1, 64)
        group = rng.choice([1, 2, 4, 5, 7, 8]) if kv <= 4 else rng.choice([1, 2, 4])
        # no more keys than the largest case in all, no more products either
        most = int(min(262144 // (seqs * max(1, kv // 4)), 64 * 8 * 32749 * 32 // (seqs * nodes * kv * group)))
        return dict(op=op, seqs=seqs, nodes=nodes, ctx=_log(rng, 1, min(131072, max(1, most))), heads=kv * group, kv=kv, dim=dim,
                    page=page, dtype=rng.choice(["bf16", "f16"]), chain=rng.random() < 0.4)
    if op == "logits":
        return dict(op=op, seqs=_log(rng, 1, 32), nodes=_log(rng, 1, 16), vocab=rng.choice([1024, 32003, 128256, 151936]),
                    hist=_log(rng, 1, 8192), dtype=rng.choice(["bf16", "f32"]) if rng.random() < 0.6 else "bf16",
                    rep=rng.random() < 0.7, bias=rng.random() < 0.5, grammar=rng.random() < 0.5)
    if op == "commit":
        nodes = _log(rng, 1, 64)
        return dict(op=op, seqs=_log(rng, 1, 32), nodes=nodes, ctx=rng.randint(1, 64), accept=rng.randint(1, min(nodes, 9)),
                    layers=_log(rng, 1, 40), kv=min(kv, 4), dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))
    return dict(op=op, seqs=rng.randint(1, 4), forks=rng.randint(1, 12), ctx=_log(rng, 1, 509), layers=_log(rng, 1, 40),
                kv=min(kv, 4), dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))


# ---------------------------------------------------------------- what a case fixes
def _lens(c):
    """Committed tokens of each sequence: ctx, then shorter ones down to about half."""
    return [c["ctx"] - (s * 389) % (c["ctx"] // 2 + 1) for s in range(c["seqs"])]


def _nodes(c):
    """Nodes of each sequence: the full tree, then smaller ones down to half."""
    return [c["nodes"] - (s * 5) % (c["nodes"] // 2 + 1) for s in range(c["seqs"])]


def _accepts(c):
    """Accepted nodes of each sequence, the root included."""
    return [min(n, 1 + (c["accept"] - 1 + s) % c["accept"]) for s, n in enumerate(_nodes(c))]


def _fork_sources(c):
    return [(f * f + f) % c["seqs"] for f in range(c["forks"])]


# ---------------------------------------------------------------- prepare
def _trees(c, rng, chain=False, accepts=None):
    """Random trees, parents first: masks and, with `accepts`, an accepted path of that many nodes in each."""
    masks, paths, parents = [], [], []
    for s, n in enumerate(_nodes(c)):
        path = sorted([0] + rng.sample(range(1, n), accepts[s] - 1)) if accepts else []
        up = {b: a for a, b in zip(path, path[1:])}
        m, par = [], []
        for i in range(n):
            p = -1 if i == 0 else i - 1 if chain else up.get(i, rng.randint(max(0, i - 6), i - 1))
            par.append(p)
            m.append((m[p] if p >= 0 else 0) | (1 << i))
        masks += m
        parents.append(par)
        paths.append(path)
    signed = [m - (1 << 64) if m >> 63 else m for m in masks]
    return torch.tensor(signed, dtype=torch.int64, device=DEV), paths, parents


def _offsets(c):
    off = [0]
    for n in _nodes(c):
        off.append(off[-1] + n)
    return off


def _pages(c, rng, spare=0, rows=0):
    """Page tables over shuffled pages: room for every committed token and the tree's nodes; `rows` empty rows more."""
    need = [-(-(a + b) // c["page"]) for a, b in zip(_lens(c), _nodes(c))] if "nodes" in c else [-(-a // c["page"]) for a in _lens(c)]
    order = list(range(sum(need) + spare))
    rng.shuffle(order)
    table = torch.full((c["seqs"] + rows, max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return table.to(DEV), len(order)


def _normal(shape, dtype, g):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


def prepare(case, seed):
    c = case
    rng = random.Random(seed * 1000003 + 17)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = {"case": c, "op": c["op"]}
    dt = DT[c["dtype"]]
    if c["op"] == "logits":
        rows = _offsets(c)[-1]
        S, V = c["seqs"], c["vocab"]
        st["row_off"], st["rows"], st["most"] = ints(_offsets(c)), rows, max(_nodes(c))
        st["mask"], _, _ = _trees(c, rng)
        st["logits"] = (torch.empty(rows, V, device=DEV).normal_(generator=g) * 2).to(dt)
        # text repeats itself: tokens are taken from the head of a long-tailed distribution
        tail = lambda shape: (V * torch.rand(shape, generator=g, device=DEV) ** 3).to(torch.int32)  # noqa: E731
        st["tokens"], st["hist"] = tail((rows,)), tail((S, c["hist"]))
        st["hist_len"] = ints([c["hist"] - (s * 7) % (c["hist"] // 2 + 1) for s in range(S)])
        st["prompt_len"] = st["hist_len"] // 2
        if c["rep"]:
            st["repetition"] = 1 + 0.5 * torch.rand(S, generator=g, device=DEV)
            st["frequency"] = torch.rand(S, generator=g, device=DEV) - 0.2
            st["presence"] = torch.rand(S, generator=g, device=DEV) - 0.2
        if c["bias"]:
            st["bias"] = torch.empty(S, V, device=DEV).normal_(generator=g)
        if c["grammar"]:
            st["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (rows, -(-V // 32)), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        if own:
            from speculative_decoding_moe_gb300 import dfv
            st["tree"] = dfv.TreeBatch(st["row_off"], rows, st["most"], mask=st["mask"])
            st["pen"] = dfv.LogitRules(**{k: st.get(k) for k in ("hist", "hist_len", "prompt_len", "repetition", "frequency",
                                                                "presence", "bias", "allowed")})
            st["ws"] = dfv.alloc_workspace(dfv.logits_workspace_size(rows))
        return st

    # a paged cache: [layers][pages][kv heads][tokens of a page][dim]
    layers = c.get("layers", 1)
    if c["op"] == "fork":
        st["table"], pages = _pages(c, rng, spare=2 * c["forks"] + 3, rows=c["forks"])
        st["lens"] = torch.cat([ints(_lens(c)), torch.zeros(c["forks"], dtype=torch.int32, device=DEV)])
        st["src"], st["dst"] = ints(_fork_sources(c)), ints([c["seqs"] + f for f in range(c["forks"])])
        st["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        st["refs"][st["table"][st["table"] >= 0].long()] = 1
    else:
        st["table"], pages = _pages(c, rng)
        st["lens"] = ints(_lens(c))
    shape = (layers, pages, c["kv"], c["page"], c["dim"])
    st["k"], st["v"] = _normal(shape, dt, g), _normal(shape, dt, g)
    if c["op"] != "fork":
        rows = _offsets(c)[-1]
        st["row_off"], st["rows"], st["most"] = ints(_offsets(c)), rows, max(_nodes(c))
    if c["op"] == "commit":
        accepts = _accepts(c)
        st["mask"], paths, parents = _trees(c, rng, accepts=accepts)
        # a tree's tokens are all different; the target repeats the drafted token along the accepted path only
        tokens, target = [], []
        for s, n in enumerate(_nodes(c)):
            t = rng.sample(range(100000), n + 1)
            want = [t[n]] * n
            for a, b in zip(paths[s], paths[s][1:]):
                want[a] = t[b]
            tokens += t[:n]
            target += want
        st["tokens"], st["target"] = ints(tokens), ints(target)
    if c["op"] in ("rope", "attn"):
        chain = c.get("chain", False)
        st["mask"], _, _ = _trees(c, rng, chain=chain)
        if c["op"] == "rope":
            # q, k and v as a projection leaves them: one row of all heads
            st["qkv"] = _normal((rows, c["heads"] + 2 * c["kv"], c["dim"]), dt, g)
            depth = [bin(m & (2 ** 64 - 1)).count("1") - 1 for m in st["mask"].tolist()]
            off = _offsets(c)
            st["positions"] = ints([a + depth[r] for s, a in enumerate(_lens(c)) for r in range(off[s], off[s + 1])])
        else:
            st["q"] = _normal((rows, c["heads"], c["dim"]), dt, g)
            if chain:
                st["mask"] = None
    if own:
        from speculative_decoding_moe_gb300 import dfv
        st["cache"] = dfv.KVCache(st["k"], st["v"], st["table"], st["lens"], refs=st.get("refs"))
        if c["op"] != "fork":
            st["tree"] = dfv.TreeBatch(st["row_off"], st["rows"], st["most"], mask=st["mask"])
        if c["op"] == "rope":
            st["rope"] = dfv.Rope(c["dim"], rot_dim=c["rot"], theta=c["theta"], interleaved=c["inter"], scaling=c["scaling"],
                                  factor=c["factor"], original=4096)
        if c["op"] == "attn":
            st["ws"] = dfv.alloc_workspace(dfv.tree_attention_workspace_size(st["cache"], st["tree"], c["heads"]))
        if c["op"] in ("commit", "fork"):
            st["ws"] = dfv.alloc_workspace(dfv.cache_workspace_size(st["cache"]))
    return st


# ---------------------------------------------------------------- run
def run(state):
    return {"rope": _rope, "attn": _attn, "logits": _logits, "commit": _commit, "fork": _fork}[state["op"]](state)


def _rows(st):
    """Sequence and node of each row."""
    r = torch.arange(st["rows"], device=DEV, dtype=torch.int32)
    s = torch.searchsorted(st["row_off"], r, right=True) - 1
    return s, r.long() - st["row_off"].long()[s]


def _bits(st, n):
    """[rows, n] truth values: the nodes that each row's mask holds."""
    if st["mask"] is None:
        _, i = _rows(st)
        return torch.arange(n, device=DEV)[None, :] <= i[:, None]
    return ((st["mask"][:, None] >> torch.arange(n, device=DEV)[None, :]) & 1).bool()


def _freqs(c):
    """Angular step of each pair, in 64 bits."""
    r = c["rot"]
    theta = c["theta"] * (c["factor"] ** (r / (r - 2)) if c["scaling"] == "ntk" else 1.0)
    f = theta ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "bands":  # turns over the original context, between 1 and 32
        ramp = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = (1 - ramp) * f / c["factor"] + ramp * f
    return f, (0.1 * math.log(c["factor"]) + 1 if c["scaling"] == "bands" else 1.0)


def _rope(st):
    c = st["case"]
    H, K = c["heads"], c["kv"]
    q, k, v = st["qkv"][:, :H], st["qkv"][:, H:H + K], st["qkv"][:, H + K:]
    if own:
        from speculative_decoding_moe_gb300 import dfv
        out = dfv.rope_append(st["cache"], 0, st["tree"], st["rope"], q, k, v, st["positions"])
        return {"q": out, "k": st["k"], "v": st["v"]}
    f, scale = _freqs(c)
    angle = st["positions"].double()[:, None] * f[None, :]
    cos, sin = (angle.cos() * scale).float()[:, None, :], (angle.sin() * scale).float()[:, None, :]

    def turn(x):
        x, r = x.float(), c["rot"]
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
        y, z = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y, z], -1).flatten(-2) if c["inter"] else torch.cat([y, z], -1)
        return torch.cat([y, x[..., r:]], -1).to(DT[c["dtype"]])

    s, i = _rows(st)
    at = st["lens"].long()[s] + i
    page = st["table"][s, at // c["page"]].long()
    st["k"][0, page, :, at % c["page"]] = turn(k)
    st["v"][0, page, :, at % c["page"]] = v
    return {"q": turn(q), "k": st["k"], "v": st["v"]}


def _attn(st):
    c = st["case"]
    if own:
        from speculative_decoding_moe_gb300 import dfv
        lse = torch.empty(st["rows"], c["heads"], device=DEV)
        return {"o": dfv.tree_attention(st["cache"], 0, st["tree"], st["q"], st["ws"], lse=lse), "lse": lse}
    return _attend(st, torch.float32, DT[c["dtype"]])


def _attend(st, wide, to):
    """Padded to the longest sequence and the largest tree."""
    c = st["case"]
    S, N, K, G, D = c["seqs"], st["most"], c["kv"], c["heads"] // c["kv"], c["dim"]
    s, i = _rows(st)
    table = st["table"].long().clamp_min(0)
    T = table.shape[1] * c["page"]
    k = st["k"][0][table].permute(0, 2, 1, 3, 4).reshape(S, K, T, D).to(wide)
    v = st["v"][0][table].permute(0, 2, 1, 3, 4).reshape(S, K, T, D).to(wide)
    q = torch.zeros(S, N, K, G, D, dtype=wide, device=DEV)
    q[s, i] = st["q"].to(wide).reshape(-1, K, G, D)
    lens = st["lens"].long()
    key = torch.arange(T, device=DEV)[None, :] - lens[:, None]  # below 0: committed, then the node's number
    bits = torch.zeros(S, N, N, dtype=torch.bool, device=DEV)
    bits[s, i] = _bits(st, N)
    node = key.clamp(0, N - 1)[:, None, :].expand(S, N, T)
    seen = (key < 0)[:, None, :] | ((key < N)[:, None, :] & bits.gather(2, node))
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(S, K, N * G, D), k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    x = x.reshape(S, K, N, G, T).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    den = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(S, K, N * G, T), v).reshape(S, K, N, G, D)
    o = torch.where(den > 0, o / den, torch.zeros_like(o))
    lse = top + den.log()
    o = o.permute(0, 2, 1, 3, 4).reshape(S, N, K * G, D)[s, i]
    return {"o": o.to(to), "lse": lse.permute(0, 2, 1, 3, 4).reshape(S, N, K * G)[s, i]}


def _logits(st):
    c = st["case"]
    if own:
        from speculative_decoding_moe_gb300 import dfv
        out, best = dfv.logits_process(st["logits"], st["tree"], st["tokens"], st["pen"], st["ws"])
        return {"logits": out, "best": best}
    x = _ruled(st, torch.float32).to(DT[c["dtype"]])
    top = x.amax(-1, keepdim=True)  # ties: the lowest index
    at = torch.where(x == top, torch.arange(c["vocab"], device=DEV, dtype=torch.int32), c["vocab"])
    return {"logits": x, "best": at.amin(-1)}


def _ruled(st, wide):
    c = st["case"]
    V, N = c["vocab"], st["most"]
    s, i = _rows(st)
    x = st["logits"].to(wide)
    if c["rep"]:
        at = torch.arange(c["hist"], device=DEV)[None, :]
        there = at < st["hist_len"][:, None]
        count = lambda w: torch.zeros(c["seqs"], V, dtype=torch.int32, device=DEV).scatter_add_(1, st["hist"].long(), w.int())  # noqa: E731
        seen = count(there) > 0
        cnt = count(there & (at >= st["prompt_len"][:, None]))[s]  # generated tokens only
        # and the drafted tokens on the row's own path
        padded = torch.zeros(c["seqs"], N, dtype=torch.int64, device=DEV)
        padded[s, i] = st["tokens"].long()
        cnt.scatter_add_(1, padded[s], _bits(st, N).int())
        met = seen[s] | (cnt > 0)
        r, f, p = (st[k].to(wide)[s][:, None] for k in ("repetition", "frequency", "presence"))
        x = torch.where(met, torch.where(x > 0, x / r, x * r), x)
        x = x - f * cnt.to(wide)
        x = x - p * (cnt > 0).to(wide)
    if c["bias"]:
        x = x + st["bias"].to(wide)[s]
    if c["grammar"]:
        at = torch.arange(V, device=DEV)
        x = torch.where(((st["allowed"][:, at // 32] >> (at % 32).int()) & 1).bool(), x, -math.inf)
    return x


def _commit(st):
    c = st["case"]
    if own:
        from speculative_decoding_moe_gb300 import dfv
        path, tau = dfv.accept_tree(st["tree"], st["tokens"], st["target"])
        lens = torch.empty_like(st["lens"])
        dfv.cache_commit(st["cache"], st["tree"], path, tau, st["ws"], new_lens=lens)
        return {"path": path, "tau": tau, "lens": lens, "k": st["k"], "v": st["v"]}
    S, N = c["seqs"], st["most"]
    s, i = _rows(st)
    j = torch.arange(N, device=DEV)
    bits = torch.zeros(S, N, N, dtype=torch.bool, device=DEV)
    bits[s, i] = _bits(st, N)
    tok, want, real = (torch.zeros(S, N, dtype=torch.int32, device=DEV) for _ in range(3))
    tok[s, i], want[s, i], real[s, i] = st["tokens"], st["target"], 1
    # the parent is the highest node below the node in its mask; an edge holds where the target, at the parent, wants the
    # node's token and no lower sibling has the same
    up = torch.where(bits & (j[None, :] < j[:, None]), j, -1).amax(-1)
    same = (up[:, :, None] == up[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & (j[None, :] < j[:, None])
    holds = (up >= 0) & (tok == want.gather(1, up.clamp_min(0))) & ~same.any(-1) & real.bool()
    holds[:, 0] = True
    kept = (holds[:, None, :] | ~bits).all(-1) & real.bool()
    tau = kept.sum(-1).to(torch.int32)
    path = torch.where(kept, j, N).sort(-1).values
    src = torch.where(path < N, path, j)  # nodes beyond the path stay
    path = torch.where(path < N, path, -1).to(torch.int32)
    lens = st["lens"].long()[:, None]
    seq = torch.arange(S, device=DEV)[:, None]
    moved = (path >= 0)
    to, fro = (lens + j)[moved], (lens + src)[moved]
    seq = seq.expand(S, N)[moved]
    to_page, fro_page = st["table"][seq, to // c["page"]].long(), st["table"][seq, fro // c["page"]].long()
    for x in (st["k"], st["v"]):
        x[:, to_page, :, to % c["page"]] = x[:, fro_page, :, fro % c["page"]].clone()
    return {"path": path, "tau": tau, "lens": st["lens"] + tau, "k": st["k"], "v": st["v"]}


def _fork(st):
    c = st["case"]
    table, refs, lens, src, dst = st["table"], st["refs"], st["lens"], st["src"].long(), st["dst"].long()
    if own:
        from speculative_decoding_moe_gb300 import dfv
        dfv.pages_free(st["cache"], st["dst"])
        dfv.pages_fork(st["cache"], st["src"], st["dst"], st["ws"])
    else:
        n, page = refs.numel(), c["page"]
        old = table[dst].long().flatten()
        refs.scatter_add_(0, old.clamp_min(0), -(old >= 0).int())
        # whole pages are shared, a last page in use is copied to the lowest free page
        full, rest = lens[src] // page, lens[src] % page
        at = torch.arange(table.shape[1], device=DEV)[None, :]
        new = torch.where(at < full[:, None], table[src], -1)
        free = torch.where(refs == 0, torch.arange(n, device=DEV), n).sort().values
        got = torch.where(rest > 0, free[((rest > 0).cumsum(0) - 1).clamp_min(0)].to(torch.int32), -1)
        last = table[src, full.long()].long().clamp_min(0)
        new = torch.where((at == full[:, None]) & (rest > 0)[:, None], got[:, None], new)
        table[dst] = new
        lens[dst] = lens[src]
        flat = new.long().flatten()
        refs.scatter_add_(0, flat.clamp_min(0), (flat >= 0).int())
        # rows in use only; a sequence without a last page in use copies a row onto itself
        t = torch.arange(page, device=DEV)[None, :]
        use = t < rest[:, None]
        fro = torch.where(rest > 0, last, 0)
        to = torch.where(rest > 0, got.long(), 0)
        fro, to, t = fro[:, None].expand_as(use)[use], to[:, None].expand_as(use)[use], t.expand_as(use)[use]
        for x in (st["k"], st["v"]):
            x[:, to, :, t] = x[:, fro, :, t]
    return {"table": table, "refs": refs, "lens": lens, "k": st["k"], "v": st["v"]}


# ---------------------------------------------------------------- work and exact
def work(case):
    c = case
    e = SIZE[c["dtype"]]
    nodes = _nodes(c) if "nodes" in c else []
    rows = sum(nodes)
    if c["op"] == "logits":
        V = c["vocab"]
        b = rows * V * 2 * e + rows * 8
        b += c["seqs"] * c["hist"] * 4 if c["rep"] else 0
        b += c["seqs"] * V * 4 if c["bias"] else 0
        b += rows * -(-V // 32) * 4 if c["grammar"] else 0
        return {"bytes": b, "flops": rows * V * (4 * c["rep"] + c["bias"] + 1)}
    row = c["kv"] * c["dim"] * e
    if c["op"] == "rope":
        return {"bytes": rows * (2 * (c["heads"] + 2 * c["kv"]) * c["dim"] * e + 4), "flops": rows * (c["heads"] + c["kv"]) * c["rot"] * 3}
    if c["op"] == "attn":
        keys = sum(a + b for a, b in zip(_lens(c), nodes))
        return {"bytes": 2 * keys * row + 2 * rows * c["heads"] * c["dim"] * e + rows * c["heads"] * 4,
                "flops": 4 * c["heads"] * c["dim"] * sum(n * (a + (n + 1) // 2) for a, n in zip(_lens(c), nodes))}
    if c["op"] == "commit":
        # the root stays where it is; the other accepted rows are read and written, keys and values
        moved = sum(a - 1 for a in _accepts(c))
        return {"bytes": moved * c["layers"] * row * 4 + rows * 16 + c["seqs"] * (8 + 4 * c["nodes"]), "flops": rows}
    used = sum(_lens(c)[s] % c["page"] for s in _fork_sources(c))
    table = c["forks"] * -(-c["ctx"] // c["page"]) * 4
    return {"bytes": used * c["layers"] * row * 4 + 4 * table, "flops": c["forks"]}


def exact(case, seed):
    """The operators' definitions, row by row, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op == "logits":
        off, out = st["row_off"].tolist(), []
        mask = [m & (2 ** 64 - 1) for m in st["mask"].tolist()]
        tokens, hist = st["tokens"].tolist(), st["hist"].long()
        for s in range(c["seqs"]):
            said = hist[s, :int(st["hist_len"][s])]
            made = torch.bincount(said[int(st["prompt_len"][s]):], minlength=c["vocab"])
            any_ = torch.bincount(said, minlength=c["vocab"])
            for r in range(off[s], off[s + 1]):
                x = st["logits"][r].double()
                if c["rep"]:
                    path = torch.tensor([tokens[off[s] + j] for j in range(off[s + 1] - off[s]) if mask[r] >> j & 1], device=DEV)
                    own_ = torch.bincount(path, minlength=c["vocab"])
                    n, met = made + own_, (any_ + own_) > 0
                    k = float(st["repetition"][s])
                    x[met] = torch.where(x[met] > 0, x[met] / k, x[met] * k)
                    x -= float(st["frequency"][s]) * n + float(st["presence"][s]) * (n > 0)
                if c["bias"]:
                    x += st["bias"][s].double()
                if c["grammar"]:
                    w = st["allowed"][r].long()[:, None] >> torch.arange(32, device=DEV)
                    x[~(w & 1).bool().flatten()[:c["vocab"]]] = -math.inf
                out.append(x)
        return {"logits": torch.stack(out), "best": None}
    if op == "attn":
        off, lens, G = st["row_off"].tolist(), st["lens"].tolist(), c["heads"] // c["kv"]
        o = torch.zeros(st["rows"], c["heads"], c["dim"], dtype=torch.float64, device=DEV)
        lse = torch.zeros(st["rows"], c["heads"], dtype=torch.float64, device=DEV)
        mask = None if st["mask"] is None else [m & (2 ** 64 - 1) for m in st["mask"].tolist()]
        for s in range(c["seqs"]):
            n = off[s + 1] - off[s]
            T = lens[s] + n
            pages = st["table"][s, :-(-T // c["page"])].long()
            sees = torch.ones(n, T, dtype=torch.bool, device=DEV)
            sees[:, lens[s]:] = torch.tensor([[(j <= i) if mask is None else bool(mask[off[s] + i] >> j & 1) for j in range(n)]
                                              for i in range(n)], device=DEV)
            for h in range(c["kv"]):
                k = st["k"][0, pages, h].reshape(-1, c["dim"])[:T].double()
                v = st["v"][0, pages, h].reshape(-1, c["dim"])[:T].double()
                x = torch.einsum("ngd,td->ngt", st["q"][off[s]:off[s + 1], h * G:(h + 1) * G].double(), k) / math.sqrt(c["dim"])
                x = x.masked_fill(~sees[:, None, :], -math.inf)
                lse[off[s]:off[s + 1], h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                o[off[s]:off[s + 1], h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(x, -1), v)
        return {"o": o, "lse": lse}
    if op == "rope":
        f, scale = _freqs(c)
        f, r, H, K = f.tolist(), c["rot"], c["heads"], c["kv"]
        x = st["qkv"].double()
        y = x.clone()
        for m, w in enumerate(f):
            a, b = (2 * m, 2 * m + 1) if c["inter"] else (m, m + r // 2)
            t = torch.polar(torch.full_like(st["positions"], 1, dtype=torch.float64) * scale, st["positions"].double() * w)[:, None]
            z = torch.complex(x[..., a], x[..., b]) * t
            y[..., a], y[..., b] = z.real, z.imag
        k, v = st["k"].double(), st["v"].double()
        off, lens, table = st["row_off"].tolist(), st["lens"].tolist(), st["table"].tolist()
        for s in range(c["seqs"]):
            for i in range(off[s + 1] - off[s]):
                at = lens[s] + i
                p = table[s][at // c["page"]]
                k[0, p, :, at % c["page"]] = y[off[s] + i, H:H + K]
                v[0, p, :, at % c["page"]] = x[off[s] + i, H + K:]
        return {"q": y[:, :H], "k": k, "v": v}
    return None  # commit and fork move what is there
