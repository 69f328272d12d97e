"""Operators that bring a prompt into the paged cache and read the cache in 8 bits: the cases that are measured, and their plain forms.

A prompt's rows get the norms of their queries and keys for each head, their rotary positions and their place in the cache
in one pass (append); a cache in 8 bits (e4m3 codes, one power of two for each token and head) is written by the same pass and read
back as packed rows, as a prompt that comes in chunks needs it (store8); the rows attend causally to their own and all
earlier tokens (prompt); drafted nodes or single new tokens attend to a cache in 8 bits (attn8).

`own` false: elementary torch operations, in 32 bits (64 for angles), rounded once.  `own` true: the framework's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
LOW, HIGH = -100, 120  # exponents of the codes' power of two


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short question to an idle server: latency only
        dict(name="prompt short", op="prompt", seqs=1, rows=137, prefix=0, heads=32, kv=4, dim=128, dtype="bf16"),
        # sixteen requests that arrive together, ragged
        dict(name="prompt packed", op="prompt", seqs=16, rows=2039, prefix=0, heads=32, kv=4, dim=128, dtype="bf16"),
        # one long document: the largest
        dict(name="prompt long", op="prompt", seqs=1, rows=16381, prefix=0, heads=32, kv=4, dim=128, dtype="bf16"),
        # the next chunk of two long documents whose earlier chunks are there already; narrow heads
        dict(name="prompt chunk", op="prompt", seqs=2, rows=1021, prefix=30011, heads=32, kv=8, dim=64, dtype="f16"),
        # one new token of one request: latency only
        dict(name="append decode", op="append", seqs=1, rows=1, ctx=4097, heads=32, kv=4, dim=128, rot=128, inter=False, norm=True,
             theta=1e6, page=16, dtype="bf16"),
        # eight prompts in full
        dict(name="append prompts", op="append", seqs=8, rows=2039, ctx=0, heads=32, kv=4, dim=128, rot=128, inter=False, norm=True,
             theta=1e6, page=16, dtype="bf16"),
        # the last few rows of a prompt into a cache in 8 bits, and what the sequence holds read back
        dict(name="store8 tail", op="store8", seqs=1, rows=19, ctx=509, heads=32, kv=4, dim=128, rot=128, inter=False, norm=True,
             theta=1e6, page=16, dtype="bf16"),
        # chunks of four long prompts into a cache in 8 bits, and what the sequences hold read back for their attention
        dict(name="store8 chunks", op="store8", seqs=4, rows=1021, ctx=16381, heads=32, kv=8, dim=64, rot=32, inter=True, norm=True,
             theta=1e4, page=64, dtype="bf16"),
        # one token of one request over a short cache
        dict(name="attn8 decode", op="attn8", seqs=1, nodes=1, ctx=1021, heads=32, kv=4, dim=128, page=16, dtype="bf16"),
        # the same over a long document, narrow heads, larger pages
        dict(name="attn8 long decode", op="attn8", seqs=1, nodes=1, ctx=131071, heads=32, kv=8, dim=64, page=64, dtype="bf16"),
        # one token of each of 64 requests with ragged lengths
        dict(name="attn8 batch decode", op="attn8", seqs=64, nodes=1, ctx=8191, heads=32, kv=4, dim=128, page=16, dtype="bf16"),
        # 32 requests with drafted trees of 16 nodes
        dict(name="attn8 trees", op="attn8", seqs=32, nodes=16, ctx=8191, heads=32, kv=4, dim=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "store8", "attn8", "attn8"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    group = rng.choice([1, 2, 4, 5, 7, 8]) if kv <= 4 else rng.choice([1, 2, 4])
    heads = kv * group
    if op == "prompt":
        # no more scores than the largest case has
        seqs, most = _log(rng, 1, 16), 32 * 16381 ** 2
        rows = _log(rng, 1, min(16381, int(math.sqrt(most / (seqs * heads)))))
        room = min(32768, most // (seqs * heads * rows) - rows)
        prefix = 0 if rng.random() < 0.5 or room < 1 else _log(rng, 1, room)
        return dict(op=op, seqs=seqs, rows=rows, prefix=prefix, heads=heads, kv=kv, dim=dim, dtype=rng.choice(["bf16", "f16"]))
    if op in ("append", "store8"):
        seqs = _log(rng, 1, 16)
        rows = _log(rng, 1, min(2039, 16384 // seqs))
        return dict(op=op, seqs=seqs, rows=rows, ctx=_log(rng, 1, min(32768, 65536 // seqs)) - 1, heads=heads, kv=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2]), inter=rng.random() < 0.5, norm=rng.random() < 0.7, theta=rng.choice([1e4, 1e6]),
                    page=page, dtype=rng.choice(["bf16", "f16"]) if op == "append" else "bf16")
    seqs = _log(rng, 1, 64)
    nodes = 1 if rng.random() < 0.5 else _log(rng, 1, 64)
    # no more keys than the largest case in all, no more products than the trees' either
    most = int(min(64 * 8191 * 4 // (seqs * kv), 32 * 16 * 8191 * 32 // (seqs * nodes * heads)))
    return dict(op=op, seqs=seqs, nodes=nodes, ctx=_log(rng, 1, min(131072, max(1, most))), heads=heads, kv=kv, dim=dim, page=page,
                dtype="bf16")


# ---------------------------------------------------------------- what a case fixes
def _less(most, s, step):
    return most - (s * step) % (most // 2 + 1)


def _rows(c):
    """New rows of each sequence: the most, then fewer ones down to half."""
    return [_less(c["nodes"] if c["op"] == "attn8" else c["rows"], s, 5 if c["op"] == "attn8" else 389) for s in range(c["seqs"])]


def _before(c):
    """Tokens of each sequence that are there before the new ones."""
    n = c["prefix"] if c["op"] == "prompt" else c["ctx"]
    return [_less(n, s, 397) for s in range(c["seqs"])]


def _off(counts):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return off


# ---------------------------------------------------------------- prepare
def _normal(shape, dtype, g):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


def _coded(x):
    """Codes and exponent bytes of values in 32 bits: e is the smallest power with max |x| <= 448 * 2^e."""
    m, at = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, at - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH)
    return torch.ldexp(x, -e[..., None]).to(E4M3), (e + 127).to(torch.uint8)


def _valued(codes, exps):
    """What codes stand for, in 32 bits."""
    return torch.ldexp(codes.float(), exps.int()[..., None] - 127)


def prepare(case, seed):
    c = case
    rng = random.Random(seed * 1000003 + 29)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    dt = DT[c["dtype"]]
    news, olds = _rows(c), _before(c)
    off = _off(news)
    H, K, D = c["heads"], c["kv"], c["dim"]
    st = {"case": c, "op": c["op"], "n": off[-1], "most": max(news), "row_off": ints(off)}
    if c["op"] == "prompt":
        keys = _off([a + b for a, b in zip(news, olds)])
        st["key_off"], st["keys"], st["most_keys"] = ints(keys), keys[-1], max(a + b for a, b in zip(news, olds))
        st["q"], st["k"], st["v"] = _normal((off[-1], H, D), dt, g), _normal((keys[-1], K, D), dt, g), _normal((keys[-1], K, D), dt, g)
        if own:
            from speculative_decoding_moe_gb300 import dfv
            st["batch"] = dfv.RowBatch(st["row_off"], off[-1], max(news))
            st["key_batch"] = dfv.RowBatch(st["key_off"], keys[-1], st["most_keys"]) if c["prefix"] else None
            st["ws"] = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(st["batch"], H, K, D))
        return st

    # a paged cache: [layers][pages][kv heads][tokens of a page][dim]; shuffled pages
    page = c["page"]
    need = [-(-(a + b) // page) for a, b in zip(olds, news)]
    order = list(range(sum(need)))
    rng.shuffle(order)
    table = torch.full((c["seqs"], max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    st["table"], st["lens"] = table.to(DEV), ints(olds)
    shape = (1, len(order), K, page, D)
    st["k"], st["v"] = _normal(shape, torch.float32, g), _normal(shape, torch.float32, g)
    if c["op"] == "append":
        st["k"], st["v"] = st["k"].to(dt), st["v"].to(dt)
    else:
        # tokens differ in their size
        for x in ("k", "v"):
            st[x] *= torch.exp(0.5 * _normal(shape[:4] + (1,), torch.float32, g))
            st[x], st[x + "_exp"] = _coded(st[x])
    if c["op"] == "attn8":
        st["q"] = _normal((off[-1], H, D), dt, g)
        masks = []  # random trees, parents first: bit j of a node's mask is set for its ancestors and itself
        for n in news:
            m = []
            for i in range(n):
                m.append((m[rng.randint(max(0, i - 6), i - 1)] if i else 0) | (1 << i))
            masks += m
        st["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    else:
        # q, k and v as a projection leaves them: one row of all heads
        st["qkv"] = _normal((off[-1], H + 2 * K, D), dt, g)
        st["positions"] = ints([a + i for a, n in zip(olds, news) for i in range(n)])
        st["q_gain"] = st["k_gain"] = None
        if c["norm"]:
            st["q_gain"], st["k_gain"] = ((1 + 0.2 * _normal((D,), torch.float32, g)).to(dt) for _ in range(2))
    if own:
        from speculative_decoding_moe_gb300 import dfv
        st["cache"] = dfv.KVCache(st["k"], st["v"], st["table"], st["lens"], k_exp=st.get("k_exp"), v_exp=st.get("v_exp"))
        if c["op"] == "attn8":
            st["batch"] = dfv.TreeBatch(st["row_off"], off[-1], max(news), mask=st["mask"])
            st["ws"] = dfv.alloc_workspace(dfv.tree_attention_workspace_size(st["cache"], st["batch"], H))
        else:
            st["batch"] = dfv.RowBatch(st["row_off"], off[-1], max(news))
            st["rope"] = dfv.Rope(D, rot_dim=c["rot"], theta=c["theta"], interleaved=c["inter"])
    if c["op"] == "store8":
        held = [a + b for a, b in zip(olds, news)]
        st["held_off"], st["held"], st["most_held"] = ints(_off(held)), sum(held), max(held)
        if own:
            st["held_batch"] = dfv.RowBatch(st["held_off"], sum(held), max(held))
    return st


# ---------------------------------------------------------------- run
def run(state):
    return {"prompt": _prompt, "append": _append, "store8": _store8, "attn8": _attn8}[state["op"]](state)


def _of_rows(off, n):
    """Sequence and number within it of each packed row."""
    r = torch.arange(n, device=DEV, dtype=torch.int32)
    s = torch.searchsorted(off, r, right=True) - 1
    return s, r.long() - off.long()[s]


def _softmax_product(x, seen, v):
    """(o, lse) of scores [..., rows, keys], in place, with what each row sees."""
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x.sub_(top).exp_()
    den = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v)
    return torch.where(den > 0, o / den, torch.zeros_like(o)), (top + den.log()).squeeze(-1)


def _prompt(st):
    c = st["case"]
    H, K, D = c["heads"], c["kv"], c["dim"]
    G = H // K
    if own:
        from speculative_decoding_moe_gb300 import dfv
        lse = torch.empty(st["n"], H, device=DEV)
        return {"o": dfv.prompt_attention(st["batch"], st["q"], st["k"], st["v"], st["ws"], keys=st["key_batch"], lse=lse), "lse": lse}
    # padded to the longest sequence
    S, N, T = c["seqs"], st["most"], st["most_keys"]
    s, i = _of_rows(st["row_off"], st["n"])
    sk, j = _of_rows(st["key_off"], st["keys"])
    q = torch.zeros(S, N, K, G, D, device=DEV)
    q[s, i] = st["q"].float().reshape(-1, K, G, D)
    k, v = torch.zeros(S, K, T, D, device=DEV), torch.zeros(S, K, T, D, device=DEV)
    k[sk, :, j], v[sk, :, j] = st["k"].float(), st["v"].float()
    news, keys = st["row_off"].diff().long(), st["key_off"].diff().long()
    last = torch.arange(N, device=DEV)[None, :] + (keys - news)[:, None]  # the last key that each row sees
    seen = torch.arange(T, device=DEV) <= last[:, :, None]
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, K, G * N, D), k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    x = x.reshape(S, K, G, N, T)
    o, lse = _softmax_product(x, seen[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, H, D)[s, i]
    return {"o": o.to(DT[c["dtype"]]), "lse": lse.permute(0, 3, 1, 2).reshape(S, N, H)[s, i]}


def _turned(st):
    """Queries, keys and values of the new rows, normed and turned, in 32 bits."""
    c = st["case"]
    H, K, r = c["heads"], c["kv"], c["rot"]
    f = c["theta"] ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    angle = st["positions"].double()[:, None] * f[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
        y, z = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y, z], -1).flatten(-2) if c["inter"] else torch.cat([y, z], -1)
        return torch.cat([y, x[..., r:]], -1)

    q, k, v = st["qkv"][:, :H], st["qkv"][:, H:H + K], st["qkv"][:, H + K:]
    return turn(q, st["q_gain"]), turn(k, st["k_gain"]), v.float()


def _places(st):
    s, i = _of_rows(st["row_off"], st["n"])
    at = st["lens"].long()[s] + i
    return st["table"][s, at // st["case"]["page"]].long(), at % st["case"]["page"]


def _own_append(st):
    from speculative_decoding_moe_gb300 import dfv
    c = st["case"]
    H, K = c["heads"], c["kv"]
    q, k, v = st["qkv"][:, :H], st["qkv"][:, H:H + K], st["qkv"][:, H + K:]
    return dfv.norm_rope_append(st["cache"], 0, st["batch"], st["rope"], q, k, v, st["positions"], q_gain=st["q_gain"], k_gain=st["k_gain"], eps=EPS)


def _append(st):
    if own:
        return {"q": _own_append(st), "k": st["k"], "v": st["v"]}
    q, k, v = _turned(st)
    page, row = _places(st)
    dt = DT[st["case"]["dtype"]]
    st["k"][0, page, :, row], st["v"][0, page, :, row] = k.to(dt), v.to(dt)
    return {"q": q.to(dt), "k": st["k"], "v": st["v"]}


def _store8(st):
    if own:
        from speculative_decoding_moe_gb300 import dfv
        q = _own_append(st)
        k, v = dfv.cache_read(st["cache"], 0, st["held_batch"])
        return {"q": q, "k": k, "v": v}
    q, k, v = _turned(st)
    page, row = _places(st)
    s, i = _of_rows(st["held_off"], st["held"])
    held_page, held_row = st["table"][s, i // st["case"]["page"]].long(), i % st["case"]["page"]
    out = {"q": q.bfloat16()}
    for name, x in (("k", k), ("v", v)):
        codes, exps = _coded(x)
        st[name].view(torch.uint8)[0, page, :, row] = codes.view(torch.uint8)
        st[name + "_exp"][0, page, :, row] = exps
        codes = st[name].view(torch.uint8)[0, held_page, :, held_row].view(E4M3)
        out[name] = _valued(codes, st[name + "_exp"][0, held_page, :, held_row]).bfloat16()
    return out


def _attn8(st):
    c = st["case"]
    S, N, K, D = c["seqs"], st["most"], c["kv"], c["dim"]
    G = c["heads"] // K
    if own:
        from speculative_decoding_moe_gb300 import dfv
        lse = torch.empty(st["n"], c["heads"], device=DEV)
        return {"o": dfv.tree_attention(st["cache"], 0, st["batch"], st["q"], st["ws"], lse=lse), "lse": lse}
    # padded to the longest sequence and the largest tree
    s, i = _of_rows(st["row_off"], st["n"])
    table = st["table"].long().clamp_min(0)
    T = table.shape[1] * c["page"]
    flat = lambda x: _valued(x[0].view(torch.uint8)[0][table].view(E4M3), x[1][0][table]).permute(0, 2, 1, 3, 4).reshape(S, K, T, D)  # noqa: E731
    k, v = flat((st["k"], st["k_exp"])), flat((st["v"], st["v_exp"]))
    q = torch.zeros(S, N, K, G, D, device=DEV)
    q[s, i] = st["q"].float().reshape(-1, K, G, D)
    key = torch.arange(T, device=DEV)[None, :] - st["lens"].long()[:, None]  # below 0: there before, then the node's number
    bits = torch.zeros(S, N, N, dtype=torch.bool, device=DEV)
    bits[s, i] = ((st["mask"][:, None] >> torch.arange(N, device=DEV)[None, :]) & 1).bool()
    node = key.clamp(0, N - 1)[:, None, :].expand(S, N, T)
    seen = (key < 0)[:, None, :] | ((key < N)[:, None, :] & bits.gather(2, node))
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, K, G * N, D), k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    o, lse = _softmax_product(x.reshape(S, K, G, N, T), seen[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, K * G, D)[s, i]
    return {"o": o.to(DT[c["dtype"]]), "lse": lse.permute(0, 3, 1, 2).reshape(S, N, K * G)[s, i]}


# ---------------------------------------------------------------- work and exact
def work(case):
    c = case
    news, olds = _rows(c), _before(c)
    rows, H, K, D = sum(news), c["heads"], c["kv"], c["dim"]
    if c["op"] == "prompt":
        keys = rows + sum(olds)
        return {"bytes": (2 * rows * H + 2 * keys * K) * D * 2 + rows * H * 4, "flops": 4 * H * D * sum(n * a + n * (n + 1) // 2 for a, n in zip(olds, news))}
    if c["op"] == "attn8":
        keys = rows + sum(olds)
        return {"bytes": 2 * keys * K * (D + 1) + 2 * rows * H * D * 2 + rows * (H * 4 + 8),
                "flops": 4 * H * D * sum(n * (a + (n + 1) // 2) for a, n in zip(olds, news))}
    flops = rows * (H + K) * (3 * c["rot"] + 4 * D * c["norm"])
    if c["op"] == "append":
        return {"bytes": rows * (2 * (H + 2 * K) * D * 2 + 4), "flops": flops}
    held = rows + sum(olds)  # what was there is read once; the new rows' codes are written, and their values go on from the pass that has them
    return {"bytes": rows * (2 * H + 2 * K) * D * 2 + rows * 4 + 2 * rows * K * (D + 1) + 2 * sum(olds) * K * (D + 1) + 2 * held * K * D * 2,
            "flops": flops + 4 * rows * K * D + 2 * held * K * D}


def _nearest8(x):
    """Values in 64 bits, a row's last dimension with one power of two, rounded to what 8 bits hold (four significant bits, steps of 2^-9 at least)."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448)).nan_to_num(neginf=LOW)
    e = torch.where(top > 448 * 2.0 ** e, e + 1, e)  # a logarithm next to a whole number
    e = torch.where(top <= 448 * 2.0 ** (e - 1), e - 1, e).clamp(LOW, HIGH)
    y = x / 2.0 ** e
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step * 2.0 ** e


def exact(case, seed):
    """The operators' definitions, sequence by sequence, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c, news, olds = case, _rows(case), _before(case)
    H, K, D = c["heads"], c["kv"], c["dim"]
    G = H // K
    off = _off(news)
    if c["op"] in ("prompt", "attn8"):
        o = torch.zeros(off[-1], H, D, dtype=torch.float64, device=DEV)
        lse = torch.zeros(off[-1], H, dtype=torch.float64, device=DEV)
        at = 0
        masks = None if c["op"] == "prompt" else [m & (2 ** 64 - 1) for m in st["mask"].tolist()]
        for s, (n, a) in enumerate(zip(news, olds)):
            for h in range(K):
                if masks is None:
                    k, v = st["k"][at:at + a + n, h].double(), st["v"][at:at + a + n, h].double()
                else:
                    pages = st["table"][s, :-(-(a + n) // c["page"])].long()
                    k, v = ((st[x].view(torch.uint8)[0, pages, h].view(E4M3).double() * 2.0 ** (st[x + "_exp"][0, pages, h].double()[..., None] - 127))
                            .reshape(-1, D)[:a + n] for x in ("k", "v"))
                step = max(1, min(n, 2 ** 27 // ((a + n) * G)))
                for i in range(0, n, step):
                    m = min(n, i + step)
                    if masks is None:
                        sees = torch.arange(a + m, device=DEV)[None, :] <= a + torch.arange(i, m, device=DEV)[:, None]
                    else:
                        sees = torch.ones(m - i, a + n, dtype=torch.bool, device=DEV)
                        sees[:, a:] = torch.tensor([[bool(masks[off[s] + w] >> j & 1) for j in range(n)] for w in range(i, m)], device=DEV)
                    q = st["q"][off[s] + i:off[s] + m, h * G:(h + 1) * G].double()
                    x = torch.einsum("ngd,td->ngt", q, k[:sees.shape[1]]) / math.sqrt(D)
                    x = x.masked_fill(~sees[:, None, :], -math.inf)
                    lse[off[s] + i:off[s] + m, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                    o[off[s] + i:off[s] + m, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(x, -1), v[:sees.shape[1]])
            at += a + n
        return {"o": o, "lse": lse}

    r = c["rot"]
    x = st["qkv"].double()
    for heads, gain in ((slice(0, H), st["q_gain"]), (slice(H, H + K), st["k_gain"])):
        if gain is not None:
            x[:, heads] = gain.double() * x[:, heads] / torch.sqrt((x[:, heads] ** 2).sum(-1, keepdim=True) / D + EPS)
    y = x.clone()
    for m in range(r // 2):
        a, b = (2 * m, 2 * m + 1) if c["inter"] else (m, m + r // 2)
        t = torch.polar(torch.ones_like(st["positions"], dtype=torch.float64), st["positions"].double() * c["theta"] ** (-2.0 * m / r))[:, None]
        z = torch.complex(x[:, :H + K, a], x[:, :H + K, b]) * t
        y[:, :H + K, a], y[:, :H + K, b] = z.real, z.imag
    lens, table = st["lens"].long(), st["table"].long()
    k, v = ((st["k"].double(), st["v"].double()) if c["op"] == "append" else
            (st[w].double() * 2.0 ** (st[w + "_exp"].double()[..., None] - 127) for w in ("k", "v")))
    back = {"k": [], "v": []}
    for s, n in enumerate(news):
        at = lens[s] + torch.arange(n, device=DEV)
        pages, rows = table[s, at // c["page"]], at % c["page"]
        new_k, new_v = y[off[s]:off[s + 1], H:H + K], x[off[s]:off[s + 1], H + K:]
        if c["op"] == "store8":
            new_k, new_v = _nearest8(new_k), _nearest8(new_v)
        k[0, pages, :, rows], v[0, pages, :, rows] = new_k, new_v
        if c["op"] == "store8":
            at = torch.arange(olds[s] + n, device=DEV)
            for w, z in (("k", k), ("v", v)):
                back[w].append(z[0, table[s, at // c["page"]], :, at % c["page"]])
    if c["op"] == "append":
        return {"q": y[:, :H], "k": k, "v": v}
    return {"q": y[:, :H], "k": torch.cat(back["k"]), "v": torch.cat(back["v"])}
