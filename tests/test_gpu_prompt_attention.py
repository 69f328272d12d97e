"""Causal attention of packed prompts on the GPU against its definition in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests._prompt_util import attention, check, offsets

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, rows, keys, heads, kv, dim, dtype, seed=0, lead=0, tail=0, size=1.0):
        """rows[s], keys[s] of each sequence; `lead` rows belong to nobody in front, `tail` behind."""
        g = torch.Generator().manual_seed(seed)
        self.off, self.koff = offsets(rows, lead), offsets(keys, lead)
        self.n, self.nk, self.rows, self.keys = self.off[-1] + tail, self.koff[-1] + tail, rows, keys
        self.n, self.nk = max(self.n, 1), max(self.nk, 1)
        self.H, self.K, self.D, self.dtype = heads, kv, dim, dtype
        self.q = (size * torch.randn(self.n, heads, dim, generator=g)).to(dtype)
        self.k = torch.randn(self.nk, kv, dim, generator=g).to(dtype)
        self.v = torch.randn(self.nk, kv, dim, generator=g).to(dtype)

    def batches(self, dfv, most=None):
        rows = dfv.RowBatch(i32(self.off), self.n, max(max(self.rows), 1))
        return rows, dfv.RowBatch(i32(self.koff), self.nk, most or max(max(self.keys), 1))

    def run(self, dfv, q=None, k=None, v=None, most=None, lse=True, **kw):
        rows, keys = self.batches(dfv, most)
        ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, self.H, self.K, self.D))
        L = torch.full((self.n, self.H), 7.0, device="cuda") if lse else None
        out = torch.full((self.n, self.H, self.D), 9.0, dtype=self.dtype, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dfv.prompt_attention(rows, self.q.cuda() if q is None else q, self.k.cuda() if k is None else k,
                             self.v.cuda() if v is None else v, ws, keys=keys, out=out, lse=L, err=err, **kw)
        assert dfv.read_device_error(ws) == 0
        return out, L, int(err.item())

    def want(self, scale=None):
        return attention(self.q, self.k, self.v, self.off, self.koff, scale or self.D ** -0.5)

    def check(self, dfv, scale=None, **kw):
        out, L, err = self.run(dfv, **({} if scale is None else dict(scale=scale)), **kw)
        assert err == 0
        r0, r1 = self.off[0], self.off[-1]
        o, lse, a, big = self.want(scale)
        check(out[r0:r1], None if L is None else L[r0:r1], self.dtype, self.D, max(max(self.keys), 1), o[r0:r1], lse[r0:r1], a[r0:r1], big[r0:r1])
        for x, was in ((out, 9.0), (L, 7.0)):  # rows that belong to nobody
            if x is not None:
                assert bool((x[:r0] == was).all()) and bool((x[r1:] == was).all())


LENGTHS = [([1], [1]), ([2], [2]), ([31], [31]), ([33], [33]), ([128], [128]), ([129], [129]), ([257], [257]), ([1, 0, 64, 130], [1, 0, 64, 130]),
           ([5, 17], [200, 17]), ([1, 1, 1], [1, 128, 129]), ([40], [300]), ([3], [1300]), ([2, 70], [1100, 70]), ([300], [1500])]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,kv,dim", [(8, 1, 128), (4, 2, 64), (7, 1, 128), (3, 3, 64), (16, 1, 64), (5, 1, 128)])
@pytest.mark.parametrize("rows,keys", LENGTHS)
def test_lengths(dfv, rows, keys, heads, kv, dim, dtype):
    Case(rows, keys, heads, kv, dim, dtype, seed=len(rows) + heads).check(dfv)


@pytest.mark.parametrize("most", [1536, 1537])
def test_ranges_that_end_at_tiles_or_cut_them(dfv, most):
    """The same lengths as a call that may have more keys (cut and joined) and as one that may not."""
    for rows in ([200, 3, 900], [1000], [64] * 40):
        Case(rows, rows, 4, 2, 64, BF, seed=5).check(dfv, most=most)


@pytest.mark.parametrize("rows,keys,heads,kv,dim", [
    ([900, 500, 1100], [900, 500, 1100], 16, 8, 64), ([900, 500, 1100], [1000, 1500, 1100], 16, 8, 128),  # whole tiles, several a CTA
    ([5] * 39 + [20], [5] * 39 + [1601], 64, 64, 64), ([5] * 39 + [20], [7] * 39 + [1601], 64, 64, 128),  # whole, though longer: there are many
    ([0, 5, 0, 0, 70], [3, 5, 0, 9, 70], 16, 8, 64), ([130] * 9, [130] * 9, 16, 8, 128), ([256] * 4, [400] * 4, 19, 19, 64)])  # a tile a CTA
def test_every_way_to_end_the_ranges(dfv, rows, keys, heads, kv, dim):
    Case(rows, keys, heads, kv, dim, BF, seed=6, lead=2, tail=3).check(dfv)


def test_many_sequences(dfv):
    rows = [(7 * s) % 19 for s in range(700)]
    Case(rows, rows, 2, 1, 64, HF, seed=3).check(dfv)
    Case(rows, [n + (s * 5) % 40 for s, n in enumerate(rows)], 2, 1, 64, BF, seed=4).check(dfv)


@pytest.mark.parametrize("rows,keys", [([6], [2]), ([300], [3]), ([200, 9], [0, 9]), ([150], [140])])
def test_rows_without_keys(dfv, rows, keys):
    c = Case(rows, keys, 8, 1, 128, BF, seed=1)
    c.check(dfv)
    out, L, _ = c.run(dfv)
    n = rows[0] - keys[0]
    assert bool((out[:n] == 0).all()) and bool((L[:n] == -math.inf).all())


def test_rows_of_nobody_stay(dfv):
    Case([30, 100], [30, 100], 4, 2, 128, BF, lead=5, tail=9).check(dfv)


def test_no_rows_at_all(dfv):
    c = Case([0, 0], [0, 3], 4, 2, 64, BF, tail=4)
    out, L, err = c.run(dfv)
    assert err == 0 and bool((out == 9).all()) and bool((L == 7).all())


@pytest.mark.parametrize("dim,dtype", [(128, BF), (64, HF)])
def test_strides(dfv, dim, dtype):
    """Slices of one projection, and head-major keys and values."""
    c = Case([70, 150], [70, 150], 8, 2, dim, dtype, seed=9)
    qkv = torch.cat([c.q, c.k, c.v], 1).cuda()
    o, lse, a, big = c.want()
    out, L, _ = c.run(dfv, q=qkv[:, :8], k=qkv[:, 8:10], v=qkv[:, 10:])
    check(out, L, dtype, dim, 150, o, lse, a, big)
    k, v = (x.cuda().transpose(0, 1).contiguous().transpose(0, 1) for x in (c.k, c.v))
    out, L, _ = c.run(dfv, k=k, v=v)
    check(out, L, dtype, dim, 150, o, lse, a, big)
    rows, keys = c.batches(dfv)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, 8, 2, dim))
    out = torch.zeros(8, c.n, dim, dtype=dtype, device="cuda").transpose(0, 1)
    dfv.prompt_attention(rows, c.q.cuda(), c.k.cuda(), c.v.cuda(), ws, keys=keys, out=out)
    check(out, None, dtype, dim, 150, o, lse, a, big)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size,scale", [(1.0, 1.0), (8.0, None), (30.0, None), (1.0, 1e-3)])
def test_large_and_small_scores(dfv, dtype, size, scale):
    """Scores whose maximum grows by far more than 2^8 from key to key, within a block's halves too."""
    c = Case([200], [420], 4, 1, 128, dtype, seed=2, size=size)
    ramp = torch.linspace(0.1, 6.0, 420)[torch.randperm(420, generator=torch.Generator().manual_seed(1))]
    c.k = (c.k.float() * ramp[:, None, None]).to(dtype)
    c.check(dfv, scale=scale)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("keys", [150, 1200])
def test_what_is_masked_does_not_count(dfv, dtype, dim, keys):
    """NaN and infinities in keys and values that a row does not see, and in rows of nobody, leave it as it was bit for
    bit; rows that see an infinite value have it."""
    n = 100
    c = Case([n, 20], [keys, 20], 8, 2, dim, dtype, seed=6, lead=3, tail=40)
    k, v = c.k.cuda(), c.v.cuda()
    was, lse, _ = c.run(dfv, k=k, v=v)
    at = c.koff[0] + keys - 30  # the key that row n - 30 is the first to see
    for x in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        for t in (k2, v2):
            t[:c.koff[0]] = x
            t[c.koff[-1]:] = x
        v2[at:at + 2, 1, 5] = x
        k2[at + 1] = x
        out, L, _ = c.run(dfv, k=k2, v=v2)
        first = c.off[0] + n - 30
        assert torch.equal(out[:first], was[:first]) and torch.equal(L[:first], lse[:first])
        assert torch.equal(out[c.off[1]:], was[c.off[1]:]) and torch.equal(L[c.off[1]:], lse[c.off[1]:])
        group = out[first, 4:]  # heads of kv head 1
        assert bool((~torch.isfinite(group[:, 5])).all()) and bool(torch.isfinite(group[:, :5]).all())
        assert torch.equal(out[first, :4], was[first, :4])
        if x == x:
            assert bool((group[:, 5] == x).all())


def test_a_nan_query_stays_in_its_row(dfv):
    c = Case([90], [90], 4, 1, 64, BF, seed=8)
    was, _, _ = c.run(dfv)
    q = c.q.cuda()
    q[40, 2, 7] = float("nan")
    out, L, _ = c.run(dfv, q=q)
    assert bool(torch.isnan(out[40, 2]).all()) and bool(torch.isnan(L[40, 2]))
    keep = torch.ones(90, 4, dtype=torch.bool)
    keep[40, 2] = False
    assert torch.equal(out[keep.cuda()], was[keep.cuda()])


def test_offsets_out_of_range(dfv):
    c = Case([30, 40, 20], [30, 40, 20], 4, 2, 64, BF, seed=8)
    was, _, _ = c.run(dfv)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(c.batches(dfv)[0], 4, 2, 64))
    for off in ([0, 30, 91, 90], [0, 30, 20, 90], [-1, 30, 70, 90], [0, 30, 70, 1 << 30]):
        out = torch.full_like(was, 9.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dfv.prompt_attention(dfv.RowBatch(i32(off), 90, 40), c.q.cuda(), c.k.cuda(), c.v.cuda(), ws, out=out, err=err)
        assert int(err.item()) == dfv.KVERR_LEN and dfv.read_device_error(ws) == 0
        for s in range(3):
            if 0 <= off[s] <= off[s + 1] <= 90 and off[s + 1] - off[s] <= 40 and off[s:s + 2] == c.off[s:s + 2]:
                assert torch.equal(out[off[s]:off[s + 1]], was[off[s]:off[s + 1]])


def test_the_same_bits_every_time_and_in_a_graph(dfv):
    c = Case([700, 90], [1500, 90], 8, 1, 128, BF, seed=11)
    rows, keys = c.batches(dfv)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, 8, 1, 128))
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    was = dfv.prompt_attention(rows, q, k, v, ws, keys=keys)
    for _ in range(3):
        assert torch.equal(dfv.prompt_attention(rows, q, k, v, ws, keys=keys), was)
    out = torch.zeros_like(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfv.prompt_attention(rows, q, k, v, ws, keys=keys, out=out)
    g.replay()
    assert torch.equal(out, was)
    # other lengths through the same graph
    rows.row_off.copy_(i32([0, 300, 790]))
    keys.row_off.copy_(i32([0, 1100, 1590]))
    rows2, keys2 = dfv.RowBatch(i32([0, 300, 790]), 790, 700), dfv.RowBatch(i32([0, 1100, 1590]), 1590, 1500)
    want = dfv.prompt_attention(rows2, q, k, v, ws, keys=keys2)
    g.replay()
    assert torch.equal(out, want)


def test_another_stream(dfv):
    c = Case([300], [300], 8, 2, 128, BF, seed=12)
    s = torch.cuda.Stream()
    rows, keys = c.batches(dfv)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, 8, 2, 128))
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    was = dfv.prompt_attention(rows, q, k, v, ws, keys=keys)
    s.wait_stream(torch.cuda.current_stream())
    out = dfv.prompt_attention(rows, q, k, v, ws, keys=keys, stream=s)
    s.synchronize()
    assert torch.equal(out, was)


def test_long(dfv):
    """A sequence of several thousand keys, against the definition on a sample of its rows."""
    n, D = 5003, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(BF) for h in (8, 1, 1))
    rows = dfv.RowBatch(i32([0, n]), n, n)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, 8, 1, D))
    lse = torch.empty(n, 8, device="cuda")
    out = dfv.prompt_attention(rows, q, k, v, ws, lse=lse)
    for i in list(range(0, n, 401)) + [n - 1]:
        o, w, a, big = attention(q[i:i + 1].cpu(), k[:i + 1].cpu(), v[:i + 1].cpu(), [0, 1], [0, i + 1], D ** -0.5)
        check(out[i:i + 1], lse[i:i + 1], BF, D, n, o, w, a, big)
