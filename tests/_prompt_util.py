"""Helpers of the prompt tests: packed prompts, and the operators' definitions in 64 bits on the CPU, without the library."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # torch.finfo(t).eps / 2
E4M3 = torch.float8_e4m3fn
LOW, HIGH = -100, 120


def offsets(counts, start=0):
    off = [start]
    for n in counts:
        off.append(off[-1] + n)
    return off


def attention(q, k, v, row_off, key_off, scale):
    """(o, lse, p @ |v|, largest scale * sum |q k|) by the definition, sequence by sequence; what a row does not attend to is
    left out of its sums."""
    rows, H, D = q.shape
    G = H // k.shape[1]
    o, a = torch.zeros(rows, H, D, dtype=torch.float64), torch.zeros(rows, H, D, dtype=torch.float64)
    lse, big = torch.full((rows, H), -math.inf, dtype=torch.float64), torch.zeros(rows, H, dtype=torch.float64)
    for s in range(len(row_off) - 1):
        r0, r1, k0, k1 = row_off[s], row_off[s + 1], key_off[s], key_off[s + 1]
        n, nk = r1 - r0, k1 - k0
        for i in range(n):
            see = nk - n + i + 1
            if see <= 0:
                continue
            kk, vv = (x[k0:k0 + min(see, nk)].double().repeat_interleave(G, 1) for x in (k, v))  # [keys, H, D]
            qq = q[r0 + i].double()
            x = scale * torch.einsum("hd,khd->hk", qq, kk)
            lse[r0 + i] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            o[r0 + i], a[r0 + i] = torch.einsum("hk,khd->hd", p, vv), torch.einsum("hk,khd->hd", p, vv.abs())
            big[r0 + i] = (scale * torch.einsum("hd,khd->hk", qq.abs(), kk.abs())).amax(-1)
    return o, lse, a, big


def tolerances(dtype, D, keys, o, lse, a, big):
    """Output: half a step of the type for its rounding and one for the rounding of p (weighted by |v|), plus twice the
    fp32 errors of p: the dot product's D + 2 roundings of at most `big`, 2^-21 for exp2 and its argument's rounding at
    |x| <= 2 big, one rounding per key in the sums.  lse: the same fp32 errors once."""
    u = 2.0 ** -24
    f = (D + 2) * u * big + 2.0 ** -21 + 4 * u * big + (keys + 16) * u
    half = HALF_STEP[dtype]
    to = half * o.abs() + (half + 2 * f[..., None]) * a * (1 + half) + 1e-30
    if dtype == torch.float16:  # its subnormals: spacing 2^-24, for p and for the output
        to = to + 2.0 ** -25 * (1 + a)
    tl = f + 4 * u * torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)) + 4 * u
    return to, tl


def check(got_o, got_lse, dtype, D, keys, o, lse, a, big):
    to, tl = tolerances(dtype, D, keys, o, lse, a, big)
    d = (got_o.double().cpu() - o).abs()
    assert bool((d <= to).all()), "output off by %g of its tolerance" % float((d / to).max())
    if got_lse is not None:
        g = got_lse.double().cpu()
        none = torch.isinf(lse)
        assert bool((g[none] == -math.inf).all())
        d = (g - lse).abs()[~none]
        assert bool((d <= tl[~none]).all()), "lse off by %g of its tolerance" % float((d / tl[~none]).max())


# ---------------------------------------------------------------- codes
def coded(x):
    """(values, codes, exponents) of 64-bit values by the definition: e is the smallest integer with max |x| <= 448 * 2^e over
    the last dimension, the code is the nearest of e4m3's values (ties to even)."""
    top = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, at = torch.frexp(top)
    e = torch.where(m > 0, at - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH)
    y = torch.ldexp(x, -e[..., None].double())
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6).nan_to_num(1.0, 1.0, 1.0))) - 3)
    y = torch.where(torch.isfinite(y), torch.round(y / step) * step, torch.nan)
    return torch.ldexp(y, e[..., None].double()), y, e


def valued(codes, exps):
    """64-bit values of codes (float8) and exponent bytes."""
    return codes.double() * torch.exp2(exps.double() - 127)[..., None]
