"""Helpers of the full-attention tests: the definition in 64 bits, and bounds on what the kernels'
roundings may do to a result.

A score is a sum of d products in 32 bits, each term off by at most (d + 8) 2^-23 of the terms'
magnitudes (tensor cores may cut a sum off instead of rounding it: 2^-23 a step), so with X the
largest sum of magnitudes of a row, scale included, p is off by a factor of at most
1 + e, e = (d + 8) 2^-23 X + 2^-21 (the rest: the exponent's rounding, the exponential).  The
quotient of two sums of such p is off by 2 e, and p's rounding to bf16 by 2^-8 more, of the terms'
magnitudes m = sum p |v| / sum p.  out itself is rounded to bf16."""
import math

import torch

from ops_testlib import BF16_HALF, DEV, assert_near, randn


def cu_of(lens):
    return torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def attend(q, k, v, scale, reach):
    """q [Q, heads, d] over k, v [L, kv_heads, d] in 64 bits, query i over the first reach[i] keys.
    Returns o, lse, the terms' magnitudes m and the rows' largest sums X of magnitudes."""
    Q, heads, d = q.shape
    g = heads // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    o, m = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((Q, heads), -math.inf, dtype=torch.float64, device=q.device)
    X = torch.zeros_like(lse)
    for i in range(Q):
        n = int(reach[i])
        if n <= 0:
            continue
        x = scale * torch.einsum("hd,khd->hk", q[i], k[:n])
        lse[i] = torch.logsumexp(x, 1)
        p = torch.softmax(x, 1)
        o[i] = torch.einsum("hk,khd->hd", p, v[:n])
        m[i] = torch.einsum("hk,khd->hd", p, v[:n].abs())
        X[i] = scale * torch.einsum("hd,khd->hk", q[i].abs(), k[:n].abs()).amax(1)
    return o, lse, m, X


def reference(q, k, v, q_lens, k_lens, scale, causal=True):
    parts, a, b = [], 0, 0
    for nq, nk in zip(q_lens, k_lens):
        i = torch.arange(nq)
        reach = (i + 1 + nk - nq).clamp(0, nk) if causal else torch.full((nq,), nk)
        parts.append(attend(q[a:a + nq], k[b:b + nk], v[b:b + nk], scale, reach))
        a, b = a + nq, b + nk
    return [torch.cat([p[j] for p in parts]) for j in range(4)]


def check(out, lse, ref, d, what=""):
    o, l, m, X = ref
    e = (d + 8) * 2.0 ** -23 * X + 2.0 ** -21
    assert_near(out, o, BF16_HALF * 1.01, what + "out", atol=(BF16_HALF * 1.02 + 2 * e)[..., None] * m + 1e-30)
    if lse is not None:
        inf = l.isinf()
        assert torch.equal(lse.isinf(), inf) and (lse[inf] < 0).all(), what + "lse of empty rows"
        assert_near(lse[~inf], l[~inf], 2.0 ** -22, what + "lse", atol=e[~inf] + 2.0 ** -22)


def qkv(g, tq, tk, heads, kv_heads, d, std=1.0):
    dt = torch.bfloat16
    return (randn(g, tq, heads, d, std=std, dtype=dt), randn(g, tk, kv_heads, d, std=std, dtype=dt),
            randn(g, tk, kv_heads, d, dtype=dt))


# ---- the cache, by its description
def decode(codes, scales, keys):
    """What rows of codes stand for: [..., d] in 64 bits."""
    G = scales.shape[-1]
    out = torch.empty(*codes.shape[:-1], 32 * G, dtype=torch.float64, device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
    per = 8 if keys else 4
    for w in range(nib.shape[-1] // per):
        g, part = w % G, w // G
        c = 32 * g + per * part
        out[..., c:c + per] = nib[..., w * per:(w + 1) * per] * scales[..., g:g + 1].double()
    return out


def quantised(x):
    """What x stands for once written, in 64 bits; NaN for groups with a NaN or an infinity."""
    g = x.double().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -64) / 7).float().bfloat16().double()
    ok = g.isfinite().all(-1, keepdim=True)
    n = torch.where(ok, torch.round(g / s), torch.zeros_like(g))
    return torch.where(ok, n * s, torch.full_like(g, math.nan)).flatten(-2)


def paged(lens, page, spare=3, seed=0, width=None):
    """(block table, number of pages): pages in no order, -1 behind a sequence's last one."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    width = width or max(counts + [1])
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (width - c))
        at += c
    return torch.tensor(rows, dtype=torch.int32).reshape(len(lens), width).to(DEV), total


def spans(cache, table, n, first, last):
    """Positions [first, last) of sequence n as the cache holds them: k, v in 64 bits."""
    page = cache[0].shape[2]
    pos = torch.arange(first, last, device=DEV)
    at = table[n].long()[pos // page], pos % page
    rows = [t[at[0], :, at[1]] for t in cache]
    return decode(rows[0], rows[1], True), decode(rows[2], rows[3], False)
