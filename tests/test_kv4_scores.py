"""Attention over the cache in 4 bits where scores are large and exact: the weights of positions that
different warps and blocks have seen.

As in test_attention_scores, with digits to the base of 8 (codes 0..7): one channel of every group
is 7 for all positions, which makes the groups' scales 1, and queries have zeros there."""
import pytest
import torch

from attention_testlib import attend, check, cu_of, paged, spans
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, gen, randn
from test_attention_scores import start_near

SIZES = [131_101, 262_147, 524_309, 725_900, 726_815, 2_000_003, -131_101, -725_900]


def held(scores, v, page=16):
    """A cache of one key head with keys whose products with the queries below are `scores`."""
    n, _, d = v.shape
    k = torch.zeros(n, 1, d, device=DEV)
    k[:, 0, ::32] = 7
    for i in range(7):
        k[:, 0, channel(i, d)] = scores.abs() // 8 ** i % 8
    table, pages = paged([n], page)
    cache = kb.kda_kv4_cache(pages, page, 1, d)
    kb.kda_kv4_write(k.bfloat16(), v, cache, table)
    assert torch.equal(spans(cache, table, 0, 0, n)[0], k.double())
    return cache, table


def channel(digit, d):
    return (1 + 9 * digit) if d == 64 else (3 + 18 * digit)


def queries(sign, rows, heads, d):
    q = torch.zeros(rows, 1, heads, d, device=DEV)
    for i in range(7):
        q[..., channel(i, d)] = sign * 8.0 ** i
    return q.bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("n,sequences,heads,d", [
    (500, 1, 3, 128),      # a few warps, each with a part of its own
    (500, 1, 3, 64),
    (9000, 1, 8, 128),     # several blocks
    (9000, 1, 12, 64),     # (and 16 columns)
    (640, 480, 2, 128),    # the warps of a block, and units cut in two by blocks
    (640, 480, 2, 64),
])
def test_parts_whose_maxima_differ_by_little(size, n, sequences, heads, d):
    j = torch.arange(n, device=DEV)
    start = start_near(size, 2)
    step = 32 if n < 1000 else 512   # a slice, or several blocks' parts
    scores = start + j // step % 3 - j * 7 % 2
    v = (randn(gen(1), n, 1, d, std=0.1) + (1 - 2 * (j // step % 2))[:, None, None]).bfloat16()
    cache, table = held(scores, v)
    q = queries(-1.0 if start < 0 else 1.0, sequences, heads, d)
    lens = torch.full((sequences,), n, dtype=torch.int32, device=DEV)
    out, lse = kb.kda_kv4_attention(q, cache, table.expand(sequences, -1).contiguous(), lens, scale=1.0, want_lse=True)
    assert kb.kda_get_device_error() == 0
    o, l, m, _ = attend(q[0], *spans(cache, table, 0, 0, n), 1.0, [n])
    wide = [t.expand(sequences, *t.shape) for t in (o, l, m)]
    check(out, lse, (*wide, torch.zeros_like(wide[1])), d)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [8, 20, 40, 90])
@pytest.mark.parametrize("n,sequences,heads,d", [(500, 1, 3, 128), (9000, 1, 8, 128), (640, 480, 2, 64), (40, 3, 12, 64)])
def test_scores_beyond_whole_numbers_of_32_bits(power, n, sequences, heads, d):
    """Scores of up to 2^90 times their digits, from the queries' size (2^108, of 2^112): one position has all of a
    row, or two that are alike share it."""
    j = torch.arange(n, device=DEV)
    scores = j * 7919 % 1999
    scores[n // 3] = scores[n // 2 + 3] = 2000
    v = randn(gen(2), n, 1, d, dtype=torch.bfloat16)
    cache, table = held(scores, v)
    q = queries(2.0 ** power, sequences, heads, d)
    lens = torch.full((sequences,), n, dtype=torch.int32, device=DEV)
    out, lse = kb.kda_kv4_attention(q, cache, table.expand(sequences, -1).contiguous(), lens, scale=1.0, want_lse=True)
    assert kb.kda_get_device_error() == 0
    kd, vd = spans(cache, table, 0, 0, n)
    o, l, m, _ = attend(q[0], kd, vd, 1.0, [n])
    want = (vd[n // 3] + vd[n // 2 + 3]) / 2
    assert torch.allclose(o, want.expand_as(o), rtol=1e-12, atol=1e-12)
    wide = [t.expand(sequences, *t.shape) for t in (o, l, m)]
    check(out, lse, (*wide, torch.zeros_like(wide[1])), d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,sequences,heads", [(40, 3, 12), (500, 1, 3), (9000, 1, 8)])
def test_groups_with_one_large_channel(n, sequences, heads, d):
    """Keys with an outlier in every group, so that most codes are 0, and queries that are small there
    and large elsewhere: sums of (n + 8) q less 8 sum q, whose terms are far larger than n q.  With X
    the sum of s |q| (|n| + 16), scale included: at most d products and their sum, the d terms of
    8 sum q and its parts, and the groups' products with s, 2^-23 of X or less each."""
    g = gen(n + d)
    k = randn(g, n, 1, d)
    k[:, :, 5::32] = 70 * (1 + torch.rand(n, 1, d // 32, generator=g, device=DEV))
    v = randn(g, n, 1, d, dtype=torch.bfloat16)
    table, pages = paged([n], 16)
    cache = kb.kda_kv4_cache(pages, 16, 1, d)
    kb.kda_kv4_write(k.bfloat16(), v, cache, table)
    q = randn(g, sequences, 1, heads, d, std=4.0)
    q[..., 5::32] *= 0.002
    q = q.bfloat16()
    lens = torch.full((sequences,), n, dtype=torch.int32, device=DEV)
    out, lse = kb.kda_kv4_attention(q, cache, table.expand(sequences, -1).contiguous(), lens, want_lse=True)
    kd, vd = spans(cache, table, 0, 0, n)
    scale = d ** -0.5
    pos = torch.arange(n, device=DEV)
    s = cache[1][table[0].long()[pos // 16], 0, pos % 16].double().repeat_interleave(32, 1)   # [n, d]
    assert ((kd[:, 0] / s).abs() < 0.5).float().mean() > 0.9   # codes of 0
    for i in range(sequences):
        o, l, m, _ = attend(q[i], kd, vd, scale, [n])
        X = scale * torch.einsum("hd,kd->hk", q[i, 0].double().abs(), kd[:, 0].abs() + 16 * s).amax(1)[None]
        check(out[i], lse[i], (o, l, m, X), d)
