"""Full attention over scores that 32 bits hold exactly: what the running maximum's rounding does to
the weights of keys that were seen before it moved, or by another block.

A score is a whole number S, put together from digits: the queries hold the digits' weights, the
keys the digits, one channel each, so that every product and every sum is a whole number below 2^24.
Keys' scores differ by 1 or 2 in some hundred thousand.  The weights then depend on differences
alone, and the bounds of attention_testlib hold with X = 0: what is left is the exponent's rounding
(|x| <= 32 in powers of two: 2^-20 of a weight that is itself below 2^-8 where |x| > 16), the
exponential's, and p's to bf16."""
import numpy
import pytest
import torch

from attention_testlib import check, cu_of, reference
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, gen, randn

# around 2^17, 2^18 and 2^19; below 2^20 / log2(e), across it, above; beyond
SIZES = [131_101, 262_147, 524_309, 725_900, 726_815, 726_900, 2_000_003, -131_101, -725_900, -726_900]


def start_near(size, last):
    """A start within 64 of `size` for which the product of a score and log2(e) in 32 bits is rounded
    most differently for start + last - 1 and start + last (but for 726,815, which crosses 2^20)."""
    if size == 726_815:
        return size
    c = numpy.float32(1.4426950408889634)
    off = lambda m: float(numpy.float32(m) * c) - m * float(c)
    return max(range(size, size + 64), key=lambda m: abs(off(m + last) - off(m + last - 1)))


def prompt(scores, heads, d, queries):
    """q [queries, heads, d], k [len, 1, d] whose products are `scores` [len].  The last head's
    scores grow by 40 with every 128 keys besides, which moves the maximum for all rows of its warp."""
    sign = -1.0 if scores[0] < 0 else 1.0
    digits = scores.abs()
    q = torch.zeros(queries, heads, d, device=DEV)
    k = torch.zeros(len(scores), 1, d, device=DEV)
    for channel, weight in ((3, 65536), (20, 256), (d - 7, 1)):
        q[..., channel] = sign * weight
        k[:, 0, channel] = digits // weight % 256
    k[:, 0, 33] = torch.arange(len(scores), device=DEV) // 128
    q[:, -1, 33] = 40.0
    return q.bfloat16(), k.bfloat16()


def exact(out, lse, ref, d):
    o, l, m, _ = ref
    check(out, lse, (o, l, m, torch.zeros_like(l)), d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", SIZES)
def test_a_maximum_that_grows_by_little(size, d):
    """Scores that grow by 1 with every 128 keys, and the maximum with them."""
    j = torch.arange(600, device=DEV)
    start = start_near(size, 4)
    scores = start + j // 128 - j * 7 % 3
    q, k = prompt(scores, 4, d, 40)
    v = randn(gen(1), 600, 1, d, std=0.1, dtype=torch.bfloat16) + (1 - 2 * (j // 128 % 2))[:, None, None].bfloat16()
    for causal in (True, False):
        out, lse = kb.kda_attention_fwd(q, k, v, cu_of([40]), cu_of([600]), causal=causal, scale=1.0, want_lse=True)
        exact(out, lse, reference(q, k, v, [40], [600], 1.0, causal), d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", SIZES)
def test_parts_whose_maxima_differ_by_little(size, d):
    """Keys shared by several blocks, a part's maximum 1 from the next one's."""
    n = 5000
    j = torch.arange(n, device=DEV)
    start = start_near(size, 2)
    scores = start + j // 512 % 3 - j * 7 % 2
    q, k = prompt(scores, 4, d, 3)
    q[:, -1, 33] = 0
    v = randn(gen(2), n, 1, d, std=0.1, dtype=torch.bfloat16) + (1 - 2 * (j // 512 % 2))[:, None, None].bfloat16()
    ref = reference(q, k, v, [3], [n], 1.0)
    for cu in ((cu_of([3]), cu_of([n])), (None, None)):
        out, lse = kb.kda_attention_fwd(q, k, v, *cu, scale=1.0, want_lse=True)
        exact(out, lse, ref, d)
