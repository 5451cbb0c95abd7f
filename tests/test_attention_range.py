"""Full attention over values so large that sums over them come near what 32 bits hold: right where
the largest magnitude times the number of keys stays below 2^127 (over the cache, whose codes are
summed as n 2^-6: below 2^132), also where the running maximum lags behind."""
import pytest
import torch

from attention_testlib import check, cu_of, paged, reference, spans, attend
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, gen


def values(g, n, d, power):
    """Between 2^(power - 2) and 2^power, in one head all of a sign."""
    return ((0.25 + 0.75 * torch.rand(n, 1, d, generator=g, device=DEV)) * 2.0 ** power).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,power,queries", [(306, 118, 20), (1, 127, 1), (3000, 115, 5)])
def test_large_values_of_prompts(n, power, queries, d):
    """Scores that grow by 5.375, 2^7.75 in p, behind a tile of keys or several times."""
    j = torch.arange(n, device=DEV)
    q = torch.zeros(queries, 3, d, device=DEV)
    q[..., 9] = 1
    k = torch.zeros(n, 1, d, device=DEV)
    k[:, 0, 9] = 5.375 * (j // 128 % 4 > 0)
    q, k, v = q.bfloat16(), k.bfloat16(), values(gen(n), n, d, power)
    for causal in (True, False):
        out, lse = kb.kda_attention_fwd(q, k, v, cu_of([queries]), cu_of([n]), causal=causal, scale=1.0, want_lse=True)
        assert out.isfinite().all()
        check(out, lse, reference(q, k, v, [queries], [n], 1.0, causal), d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,power", [(96, 125), (1, 126), (9000, 118)])
def test_large_values_of_the_cache(n, power, d):
    """Scores that grow by 5.25, 2^7.57 in p."""
    j = torch.arange(n, device=DEV)
    k = torch.zeros(n, 1, d, device=DEV)
    k[:, 0, 9] = 5.25 * ((j // 32 > 0) if n < 1000 else (j // 128 % 2 > 0))
    v = values(gen(n), n, d, power)
    table, pages = paged([n], 16)
    cache = kb.kda_kv4_cache(pages, 16, 1, d)
    kb.kda_kv4_write(k.bfloat16(), v, cache, table)
    q = torch.zeros(1, 1, 3, d, device=DEV)
    q[..., 9] = 1
    out, lse = kb.kda_kv4_attention(q.bfloat16(), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                                    scale=1.0, want_lse=True)
    assert kb.kda_get_device_error() == 0 and out.isfinite().all()
    check(out[0], lse[0], attend(q[0], *spans(cache, table, 0, 0, n), 1.0, [n]), d)
