"""Units of seconds: a block's warps whose tile has no rows of a unit wait for its end, longer than
any other wait lasts."""
import math

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV


@pytest.mark.gpu
def test_a_tile_without_rows_waits_for_the_other():
    """One query of 305 heads: an odd group, so a unit to a head, with a row in its first tile and none in
    its second, over so many keys that a unit (not cut where each SM has two) takes some 2.8 seconds.
    A single wait lasts 2.1 at most, 2^20 polls of 2 us.  All keys are alike: out is the values' mean."""
    heads, n, d = 305, 450_000_000, 64
    free, _ = torch.cuda.mem_get_info()
    if free < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    kv = torch.full((n, 1, d), 0.5, dtype=torch.bfloat16, device=DEV)
    q = torch.ones(1, heads, d, dtype=torch.bfloat16, device=DEV)
    out, lse = kb.kda_attention_fwd(q, kv, kv, want_lse=True)
    assert kb.kda_get_device_error() == 0
    assert (out == 0.5).all()
    # l: 2200 additions between moves (test_attention_long) and a move for every 2^18 keys
    want = 32 * d ** -0.5 + math.log(n)
    assert (lse - want).abs().max().item() <= (2200 + n / 2 ** 18) * 2.0 ** -24 + 2.0 ** -22 * want
    del kv
    torch.cuda.empty_cache()
