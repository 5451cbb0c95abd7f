"""A single token has no next one: through the C entry point its distance may be any number that the
checks let pass, odd or larger than a tensor map's."""
import ctypes

import pytest
import torch

from attention_testlib import check, qkv, reference
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import gen


@pytest.mark.gpu
@pytest.mark.parametrize("ld", [513, (1 << 39) + 8, 1 << 40])
@pytest.mark.parametrize("which", ["q", "k", "v", "out"])
def test_any_distance_of_a_single_token(which, ld):
    q, k, v = qkv(gen(1), 1, 1, 4, 2, 128)
    out, lse = torch.empty_like(q), torch.empty(1, 4, device=q.device)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    lds = {"q": 512, "k": 256, "v": 256, "out": 512} | {which: ld}
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = kb.load().kda_attention_fwd(p(q), lds["q"], p(k), lds["k"], p(v), lds["v"], None, None, p(out), lds["out"],
                                     p(lse), 1, 1, 1, 4, 2, 128, 128 ** -0.5, 1, stream)
    assert st == 0, kb.load().kda_last_error_message()
    assert kb.kda_get_device_error() == 0
    check(out, lse, reference(q, k, v, [1], [1], 128 ** -0.5), 128)
