"""The full-attention calls refuse tensors of several GPUs, a stream of another one, and tensors
that do not fit together, on the host and before anything is allocated or launched.  The tensors
here have a device, a shape and strides and no memory, so that no GPU is needed."""
import types

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from test_ops_devices import bare

BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
CACHE = dict(k_codes=((5, 2, 16, 64), U8), k_scales=((5, 2, 16, 4), BF16),
             v_codes=((5, 2, 16, 64), U8), v_scales=((5, 2, 16, 4), BF16))
SPAN = dict(block_table=((2, 3), I32), start=((2,), I32), cu_seqlens=((3,), I32))
KV = dict(k=((6, 2, 128), BF16), v=((6, 2, 128), BF16))
CALLS = {
    "kda_attention_fwd": dict(q=((6, 4, 128), BF16), **KV, cu_seqlens_q=((3,), I32), cu_seqlens_k=((3,), I32),
                              out=((6, 4, 128), BF16), lse=((6, 4), F32)),
    "kda_kv4_write": dict(**KV, **CACHE, **SPAN),
    "kda_kv4_read": dict(block_table=((2, 3), I32), **CACHE, start=((2,), I32), cu_seqlens=((3,), I32), **KV),
    "kda_kv4_attention": dict(q=((2, 4, 128), BF16), **CACHE, block_table=((2, 3), I32), seq_lens=((2,), I32),
                              out=((2, 4, 128), BF16), lse=((2, 4), F32)),
}


def call(name, elsewhere=(), stream=None, **over):
    made = {}
    for key, (shape, dtype) in (CALLS[name] | over).items():
        made[key] = bare(shape, dtype, "cuda:1" if key in elsewhere else "cuda:0")
    if "k_codes" in made:
        made["cache"] = tuple(made.pop(key) for key in CACHE)
    if name == "kda_kv4_read":
        made["total_tokens"] = 6
    return getattr(kb, name)(**made, stream=stream)


@pytest.mark.parametrize("name,key", [(n, k) for n, a in CALLS.items() for k in list(a)[1:]])
def test_an_operand_on_another_gpu_is_refused(name, key):
    with pytest.raises(kb.KdaError, match=f"{key} is on cuda:1, expected cuda:0"):
        call(name, [key])


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_gpu_is_refused(name):
    other = types.SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(kb.KdaError, match="the stream is on cuda:1, the tensors on cuda:0"):
        call(name, stream=other)


@pytest.mark.parametrize("name,over,word", [
    ("kda_attention_fwd", dict(q=((6, 4, 128), F32)), "q must be bfloat16"),
    ("kda_attention_fwd", dict(q=((6, 512), BF16)), "at least 3 dimensions"),
    ("kda_attention_fwd", dict(k=((6, 2, 64), BF16)), "q's dimensions and head size"),
    ("kda_attention_fwd", dict(v=((5, 2, 128), BF16)), "v must have the shape"),
    ("kda_attention_fwd", dict(cu_seqlens_k=((4,), I32)), "cu_seqlens_k must have the shape"),
    ("kda_attention_fwd", dict(cu_seqlens_q=((3,), torch.int64)), "cu_seqlens_q must be int32"),
    ("kda_attention_fwd", dict(out=((6, 4, 64), BF16)), "out must have the shape"),
    ("kda_attention_fwd", dict(lse=((6, 4, 1), F32)), "lse must have the shape"),
    ("kda_kv4_write", dict(k_codes=((5, 2, 16, 64), torch.int8)), "k_codes must be"),
    ("kda_kv4_write", dict(v_scales=((5, 2, 16, 2), BF16)), "v_scales must have the shape"),
    ("kda_kv4_write", dict(block_table=((3, 3), I32)), "block_table has 3 rows for 2 sequences"),
    ("kda_kv4_write", dict(start=((3,), I32)), "start must have the shape"),
    ("kda_kv4_write", dict(k=((6, 4, 128), BF16), v=((6, 4, 128), BF16)), "k has 4 heads of 128, the cache 2 of 128"),
    ("kda_kv4_read", dict(v=((7, 2, 128), BF16)), "v has 7 tokens, expected 6"),
    ("kda_kv4_attention", dict(seq_lens=((3,), I32)), "seq_lens must have the shape"),
    ("kda_kv4_attention", dict(q=((2, 4, 64), BF16)), "q has heads of 64, the cache of 128"),
    ("kda_kv4_attention", dict(block_table=((2, 3, 1), I32)), "block_table must have 2 dimensions"),
])
def test_tensors_that_do_not_fit_are_refused(name, over, word):
    with pytest.raises(kb.KdaError, match=word):
        call(name, **over)


def test_other_refusals():
    with pytest.raises(kb.KdaError, match="tuple"):
        kb.kda_kv4_write(bare((6, 2, 128), BF16), bare((6, 2, 128), BF16), None, bare((2, 3), I32))
    with pytest.raises(kb.KdaError, match="CUDA"):
        kb.kda_attention_fwd(*(torch.zeros(2, 1, 64, dtype=BF16) for _ in range(3)))
    with pytest.raises(kb.KdaError, match="total_tokens=-1"):
        kb.kda_kv4_read(tuple(bare(s, t) for s, t in CACHE.values()), bare((2, 3), I32), -1)
