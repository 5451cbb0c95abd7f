"""Uniform batches [B, T_b, heads, d] whose B is not the number of sequences, and tensors of more
dimensions, are refused by the full-attention calls: tokens would go to other sequences' places.  On
the host, with tensors that have no memory."""
import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from test_attention_devices import BF16, CACHE, CALLS, I32
from test_ops_devices import bare

FOUR = ((2, 8, 2, 128), BF16)


def call(name, drop=(), **over):
    made = {k: bare(*v) for k, v in (CALLS[name] | over).items() if k not in drop}
    if "k_codes" in made:
        made["cache"] = tuple(made.pop(k) for k in CACHE)
    if name == "kda_kv4_read":
        made["total_tokens"] = 6
    return getattr(kb, name)(**made)


@pytest.mark.parametrize("name,over,word", [
    # 16 tokens over four rows of a table
    ("kda_kv4_write", dict(k=FOUR, v=FOUR, block_table=((4, 3), I32), start=((4,), I32)),
     "k has 2 sequences, expected 4"),
    ("kda_kv4_write", dict(k=((1, 8, 2, 128), BF16), v=((1, 8, 2, 128), BF16)), "k has 1 sequences, expected 2"),
    ("kda_kv4_read", dict(k=((3, 2, 2, 128), BF16)), "k has 3 sequences, expected 2"),
    ("kda_kv4_read", dict(v=((1, 6, 2, 128), BF16)), "v has 1 sequences, expected 2"),
])
def test_uniform_spans_of_other_numbers_of_sequences_are_refused(name, over, word):
    with pytest.raises(kb.KdaError, match=word):
        call(name, drop=("cu_seqlens",), **over)


@pytest.mark.parametrize("n_seqs", [1, 4, 16])
def test_uniform_prompts_of_other_numbers_of_sequences_are_refused(n_seqs):
    q, k = bare((2, 8, 4, 128), BF16), bare(*FOUR)
    with pytest.raises(kb.KdaError, match=f"q has 2 sequences, expected {n_seqs}"):
        kb.kda_attention_fwd(q, k, k, n_seqs=n_seqs)


@pytest.mark.parametrize("name,key,shape", [
    ("kda_attention_fwd", "q", (1, 2, 3, 4, 128)), ("kda_attention_fwd", "k", (1, 2, 3, 2, 128)),
    ("kda_kv4_write", "k", (1, 2, 3, 2, 128)), ("kda_kv4_read", "k", (1, 2, 3, 2, 128)),
    ("kda_kv4_read", "v", (1, 2, 3, 2, 128)), ("kda_kv4_attention", "q", (1, 2, 1, 4, 128)),
])
def test_more_dimensions_are_refused(name, key, shape):
    with pytest.raises(kb.KdaError, match=f"{key} must have 3 or 4 dimensions, got"):
        call(name, **{key: (shape, BF16)})
