"""A recurrent and a full-attention layer of a model, from residual stream to residual stream.

The recurrent layer is that of recurrent_block.py.  The attention layer has no positions, and
keeps its keys and values in pages, in 4 bits:

    residual's addition, RMS norm, 8 bits  ->  8-bit projection to q, k, v
    ->  k and v quantised into the cache (kda_kv4_write)
    ->  a prompt, or its next part: the cache read back (kda_kv4_read), attention over all of the
        sequence so far (kda_attention_fwd)
        a token of each sequence: attention over the cache (kda_kv4_attention)
    ->  RMS norm, 8 bits  ->  8-bit projection back

Both ways see the same keys and values, those that the cache holds.  Run as a program it feeds the
same tokens as whole prompts, as prompts in two parts, and as steps behind a shorter prompt, and
compares:

    python examples/hybrid_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from gated_delta_rule_48_gb300 import binding as kda  # noqa: E402
from recurrent_block import DeltaRuleLayer, Layer  # noqa: E402


class Cache:
    """Pages for some sequences of up to `longest` tokens each, handed out in no order."""

    def __init__(self, sequences, longest, kv_heads, head_dim, page=16):
        pages = -(-longest // page)
        order = torch.randperm(sequences * pages, generator=torch.Generator().manual_seed(0))
        self.table = order.to(torch.int32).view(sequences, pages).cuda()
        self.arrays = kda.kda_kv4_cache(sequences * pages, page, kv_heads, head_dim)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")


class AttentionLayer(Layer):
    def __init__(self, dim, heads, kv_heads, head_dim, gen):
        self.heads, self.kv_heads, self.d = heads, kv_heads, head_dim
        super().__init__(dim, heads * head_dim, (heads + 2 * kv_heads) * head_dim, gen)

    def _split(self, p):
        """q, k, v [tokens, heads, d]: columns of the projection."""
        a, b = self.heads * self.d, self.kv_heads * self.d
        return (p[:, :a].unflatten(1, (self.heads, self.d)),
                p[:, a:a + b].unflatten(1, (self.kv_heads, self.d)),
                p[:, a + b:].unflatten(1, (self.kv_heads, self.d)))

    def prompt(self, x, residual, cu, cache, lens):
        """The next `lens` tokens of each sequence (packed, cu as always)."""
        p, h = self.project_in(x, residual)
        q, k, v = self._split(p)
        kda.kda_kv4_write(k, v, cache.arrays, cache.table, cache.lens, cu)
        cache.lens += cu[1:] - cu[:-1]
        held = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()   # of the whole sequences
        k, v = kda.kda_kv4_read(cache.arrays, cache.table, sum(lens), None, held)
        o, _ = kda.kda_attention_fwd(q, k, v, cu, held)
        return self.project_out(o.flatten(1)), h

    def step(self, x, residual, cache):
        p, h = self.project_in(x, residual)
        q, k, v = self._split(p)
        one = torch.arange(len(x) + 1, dtype=torch.int32, device="cuda")
        kda.kda_kv4_write(k, v, cache.arrays, cache.table, cache.lens, one)
        cache.lens += 1
        o, _ = kda.kda_kv4_attention(q, cache.arrays, cache.table, cache.lens)
        return self.project_out(o.flatten(1)), h


class Model:
    """A recurrent layer in front of an attention layer, with both layers' states."""

    def __init__(self, dim=512, heads=8, kv_heads=2, head_dim=64, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.recurrent = DeltaRuleLayer(dim, 4, 64, gen)
        self.attention = AttentionLayer(dim, heads, kv_heads, head_dim, gen)
        self.norm = torch.ones(dim, dtype=torch.bfloat16, device="cuda")

    def start(self, sequences, longest):
        return Cache(sequences, longest, self.attention.kv_heads, self.attention.d)

    def prompt(self, x, cu, cache, lens):
        delta, h, state = self.recurrent.prompt(x, torch.zeros_like(x), cu)
        delta, h = self.attention.prompt(delta, h, cu, cache, lens)
        y, _ = kda.kda_add_rms_norm(delta, self.norm, h)
        return y, state

    def step(self, x, cache, state):
        delta, h = self.recurrent.step(x, torch.zeros_like(x), state)
        delta, h = self.attention.step(delta, h, cache)
        y, _ = kda.kda_add_rms_norm(delta, self.norm, h)
        return y


def packed(parts):
    ends = torch.tensor([0] + [len(p) for p in parts]).cumsum(0)
    return torch.cat(parts), ends.to(torch.int32).cuda()


def packed_with_residual(parts):
    x, cu = packed(parts)
    return x, torch.zeros_like(x), cu


def relative(got, want):
    got, want = got.float(), want.float()
    return ((got - want).norm() / want.norm()).item()


def compare(lens=(70, 1, 130), new=8, dim=512, seed=0):
    """The last `new` tokens of each sequence as part of their prompt, as a second part of it and as
    steps (the attention layer alone), and as steps through both layers: the relative differences
    of the latter three."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    seqs = [torch.randn(n + new, dim, device="cuda", generator=gen).bfloat16() for n in lens]
    full = [n + new for n in lens]
    ends = torch.tensor(full).cumsum(0).tolist()
    last = lambda y: torch.stack([y[e - new:e] for e in ends])
    model = Model(dim, seed=seed)
    # the attention layer: whole prompts, and prompts in two parts
    run = lambda parts, cache, lens: model.attention.prompt(*packed_with_residual(parts), cache, lens)[0]
    want = last(run(seqs, model.start(len(lens), max(full)), full))
    cache = model.start(len(lens), max(full))
    run([s[:n] for s, n in zip(seqs, lens)], cache, list(lens))
    in_parts = relative(run([s[n:] for s, n in zip(seqs, lens)], cache, full).view_as(want), want)
    # and in steps
    cache = model.start(len(lens), max(full))
    run([s[:n] for s, n in zip(seqs, lens)], cache, list(lens))
    rows = [torch.stack([s[n + t] for s, n in zip(seqs, lens)]) for t in range(new)]
    alone = relative(torch.stack([model.attention.step(x, torch.zeros_like(x), cache)[0] for x in rows], 1), want)
    # both layers: whole prompts, and steps
    want = last(model.prompt(*packed(seqs), model.start(len(lens), max(full)), full)[0])
    cache = model.start(len(lens), max(full))
    _, state = model.prompt(*packed([s[:n] for s, n in zip(seqs, lens)]), cache, list(lens))
    got = torch.stack([model.step(x, cache, state) for x in rows], 1)
    if kda.kda_get_device_error() != 0:
        raise RuntimeError(kda.load().kda_last_error_message().decode())
    return in_parts, alone, relative(got, want)


def main():
    in_parts, alone, steps = compare()
    print(f"8 tokens of 3 sequences, off those of whole prompts: attention over a second part of the "
          f"prompts {in_parts:.2e}, as steps {alone:.2e}; both layers as steps {steps:.2e}")
    return in_parts, alone, steps


if __name__ == "__main__":
    main()
