"""Full attention over so many keys that what a tensor core cuts off when it adds a product to a large
sum adds up: sums are moved on after 2^18 keys (2^17 of a warp over the cache).

Of at most 2^18 products each may be cut by the last place of the sum so far, 2^-24 of it or a
little more, and that sum is half the whole one on average: 2^18 2^-25 = 2^-7 of the terms'
magnitudes, over the cache 2^-8, beside p's rounding and the output's (attention_testlib).  l is rounded by 2^-24 with
each addition: by tiles and, in a tile, pairs, 2048 + 64 of them (and a move's and a part's few);
over the cache by single positions of a lane, 2^17 / 8.  So lse is off by 2200 2^-24 = 1.3e-4 or by
2^-10, and out by as much of itself."""

import pytest
import torch

from attention_testlib import spans
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import BF16_HALF, DEV, assert_near, gen


def definition(scores, v):
    """One query's output, lse and terms' magnitudes over v [n, 1, d], in 64 bits."""
    x = scores.double()
    p = torch.softmax(x, 0)
    v = v[:, 0].double()
    o = (p[:, None] * v).sum(0)
    return o, torch.logsumexp(x, 0), o   # (values are positive)


def near(out, lse, ref, cut, additions):
    o, l, m = ref
    e = additions * 2.0 ** -24
    assert_near(out, o.expand(out.shape), BF16_HALF * 1.01, "out", atol=(BF16_HALF * 1.02 + cut + e) * m)
    worst = (lse.double() - l).abs().max().item()
    assert worst <= e + 2.0 ** -22 * l, worst


@pytest.mark.gpu
@pytest.mark.parametrize("heads,d,n,rise", [
    (305, 64, 1 << 22, 0.0), (305, 128, 1 << 22, 0.0),   # a unit to a head, and each whole
    (305, 128, (1 << 18) + 1, 0.0), (305, 64, (1 << 20) + 77, 0.75),
    (201, 128, (1 << 22) + 1000, 0.0), (201, 64, (1 << 21) - 5, 0.75),   # each in two parts
])
def test_many_keys_of_like_weights(heads, d, n, rise):
    """All scores alike, or growing in steps behind every 200,000 keys."""
    scores = torch.arange(n, device=DEV) // 200_000 * rise
    q = torch.zeros(1, heads, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., 3], k[:, 0, 3] = 1, scores.bfloat16()
    v = (0.5 + torch.rand(n, 1, d, generator=gen(n), device=DEV)).bfloat16()
    for _ in range(2):
        out, lse = kb.kda_attention_fwd(q, k, v, scale=1.0, want_lse=True)
        assert kb.kda_get_device_error() == 0
        near(out[0], lse, definition(scores, v), 2.0 ** -7, 2200)


@pytest.mark.gpu
def test_calls_with_many_keys_side_by_side():
    """Two streams' blocks take their places from the same ones."""
    n, d = 300_000, 64
    q = torch.zeros(1, 305, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    v = [(0.5 + i + torch.rand(n, 1, d, generator=gen(i), device=DEV)).bfloat16() for i in range(2)]
    want = [kb.kda_attention_fwd(q, k, x)[0] for x in v]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in v]
    got = [[kb.kda_attention_fwd(q, k, x, stream=s)[0] for x, s in zip(v, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for row in got for a, b in zip(row, want))
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_captured_calls_with_many_keys():
    """Two graphs replayed side by side, over keys that change."""
    n, d = 300_000, 128
    q = torch.zeros(1, 305, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    v = (0.5 + torch.rand(n, 1, d, generator=gen(3), device=DEV)).bfloat16()
    kb.kda_attention_fwd(q, k, v)
    graphs, outs, streams = [], [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        outs.append(torch.empty_like(q))
        with torch.cuda.graph(graphs[-1]):
            kb.kda_attention_fwd(q, k, v, out=outs[-1])
        streams.append(torch.cuda.Stream())
    for i in range(2):
        v.copy_(0.5 + i + torch.rand(n, 1, d, generator=gen(i), device=DEV))
        want = kb.kda_attention_fwd(q, k, v)[0]
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("heads,d,n,rise", [(2, 64, 1 << 24, 0.0), (2, 128, 1 << 22, 0.0), (12, 128, (1 << 21) + 50, 0.5),
                                            (4, 64, (1 << 20) + 1234, 0.5)])
def test_many_positions_of_like_weights(heads, d, n, rise):
    """1000 sequences of the same pages, so that a block has several whole ones."""
    seqs, page = 1000, 65536
    pages = -(-n // page)
    cache = kb.kda_kv4_cache(pages, page, 1, d)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    scores = torch.arange(n, device=DEV) // 200_000 * rise
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    k[:, 0, 3] = scores.bfloat16()
    v = (0.5 + torch.rand(n, 1, d, generator=gen(n), device=DEV)).bfloat16()
    kb.kda_kv4_write(k, v, cache, table)
    del k, v
    q = torch.zeros(seqs, heads, d, dtype=torch.bfloat16, device=DEV)
    q[..., 3] = 1
    lens = torch.full((seqs,), n, dtype=torch.int32, device=DEV)
    out, lse = kb.kda_kv4_attention(q, cache, table.expand(seqs, -1).contiguous(), lens, scale=1.0, want_lse=True)
    assert kb.kda_get_device_error() == 0
    parts = [spans(cache, table, 0, a, min(a + (1 << 20), n)) for a in range(0, n, 1 << 20)]
    scores = torch.cat([p[0][:, 0, 3] for p in parts])
    top = scores.max()
    w = (scores - top).exp()
    o = sum((w[i << 20:(i + 1) << 20][:, None] * vd[:, 0]).sum(0) for i, (_, vd) in enumerate(parts)) / w.sum()
    near(out, lse, (o, top + w.sum().log(), o), 2.0 ** -8, 1 << 14)
