"""kda_attention_fwd against the definition in 64 bits (tolerances: attention_testlib), and its
refusals."""
import ctypes
import math
import threading

import pytest
import torch

from attention_testlib import check, cu_of, qkv, reference
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, gen, randn


def run(q, k, v, q_lens, k_lens, causal=True, scale=None, packed=True, **kw):
    d = q.shape[-1]
    cu = (cu_of(q_lens), cu_of(k_lens)) if packed else (None, None)
    out, lse = kb.kda_attention_fwd(q, k, v, *cu, n_seqs=len(q_lens), causal=causal, scale=scale, want_lse=True,
                                    **kw)
    assert kb.kda_get_device_error() == 0
    check(out, lse, reference(q, k, v, q_lens, k_lens, d ** -0.5 if scale is None else scale, causal), d)
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 1), (6, 2), (5, 1), (16, 1), (8, 8)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3], [130], [0, 64, 65, 127, 128, 129, 0], [300, 1, 257]])
def test_packed_prompts(lens, heads, kv_heads, d):
    q, k, v = qkv(gen(sum(lens) + heads), sum(lens), sum(lens), heads, kv_heads, d)
    run(q, k, v, lens, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [500]), ([5, 0, 70], [133, 20, 70]), ([130], [1000]),
                                           ([3, 200], [600, 384]), ([1, 1, 1], [1, 128, 129]),
                                           # fewer keys than queries: rows that reach none
                                           ([300, 2], [40, 0]), ([129, 5, 256], [0, 2, 255])])
def test_queries_behind_earlier_keys(q_lens, k_lens, causal):
    q, k, v = qkv(gen(sum(k_lens)), sum(q_lens), sum(k_lens), 6, 2, 128)
    run(q, k, v, q_lens, k_lens, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,d,length", [(4, 2, 128, 777), (12, 4, 64, 400), (32, 2, 128, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_uniform_batches(heads, kv_heads, d, length, causal):
    q, k, v = qkv(gen(length), 3 * length, 3 * length, heads, kv_heads, d)
    out, lse = run(q, k, v, [length] * 3, [length] * 3, causal, packed=False)
    four = [t.unflatten(0, (3, length)) for t in (q, k, v)]
    out4, lse4 = kb.kda_attention_fwd(*four, causal=causal, want_lse=True)
    assert torch.equal(out4.flatten(0, 1), out) and torch.equal(lse4.flatten(0, 1), lse)
    none = kb.kda_attention_fwd(*four, causal=causal)
    assert none[1] is None and torch.equal(none[0], out4)


@pytest.mark.gpu
@pytest.mark.parametrize("std,scale", [(8.0, None), (1.0, 3.0), (0.01, None), (3.0, 1e-3)])
def test_sharp_and_flat_scores(std, scale):
    """Scores of some hundreds, where one key holds all of a row and the maximum keeps growing, and
    scores that are all alike."""
    q, k, v = qkv(gen(3), 500, 500, 4, 2, 128, std)
    k *= torch.linspace(0.1, 2.0, 500, device=DEV)[:, None, None].bfloat16()
    run(q, k, v, [500], [500], scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[300, 70], [5000]])
def test_scores_beyond_whole_numbers_of_32_bits(lens):
    """Scores of 2^24 to 2^100: one key has all of a row.  Keys of one value in all channels and
    queries of signs, so that scores are multiples of powers of two, summed exactly."""
    g = gen(21)
    rows = 50
    for power in (14, 20, 40, 100):
        q = torch.where(torch.rand(rows, 4, 128, generator=g, device=DEV) < 0.5, -1.0, 1.0).bfloat16()
        k = torch.zeros(sum(lens), 2, 128, dtype=torch.bfloat16, device=DEV)
        at = torch.randperm(sum(lens), generator=torch.Generator().manual_seed(3)).to(DEV)
        k[:, :, 0] = (2.0 ** power * (at % 251 - 125))[:, None].bfloat16()
        v = randn(g, sum(lens), 2, 128, dtype=torch.bfloat16)
        q_lens = [rows - 10, 10] if len(lens) > 1 else [rows]
        out, lse = kb.kda_attention_fwd(q, k, v, cu_of(q_lens), cu_of(lens), scale=1.0, want_lse=True)
        o, l, m, _ = reference(q, k, v, q_lens, lens, 1.0)
        # (exact scores, whose differences are 0 or at least 2^power)
        check(out, lse, (o, l, m, torch.zeros_like(l)), 128)


@pytest.mark.gpu
def test_a_long_sequence():
    q, k, v = qkv(gen(5), 20, 5000, 8, 1, 128)
    run(q, k, v, [20], [5000])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens", [([3, 0, 70, 1], [2900, 10, 3333, 513]), ([300], [2000]),
                                           ([40, 5], [1, 4000]), ([260, 260], [130, 1000])])
def test_keys_shared_by_several_blocks(q_lens, k_lens, causal, d):
    """Few rows over many keys, and rows that reach none of a part's keys, or none at all."""
    q, k, v = qkv(gen(sum(k_lens)), sum(q_lens), sum(k_lens), 6, 1, d, std=2.0)
    run(q, k, v, q_lens, k_lens, causal)
    first = kb.kda_attention_fwd(q, k, v, cu_of(q_lens), cu_of(k_lens), causal=causal)[0]
    for _ in range(3):
        again = kb.kda_attention_fwd(q, k, v, cu_of(q_lens), cu_of(k_lens), causal=causal)[0]
        assert torch.equal(again, first)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,tq,tk", [(3, 200, 1500), (1, 1100, 1100), (2, 600, 130), (5, 33, 2049)])
def test_uniform_batches_cut_into_parts(n, tq, tk, causal):
    q, k, v = qkv(gen(tq), n * tq, n * tk, 4, 2, 128)
    run(q, k, v, [tq] * n, [tk] * n, causal, packed=False)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [96, 128, 192, 256])
def test_large_groups(heads):
    """Few tokens to a tile, down to one; groups of more heads than a tile has rows."""
    lens = [5, 0, 1, 140]
    q, k, v = qkv(gen(heads), sum(lens), sum(lens), heads, 1, 64)
    run(q, k, v, lens, lens)
    q, k, v = qkv(gen(heads), 3, 2000, heads, 1, 128)
    run(q, k, v, [1, 2], [700, 1300])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [64, 65, 100])
def test_many_sequences_with_few_heads(n):
    """More sequences than the line holds, some long enough to be cut."""
    q_lens = [(7 * i) % 5 for i in range(n)]
    k_lens = [(131 * i) % 400 if i % 33 else 3000 for i in range(n)]
    q, k, v = qkv(gen(n), sum(q_lens), sum(k_lens), 2, 1, 128)
    run(q, k, v, q_lens, k_lens)
    run(q, k, v, q_lens, k_lens, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinite_values_in_one_part_of_the_keys(bad):
    q, k, v = qkv(gen(18), 40, 3000, 4, 1, 128)
    want = kb.kda_attention_fwd(q, k, v)[0]
    for at in (0, 1000, 2959, 2960, 2975, 2999):
        v2 = v.clone()
        v2[at, 0, 7] = bad
        out = kb.kda_attention_fwd(q, k, v2)[0]
        first = max(0, at - 2960)   # the first query that reaches it
        hit = out[first:, :, 7].float()
        assert hit.isnan().all() if bad != bad else (hit == bad).all()
        out[first:, :, 7] = want[first:, :, 7]
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_columns_of_wider_buffers(d):
    g = gen(9)
    lens = [150, 0, 31]
    wide = randn(g, 181, 8 * d + 48, dtype=torch.bfloat16)
    q, k, v = (wide[:, 8 + a * d:8 + b * d].unflatten(1, (b - a, d)) for a, b in ((0, 4), (4, 6), (6, 8)))
    buf = torch.full((181, 4 * d + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:, 16:16 + 4 * d].unflatten(1, (4, d))
    got, _ = run(q, k, v, lens, lens, out=out)
    assert got is out and (buf[:, :16] == 7).all() and (buf[:, 16 + 4 * d:] == 7).all()
    lse = torch.empty(181, 4, device=DEV)
    dense, lse2 = kb.kda_attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), cu_of(lens), lse=lse)
    assert lse2 is lse and torch.equal(dense, out)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("causal", [True, False])
def test_what_a_query_does_not_reach_has_no_influence(bad, causal):
    """Keys and values of other sequences, later ones of the same, and rows behind the last."""
    lens = [70, 100, 200, 33]
    T = sum(lens)
    q, k, v = qkv(gen(11), T, T, 4, 2, 128)
    want, want_lse = run(q, k, v, lens, lens, causal)
    for at in (0, 69, 70, 169, 170, 299, 300, 369, 370, 402):
        k2, v2 = k.clone(), v.clone()
        k2[at], v2[at] = bad, bad
        out, lse = kb.kda_attention_fwd(q, k2, v2, cu_of(lens), causal=causal, want_lse=True)
        first = 0
        for n in lens:
            clean = slice(first, first + n)
            if first <= at < first + n:
                clean = slice(first, at if causal else first)
            assert torch.equal(out[clean], want[clean]), (at, first)
            assert torch.equal(lse[clean], want_lse[clean])
            first += n
    # a value alone: the queries that reach it get it, in its channel
    for at in (170, 251, 369):
        v2 = v.clone()
        v2[at, 1, 5] = bad
        out, _ = kb.kda_attention_fwd(q, k, v2, cu_of(lens), causal=causal)
        reached = torch.zeros(T, dtype=torch.bool, device=DEV)
        reached[at if causal else 170:370] = True
        hit = out[reached][:, 2:, 5].float()
        assert hit.isnan().all() if bad != bad else (hit == bad).all()
        out[reached, 2:, 5] = want[reached, 2:, 5]
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_scores_that_are_infinite_or_nan():
    """A key a query does reach: an infinite score takes the whole row (NaN), one of minus infinity
    has no part in it."""
    q, k, v = qkv(gen(12), 64, 64, 1, 1, 64)
    q.abs_()
    k2 = k.clone()
    k2[10] = -math.inf
    out, lse = kb.kda_attention_fwd(q, k2, v, cu_of([64]), want_lse=True)
    keep = [i for i in range(64) if i != 10]
    # without key 10: queries behind it, over one key less
    check(out[11:], lse[11:], reference(q[11:], k[keep], v[keep], [53], [63], 0.125), 64)
    k2[10] = math.nan
    out, lse = kb.kda_attention_fwd(q, k2, v, cu_of([64]), want_lse=True)
    assert out[10:].isnan().all() and lse[10:].isnan().all() and out[:10].isfinite().all()
    k2[10] = math.inf
    out, _ = kb.kda_attention_fwd(q, k2, v, cu_of([64]))
    assert out[10:].isnan().all() and out[:10].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[0, 0], []])
def test_nothing_to_do(lens):
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = kb.kda_attention_fwd(q, k, k, cu_of(lens), want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # queries without any key
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = kb.kda_attention_fwd(q, k, k, want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
def test_results_do_not_depend_on_the_run():
    lens = [900, 33, 0, 410]
    q, k, v = qkv(gen(13), sum(lens), sum(lens), 8, 2, 128)
    first = kb.kda_attention_fwd(q, k, v, cu_of(lens))[0]
    for _ in range(5):
        assert torch.equal(kb.kda_attention_fwd(q, k, v, cu_of(lens))[0], first)
    # what else is in the batch may change how keys are shared by blocks, so it changes no more
    # than roundings
    alone = kb.kda_attention_fwd(q[:900], k[:900], v[:900], cu_of([900]), want_lse=True)
    check(*alone, reference(q[:900], k[:900], v[:900], [900], [900], 128 ** -0.5), 128)


@pytest.mark.gpu
def test_streams_graphs_and_threads():
    lens = [200, 300]
    q, k, v = qkv(gen(14), 500, 500, 4, 2, 128)
    cu = cu_of(lens)
    want = kb.kda_attention_fwd(q, k, v, cu)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kb.kda_attention_fwd(q, k, v, cu, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        kb.kda_attention_fwd(q, k, v, cu, out=out)
    q2, k2, v2 = qkv(gen(15), 500, 500, 4, 2, 128)
    want2 = kb.kda_attention_fwd(q2, k2, v2, cu_of([500, 0]))[0]
    for a, b in ((q, q2), (k, k2), (v, v2)):
        a.copy_(b)
    cu.copy_(cu_of([500, 0]))
    graph.replay()
    assert torch.equal(out, want2)
    results = [None] * 2

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                results[i] = kb.kda_attention_fwd(q, k, v, cu)[0]
        s.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert torch.equal(results[0], want2) and torch.equal(results[1], want2)


@pytest.mark.gpu
def test_shared_keys_in_graphs_and_threads():
    """The calls that take a workspace: two captured graphs replayed side by side, two threads."""
    q, k, v = qkv(gen(19), 40, 6000, 8, 1, 128)
    cq, ck = cu_of([30, 10]), cu_of([4000, 2000])
    graphs, outs, streams = [], [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        outs.append((torch.empty_like(q), torch.empty(40, 8, device=DEV)))
        with torch.cuda.graph(graphs[-1]):
            kb.kda_attention_fwd(q, k, v, cq, ck, out=outs[-1][0], lse=outs[-1][1])
        streams.append(torch.cuda.Stream())
    for q_lens, k_lens in (([30, 10], [4000, 2000]), ([40, 0], [0, 6000]), ([1, 39], [5999, 1])):
        cq.copy_(cu_of(q_lens))
        ck.copy_(cu_of(k_lens))
        want = kb.kda_attention_fwd(q, k, v, cq, ck, want_lse=True)
        check(*want, reference(q, k, v, q_lens, k_lens, 128 ** -0.5), 128)
        torch.cuda.synchronize()
        for _ in range(10):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    results = [None] * 2

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                results[i] = kb.kda_attention_fwd(q, k, v, cq, ck)[0]
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert torch.equal(results[0], want[0]) and torch.equal(results[1], want[0])
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_batches_of_unlike_numbers_are_refused():
    q, k = (torch.zeros(b, 8, 2, 64, dtype=torch.bfloat16, device=DEV) for b in (2, 4))
    with pytest.raises(kb.KdaError, match="q has 2 sequences, k 4"):
        kb.kda_attention_fwd(q, k, k)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 5, 4, 10], [1, 5, 8, 10], [0, 5, 8, 9], [0, 5, 8, 4000], [0, -7, 8, 10]])
def test_malformed_cu_seqlens_are_reported(cu):
    q, k, v = qkv(gen(16), 10, 10, 2, 1, 64)
    for which in (0, 1):
        good = cu_of([5, 3, 2])
        bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
        kb.kda_attention_fwd(q, k, v, *((bad, good) if which == 0 else (good, bad)))
        assert kb.kda_get_device_error() == 5
        assert b"cu_seqlens" in kb.load().kda_last_error_message()
    run(q, k, v, [5, 3, 2], [5, 3, 2])


@pytest.mark.gpu
def test_tokens_far_apart():
    """Places behind 2^31 elements: the results of the same tokens side by side."""
    pitch = 2_400_000_000 // 8 * 8
    q, k, v = qkv(gen(17), 3, 3, 4, 2, 64)
    want = kb.kda_attention_fwd(q, k, v)[0]
    buf = torch.empty(2 * pitch + 4096, dtype=torch.bfloat16, device=DEV)
    far = []
    for i, (t, heads) in enumerate(((q, 4), (k, 2), (v, 2), (torch.zeros_like(q), 4))):
        far.append(buf.as_strided((3, heads, 64), (pitch, 64, 1), 512 * i).copy_(t))
    kb.kda_attention_fwd(*far[:3], out=far[3])
    assert torch.equal(far[3], want) and kb.kda_get_device_error() == 0
    del far, buf
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_tensors_with_other_strides_are_refused():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    for t in (torch.zeros(2, 64, 4, dtype=torch.bfloat16, device=DEV).transpose(1, 2),
              torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV)[:, ::2]):
        with pytest.raises(kb.KdaError, match="heads of a token must be dense"):
            kb.kda_attention_fwd(q, t, q)
    with pytest.raises(kb.KdaError, match="16-byte"):
        kb.kda_attention_fwd(q, q, torch.zeros(600, dtype=torch.bfloat16, device=DEV)[1:513].view(2, 4, 64))


# ---- refusals: on the host, before anything is launched
BASE = 1 << 40


def P(i, off=0):
    return ctypes.c_void_p(BASE + (i << 32) + off)


def call(**over):
    p = dict(q=P(0), ld_q=512, k=P(1), ld_k=256, v=P(2), ld_v=256, cu_q=P(3), cu_k=P(4), out=P(5), ld_out=512,
             lse=P(6), Tq=10, Tk=20, N=2, H=4, Hk=2, d=128, scale=1.0, causal=1, stream=None)
    p.update(over)
    return kb.load().kda_attention_fwd(*p.values())


@pytest.mark.parametrize("over,word", [
    (dict(Tq=-1), b"total_q=-1"), (dict(Tk=-1), b"total_k=-1"), (dict(N=-1), b"n_seqs=-1"),
    (dict(N=0), b"n_seqs = 0"), (dict(H=0), b"n_heads=0"), (dict(Hk=0), b"n_kv_heads=0"),
    (dict(H=3), b"not a multiple"), (dict(scale=0.0), b"scale"), (dict(scale=-1.0), b"scale"),
    (dict(scale=math.inf), b"scale"), (dict(scale=math.nan), b"scale"),
    (dict(cu_q=None), b"cu_seqlens_q is NULL"), (dict(cu_k=None), b"cu_seqlens_k is NULL"),
    (dict(cu_q=None, cu_k=None, Tq=9), b"not a multiple of n_seqs"),
    (dict(cu_q=None, cu_k=None, Tk=9), b"not a multiple of n_seqs"),
    (dict(q=None), b"q is NULL"), (dict(k=None), b"k is NULL"), (dict(v=None), b"v is NULL"),
    (dict(out=None), b"out is NULL"), (dict(q=P(0, 8)), b"16-byte"), (dict(k=P(1, 2)), b"16-byte"),
    (dict(ld_v=257), b"16-byte"), (dict(ld_out=511), b"leading dimension"), (dict(ld_k=200), b"leading dimension"),
    (dict(out=P(5, 8)), b"16-byte"), (dict(q=P(0, 1)), b"not aligned"), (dict(lse=P(6, 2)), b"not aligned"),
    (dict(cu_q=P(3, 2)), b"not aligned"), (dict(out=P(0)), b"out overlaps q"), (dict(out=P(2)), b"out overlaps v"),
    (dict(lse=P(1)), b"lse overlaps k"), (dict(lse=P(5, 16)), b"lse overlaps out"),
    (dict(lse=P(3)), b"lse overlaps cu_seqlens_q"),
])
def test_refusals(over, word):
    assert call(**over) == 1
    assert word in kb.load().kda_last_error_message()


def test_a_scale_that_overflows_is_refused():
    assert call(scale=3e38) == 1 and b"scale" in kb.load().kda_last_error_message()


def test_unsupported_and_empty():
    assert call(d=96) == 2 and call(d=256) == 2
    assert call(Tq=1 << 31) == 2 and call(H=65538, ld_q=65538 * 128, ld_out=65538 * 128) == 2
    assert call(Tq=0) == 0
    assert call(Tq=0, q=None, out=None, cu_q=None, cu_k=None, N=0, Tk=0) == 0
