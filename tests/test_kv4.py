"""The paged cache in 4 bits: kda_kv4_write and kda_kv4_read against the definition (bit for bit:
the quotient x / s of two bf16 values is never so near the middle of two whole numbers that 32 bits
would round it to the other side), kda_kv4_attention against 64 bits (tolerances:
attention_testlib), and their refusals."""
import ctypes
import math
import threading

import pytest
import torch

from attention_testlib import attend, check, cu_of, decode, paged, quantised, spans
from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, gen, randn


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def written(cache, table, page, start, lens, k, v):
    """The cache's arrays as the write should leave them, from those before."""
    want = [t.clone() for t in cache]
    at = 0
    for n, (a, length) in enumerate(zip(start, lens)):
        for i in range(length if a >= 0 else 0):
            slot = int(table[n, (a + i) // page]), (a + i) % page
            for j, x in ((0, k), (2, v)):
                g = x[at + i].double().unflatten(-1, (-1, 32))
                s = (g.abs().amax(-1).clamp(min=2.0 ** -64) / 7).float().bfloat16()
                want[j + 1][slot[0], :, slot[1]] = s
        at += length
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("start,lens", [([0], [1]), ([5, 0, 63, 16], [3, 0, 1, 40]), ([0, 300], [300, 17]),
                                        ([-1, 7, -5], [4, 9, 0])])
def test_what_is_written_is_read_back(start, lens, page, heads, d):
    g = gen(sum(lens) + page)
    T = sum(lens)
    k, v = (randn(g, T, heads, d, std=2.0, dtype=torch.bfloat16) for _ in range(2))
    k[:, :, ::7] *= 10
    table, pages = paged([max(a, 0) + n for a, n in zip(start, lens)], page)
    cache = kb.kda_kv4_cache(pages, page, heads, d)
    for t in cache:
        t.view(torch.uint8).fill_(0x5a)
    before = [t.clone() for t in cache]
    kb.kda_kv4_write(k, v, cache, table, ints(*start), cu_of(lens))
    assert kb.kda_get_device_error() == 0
    scales = written(before, table, page, start, lens, k, v)
    assert torch.equal(cache[1], scales[1]) and torch.equal(cache[3], scales[3])
    k2, v2 = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    kb.kda_kv4_read(cache, table, T, ints(*start), cu_of(lens), k=k2, v=v2)
    assert kb.kda_get_device_error() == 0
    at, touched = 0, torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    for n, (a, length) in enumerate(zip(start, lens)):
        rows = slice(at, at + length)
        if a < 0:
            assert (k2[rows] == 9).all() and (v2[rows] == 9).all()
        elif length:
            ck, cv = spans(cache, table, n, a, a + length)
            assert torch.equal(ck, quantised(k[rows])) and torch.equal(cv, quantised(v[rows]))
            assert torch.equal(k2[rows], ck.bfloat16()) and torch.equal(v2[rows], cv.bfloat16())
            pos = torch.arange(a, a + length, device=DEV)
            touched[table[n].long()[pos // page], pos % page] = True
        at += length
    for t, b in zip(cache, before):   # every other place is as it was
        assert torch.equal(t.transpose(1, 2)[~touched], b.transpose(1, 2)[~touched])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_uniform_spans_and_columns(d):
    g = gen(3)
    wide = randn(g, 6, 4 * d + 40, dtype=torch.bfloat16)
    k, v = (wide[:, 8 + a * d:8 + (a + 2) * d].unflatten(1, (2, d)) for a in (0, 2))
    table, pages = paged([2, 2, 2], 16)
    cache = kb.kda_kv4_cache(pages, 16, 2, d)
    kb.kda_kv4_write(k, v, cache, table)
    k2, v2 = kb.kda_kv4_read(cache, table, 6)
    assert torch.equal(k2, quantised(k).bfloat16()) and torch.equal(v2, quantised(v).bfloat16())
    four = [t.contiguous().view(3, 2, 2, d) for t in (k, v)]
    cache2 = kb.kda_kv4_cache(pages, 16, 2, d)
    kb.kda_kv4_write(*four, cache2, table)
    assert all(torch.equal(a, b) for a, b in zip(cache, cache2))
    buf = torch.full((6, 2 * d + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:, 8:8 + 2 * d].unflatten(1, (2, d))
    kb.kda_kv4_read(cache, table, 6, k=out, v=v2)
    assert torch.equal(out, k2) and (buf[:, :8] == 7).all() and (buf[:, 8 + 2 * d:] == 7).all()


@pytest.mark.gpu
def test_extreme_groups():
    x = torch.zeros(9, 1, 64, device=DEV)
    x[1, 0, 3] = 1e-30                    # below the least magnitude
    x[2, 0, :32] = 3e38
    x[3, 0, 5] = math.inf
    x[4, 0, 40] = math.nan
    x[5, 0, 0], x[5, 0, 1:] = -7.0, torch.arange(63, device=DEV) / 4 - 7.0
    x[6, 0] = 2.0 ** -64
    x[7, 0, :32] = 2.0 ** -126
    x[8, 0, 31] = -math.inf
    x = x.bfloat16()
    table, pages = paged([9], 16)
    cache = kb.kda_kv4_cache(pages, 16, 1, 64)
    kb.kda_kv4_write(x, x, cache, table)
    k, v = kb.kda_kv4_read(cache, table, 9)
    want = quantised(x).bfloat16()
    for got in (k, v):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert k[3, 0, :32].isnan().all() and (k[3, 0, 32:] == 0).all() and k[8, 0, :32].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 1000000, -2 ** 31])
def test_positions_without_a_page_are_reported(bad):
    k = randn(gen(1), 40, 2, 64, dtype=torch.bfloat16)
    table, pages = paged([40], 16, spare=0)
    cache = kb.kda_kv4_cache(pages, 16, 2, 64)
    kb.kda_kv4_write(k, k, cache, table)
    held = [t.clone() for t in cache]
    broken = table.clone()
    broken[0, 1] = bad
    kb.kda_kv4_write(-k, -k, cache, broken)
    assert kb.kda_get_device_error() == 5 and b"block_table" in kb.load().kda_last_error_message()
    page = int(table[0, 1])
    assert all(torch.equal(t[page], h[page]) for t, h in zip(cache, held))
    k2 = torch.full_like(k, 3.0)
    kb.kda_kv4_read(cache, broken, 40, k=k2)
    assert kb.kda_get_device_error() == 5
    assert (k2[16:32] == 3).all() and torch.equal(k2[:16], quantised(-k[:16]).bfloat16())
    # positions behind the table's last column
    kb.kda_kv4_read(cache, table, 40, ints(20))
    assert kb.kda_get_device_error() == 5
    q = randn(gen(2), 1, 2, 64, dtype=torch.bfloat16)
    kb.kda_kv4_attention(q, cache, broken, ints(40))
    assert kb.kda_get_device_error() == 5
    kb.kda_kv4_attention(q, cache, table, ints(1000))
    assert kb.kda_get_device_error() == 5
    kb.kda_kv4_attention(q, cache, broken, ints(16))    # the bad page is not reached
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 5, 4, 10], [1, 5, 8, 10], [0, 5, 8, 9], [0, 5, 8, 4000], [0, -7, 8, 10]])
def test_malformed_cu_seqlens_are_reported(cu):
    k = randn(gen(1), 10, 2, 64, dtype=torch.bfloat16)
    table, pages = paged([16, 16, 16], 16)
    cache = kb.kda_kv4_cache(pages, 16, 2, 64)
    kb.kda_kv4_write(k, k, cache, table, None, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert kb.kda_get_device_error() == 5
    kb.kda_kv4_read(cache, table, 10, None, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert kb.kda_get_device_error() == 5


# ---- attention over the cache
def filled(lens, page, heads, d, seed=0, std=1.0):
    """A cache in which sequences of those lengths lie, and its block table."""
    g = gen(seed)
    T = sum(lens)
    table, pages = paged(lens, page, seed=seed)
    cache = kb.kda_kv4_cache(pages, page, heads, d)
    for t in cache:   # what lies behind a sequence's last token: scales of NaN, codes of any kind
        t.view(torch.uint8).fill_(0xff)
    if T:
        k, v = (randn(g, T, heads, d, std=s, dtype=torch.bfloat16) for s in (std, 1.0))
        kb.kda_kv4_write(k, v, cache, table, None, cu_of(lens))
    return cache, table


def over_cache(q, cache, table, lens, scale):
    """The definition: o, lse, m, X of all queries."""
    parts = []
    for n, length in enumerate(lens):
        k, v = spans(cache, table, n, 0, max(length, 0))
        reach = [length - q.shape[1] + 1 + i for i in range(q.shape[1])]
        parts.append(attend(q[n], k, v, scale, reach))
    return [torch.stack([p[j] for p in parts]) for j in range(4)]


def run(lens, tokens, heads, kv_heads, d, page, seed=0, std=1.0, scale=None):
    cache, table = filled([max(n, 0) for n in lens], page, kv_heads, d, seed, std)
    q = randn(gen(seed + 1), len(lens), tokens, heads, d, std=std, dtype=torch.bfloat16)
    out, lse = kb.kda_kv4_attention(q, cache, table, ints(*lens), want_lse=True, scale=scale)
    assert kb.kda_get_device_error() == 0
    ref = over_cache(q, cache, table, lens, d ** -0.5 if scale is None else scale)
    check(out, lse, ref, d)
    return q, cache, table, out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 2), (6, 2), (8, 1), (16, 1), (12, 4), (40, 2)])
@pytest.mark.parametrize("lens", [[1], [0, 17, 16, 15], [100, 333, 64, 1, 0, 31]])
def test_one_token_over_the_cache(lens, heads, kv_heads, d):
    run(lens, 1, heads, kv_heads, d, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("tokens", [1, 2, 4, 7])
def test_drafts_and_page_sizes(tokens, page):
    """Sequences shorter than the draft among them: queries that reach nothing."""
    run([130, 3, 0, 513, 2, 64], tokens, 6, 2, 128, page)
    run([41, 1], tokens, 4, 4, 64, page)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,tokens,d", [(32, 8, 1, 128), (8, 1, 5, 64), (64, 1, 3, 128)])
@pytest.mark.parametrize("lens", [[9000], [5000, 40, 7001]])
def test_long_sequences(lens, heads, kv_heads, tokens, d):
    run(lens, tokens, heads, kv_heads, d, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,tokens", [(96, 1), (128, 1), (192, 2), (40, 5)])
def test_large_groups_and_drafts(heads, tokens):
    run([300, 0, 17, 2100], tokens, heads, 1, 128, 32)
    run([30, 3], tokens, heads, 1, 64, 32)


@pytest.mark.gpu
def test_many_sequences():
    lens = [(37 * i) % 500 for i in range(300)]
    run(lens, 1, 4, 1, 128, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("std,scale", [(8.0, None), (1.0, 3.0), (0.01, None), (3.0, 1e-3)])
def test_sharp_and_flat_scores(std, scale):
    run([1500, 200], 2, 4, 2, 128, 16, std=std, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("size,scale", [(0.0, 1e-20), (0.0, 1e-38), (2.0 ** -120, 1e-20), (2.0 ** 105, None)])
def test_queries_of_zeros_and_of_extreme_sizes(size, scale):
    lens = [40, 3, 700]
    cache, table = filled(lens, 16, 2, 128)
    q = randn(gen(3), 3, 2, 4, 128, dtype=torch.bfloat16) * size
    q[:, 1, 0] = 0
    out, lse = kb.kda_kv4_attention(q, cache, table, ints(*lens), want_lse=True, scale=scale)
    check(out, lse, over_cache(q, cache, table, lens, 128 ** -0.5 if scale is None else scale), 128)


@pytest.mark.gpu
def test_short_sequences_in_graphs():
    """Units of one warp each, replayed with lengths that make them the whole block's, and back."""
    cache, table = filled([900, 60, 700, 50], 16, 2, 128)
    q = randn(gen(5), 4, 2, 8, 128, dtype=torch.bfloat16)
    sl = ints(30, 60, 1, 50)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        kb.kda_kv4_attention(q, cache, table, sl, out=out)
    for lens in ([30, 60, 1, 50], [900, 60, 700, 50], [0, 0, 0, 1], [0, 0, 0, 0], [900, 0, 0, 0]):
        sl.copy_(ints(*lens))
        out.fill_(7.0)
        graph.replay()
        ref = over_cache(q, cache, table, lens, 128 ** -0.5)
        check(out, None, ref, 128)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_lengths_below_zero_count_as_none():
    cache, table = filled([20, 20], 16, 2, 64)
    q = randn(gen(1), 2, 4, 64, dtype=torch.bfloat16)
    out, lse = kb.kda_kv4_attention(q, cache, table, ints(-5, 20), want_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and out[1].isfinite().all()
    out, lse = kb.kda_kv4_attention(q, cache, table, ints(-2 ** 31, 0), want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all() and kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_groups_that_stand_for_nan():
    """A value's group of NaN reaches the queries that reach it, in its channels; a later one none."""
    lens = [80]
    g = gen(7)
    k, v = (randn(g, 80, 1, 128, dtype=torch.bfloat16) for _ in range(2))
    v[40, 0, 70] = math.inf
    table, pages = paged(lens, 16)
    cache = kb.kda_kv4_cache(pages, 16, 1, 128)
    kb.kda_kv4_write(k, v, cache, table)
    q = randn(g, 1, 2, 128, dtype=torch.bfloat16)
    out, lse = kb.kda_kv4_attention(q, cache, table, ints(80), want_lse=True)
    nan = out.isnan()
    assert nan[..., 64:96].all() and not nan[..., :64].any() and not nan[..., 96:].any() and lse.isfinite().all()
    assert kb.kda_kv4_attention(q, cache, table, ints(40))[0].isfinite().all()
    k[40, 0, 3] = math.nan
    kb.kda_kv4_write(k, v, cache, table)
    assert kb.kda_kv4_attention(q, cache, table, ints(41))[0].isnan().all()
    assert kb.kda_kv4_attention(q, cache, table, ints(40))[0].isfinite().all()


@pytest.mark.gpu
def test_columns_streams_graphs_and_threads():
    lens = [700, 90, 0]
    q, cache, table, want, want_lse = run(lens, 2, 8, 2, 128, 64)
    wide = torch.full((3, 2, 8 * 128 + 32), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[..., 16:16 + 1024].unflatten(2, (8, 128))
    sl = ints(*lens)
    qs = torch.zeros_like(wide)[..., 8:8 + 1024].unflatten(2, (8, 128)).copy_(q)
    kb.kda_kv4_attention(qs, cache, table, sl, out=out)
    assert torch.equal(out, want) and (wide[..., :16] == 7).all() and (wide[..., 1040:] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kb.kda_kv4_attention(q, cache, table, sl, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    # two captured graphs, replayed side by side and over lengths that change
    graphs, outs, streams = [], [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        outs.append(torch.empty_like(q))
        with torch.cuda.graph(graphs[-1]):
            kb.kda_kv4_attention(q, cache, table, sl, out=outs[-1])
        streams.append(torch.cuda.Stream())
    for new in (lens, [3, 89, 1], [650, 0, 0]):
        sl.copy_(ints(*new)) if new[2] == 0 else sl.copy_(ints(new[0], new[1], 0))
        want = kb.kda_kv4_attention(q, cache, table, sl)[0]
        torch.cuda.synchronize()
        for _ in range(10):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    results = [None] * 2

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                results[i] = kb.kda_kv4_attention(q, cache, table, sl)[0]
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert torch.equal(results[0], want) and torch.equal(results[1], want)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_tables_with_wide_rows_and_shared_pages():
    """Rows of a wider table, and two sequences that begin with the same pages."""
    cache, table = filled([128, 128], 16, 2, 128)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device=DEV)
    wide[:, 3:11] = table
    wide[1, 3:7] = table[0, :4]
    part = wide[:, 3:11]
    q = randn(gen(3), 2, 1, 4, 128, dtype=torch.bfloat16)
    out, lse = kb.kda_kv4_attention(q, cache, part, ints(128, 128), want_lse=True)
    assert kb.kda_get_device_error() == 0
    check(out, lse, over_cache(q, cache, part, [128, 128], 128 ** -0.5), 128)


@pytest.mark.gpu
@pytest.mark.parametrize("big", [torch.uint8])
def test_a_cache_of_more_than_2_to_the_31_bytes(big):
    """Slots whose codes lie behind 2^31 bytes."""
    pages, page, heads, d = 70_000, 64, 8, 128
    cache = kb.kda_kv4_cache(pages, page, heads, d)
    table = torch.tensor([[69_998, 69_999]], dtype=torch.int32, device=DEV)
    small = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    few = kb.kda_kv4_cache(2, page, heads, d)
    k, v = (randn(gen(4), 100, heads, d, dtype=torch.bfloat16) for _ in range(2))
    q = randn(gen(5), 1, 16, d, dtype=torch.bfloat16)
    for c, t in ((cache, table), (few, small)):
        kb.kda_kv4_write(k, v, c, t)
    a, b = kb.kda_kv4_read(cache, table, 100), kb.kda_kv4_read(few, small, 100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(kb.kda_kv4_attention(q, cache, table, ints(100))[0],
                       kb.kda_kv4_attention(q, few, small, ints(100))[0])
    assert kb.kda_get_device_error() == 0
    del cache
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_nothing_to_do():
    cache, table = filled([16, 16], 16, 2, 64)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    kb.kda_kv4_write(e, e, cache, table, None, cu_of([0, 0]))
    k, v = kb.kda_kv4_read(cache, table, 0, None, cu_of([0, 0]))
    assert k.shape == (0, 2, 64)
    kb.kda_kv4_write(e, e, cache, table[:0], ints(), cu_of([]))
    out, lse = kb.kda_kv4_attention(e, cache, table[:0], ints(), want_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, _ = kb.kda_kv4_attention(torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device=DEV), cache, table,
                                  ints(3, 4))
    assert out.shape == (2, 0, 2, 64)
    # a cache without pages: sequences of no positions
    none = kb.kda_kv4_cache(0, 16, 2, 64)
    q = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, _ = kb.kda_kv4_attention(q, none, torch.empty(2, 0, dtype=torch.int32, device=DEV), ints(0, 0))
    assert (out == 0).all() and kb.kda_get_device_error() == 0


# ---- refusals: on the host, before anything is launched
BASE = 1 << 40


def P(i, off=0):
    return BASE + (i << 34) + off


def cache_of(**over):
    c = dict(k_codes=P(0), k_scales=P(1), v_codes=P(2), v_scales=P(3), n_pages=10, page_size=64, n_kv_heads=2,
             d=128)
    c.update(over)
    return kb.KdaKv4Cache(**c)


SPAN = dict(k=P(4), ld_k=256, v=P(5), ld_v=256, cache=None, table=P(6), ld_table=8, width=8, start=P(7), cu=P(8),
            T=10, N=2, stream=None)
ATTN = dict(q=P(4), ld_q=512, cache=None, table=P(6), ld_table=8, width=8, lens=P(7), out=P(9), ld_out=512,
            lse=P(10), N=2, tokens=1, heads=4, scale=1.0, stream=None)


def call(name, base, over):
    p, c = dict(base), {}
    for key, value in over.items():
        (p if key in p else c)[key] = value
    if "no_cache" not in c:
        p["cache"] = ctypes.byref(cache_of(**c))
    return getattr(kb.load(), name)(*p.values())


CACHE_REFUSALS = [
    (dict(no_cache=1), b"cache is NULL"), (dict(n_pages=-1), b"n_pages=-1"), (dict(width=-1), b"max_pages=-1"),
    (dict(n_kv_heads=0), b"n_kv_heads=0"), (dict(k_codes=None), b"k_codes is NULL"),
    (dict(v_scales=None), b"v_scales is NULL"), (dict(v_codes=P(2, 8)), b"v_codes is not 16-byte aligned"),
    (dict(k_scales=P(1, 2)), b"k_scales is not 16-byte aligned"), (dict(table=None), b"block_table is NULL"),
    (dict(table=P(6, 2)), b"block_table is not aligned"), (dict(ld_table=7), b"leading dimension"),
]


@pytest.mark.parametrize("name", ["kda_kv4_write", "kda_kv4_read"])
@pytest.mark.parametrize("over,word", CACHE_REFUSALS + [
    (dict(T=-1), b"total_tokens=-1"), (dict(N=-1), b"n_seqs=-1"), (dict(N=0), b"n_seqs = 0"),
    (dict(cu=None, T=9), b"not a multiple of n_seqs"), (dict(k=None), b"k is NULL"), (dict(v=None), b"v is NULL"),
    (dict(k=P(4, 8)), b"16-byte"), (dict(ld_v=260), b"16-byte"), (dict(ld_k=255), b"leading dimension"),
    (dict(start=P(7, 1)), b"start is not aligned"), (dict(cu=P(8, 2)), b"cu_seqlens is not aligned"),
])
def test_span_refusals(name, over, word):
    assert call(name, SPAN, over) == 1
    assert word in kb.load().kda_last_error_message()


@pytest.mark.parametrize("over,word", [
    (dict(k=P(0)), b"k_codes overlaps k"), (dict(v=P(3)), b"v_scales overlaps v"),
    (dict(table=P(2)), b"v_codes overlaps block_table"), (dict(cu=P(1)), b"k_scales overlaps cu_seqlens"),
    (dict(v_codes=P(0, 4096)), b"v_codes overlaps k_codes"), (dict(k_scales=P(0)), b"k_scales overlaps k_codes"),
])
def test_write_refuses_overlaps(over, word):
    assert call("kda_kv4_write", SPAN, over) == 1
    assert word in kb.load().kda_last_error_message()


@pytest.mark.parametrize("over,word", [
    (dict(k=P(0)), b"k overlaps k_codes"), (dict(v=P(4)), b"v overlaps k"), (dict(v=P(6)), b"v overlaps block_table"),
])
def test_read_refuses_overlaps(over, word):
    assert call("kda_kv4_read", SPAN, over) == 1
    assert word in kb.load().kda_last_error_message()


@pytest.mark.parametrize("over,word", CACHE_REFUSALS + [
    (dict(N=-1), b"n_seqs=-1"), (dict(tokens=-1), b"n_tokens=-1"), (dict(heads=3), b"not a multiple"),
    (dict(heads=0), b"n_heads=0"), (dict(scale=0.0), b"scale"), (dict(scale=math.nan), b"scale"),
    (dict(q=None), b"q is NULL"), (dict(lens=None), b"seq_lens is NULL"), (dict(out=None), b"out is NULL"),
    (dict(q=P(4, 2)), b"16-byte"), (dict(ld_out=516), b"16-byte"), (dict(ld_q=500), b"leading dimension"),
    (dict(lens=P(7, 3)), b"seq_lens is not aligned"), (dict(lse=P(10, 2)), b"lse is not aligned"),
    (dict(out=P(4)), b"out overlaps q"), (dict(out=P(3)), b"out overlaps v_scales"),
    (dict(lse=P(9)), b"lse overlaps out"), (dict(lse=P(6)), b"lse overlaps block_table"),
])
def test_attention_refusals(over, word):
    assert call("kda_kv4_attention", ATTN, over) == 1
    assert word in kb.load().kda_last_error_message()


@pytest.mark.parametrize("name,base", [("kda_kv4_write", SPAN), ("kda_kv4_read", SPAN), ("kda_kv4_attention", ATTN)])
def test_unsupported_and_empty(name, base):
    for over in (dict(d=96), dict(d=256), dict(page_size=8), dict(page_size=48), dict(page_size=1 << 17)):
        assert call(name, base, over) == 2
    assert call(name, base, dict(N=0, T=0) if base is SPAN else dict(N=0)) == 0


@pytest.mark.parametrize("name,base", [("kda_kv4_write", SPAN), ("kda_kv4_read", SPAN), ("kda_kv4_attention", ATTN)])
def test_caches_whose_rows_could_not_be_counted_are_refused(name, base):
    for over in (dict(n_kv_heads=32768, page_size=65536), dict(n_kv_heads=16384, page_size=65536, n_pages=(1 << 18) + 1)):
        assert call(name, base, over) == 2
        assert b"n_kv_heads=" in kb.load().kda_last_error_message()
