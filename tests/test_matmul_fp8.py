"""kda_matmul_fp8 against 64 bits, and its refusals.

Tolerance.  The products of two e4m3 values are exact.  Per 32 of them the tensor core adds once
to a 32-bit sum, and per 128 there is a scaling and an addition in registers: K / 25 additions,
each within one unit of the last place (it may truncate) of at most the sum of the terms'
magnitudes, and 8 more for the sums inside a product, the scales' product and the scaling.
Then the output's own half ulp."""
import ctypes

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, assert_near, gen, half_ulp


def operand(g, rows, K, blocks_rows, seed_scale=1.0):
    """Random e4m3 values over their whole range, rows on 16-byte boundaries, and scales."""
    v = torch.randn(rows, K + -K % 16, device=DEV, generator=g) * 60
    v = v.clamp(-448, 448).to(torch.float8_e4m3fn)[:, :K]
    n = rows if blocks_rows == 1 else -(-rows // 128)
    s = torch.exp(torch.randn(n, -(-K // 128), device=DEV, generator=g)) * seed_scale
    return v, s


def reference(a, sa, b, sb):
    K = a.shape[1]
    kb_ = torch.arange(K, device=DEV) // 128
    a64 = a.double() * sa.double()[:, kb_]
    b64 = b.double() * sb.double()[torch.arange(b.shape[0], device=DEV) // 128][:, kb_]
    return a64 @ b64.t(), a64.abs() @ b64.abs().t()


def check(M, N, K, dtype, seed=0):
    g = gen(seed + M + 3 * N + 7 * K)
    a, sa = operand(g, M, K, 1)
    b, sb = operand(g, N, K, 128, 0.01)
    ref, mag = reference(a, sa, b, sb)
    out = kb.kda_matmul_fp8(a, sa, b, sb, out_dtype=dtype)
    assert kb.kda_get_device_error() == 0
    assert_near(out, ref, half_ulp(dtype), "out", atol=(K / 25 + 8) * 2.0 ** -23 * mag)
    return a, sa, b, sb, out


# one row to several tiles in each direction, one block of columns to many, ragged everywhere
SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 2048), (2, 300, 130), (15, 129, 127), (16, 128, 256),
         (17, 1000, 640), (32, 513, 4096), (33, 64, 20), (64, 640, 1500), (65, 128, 128),
         (100, 100, 100), (128, 128, 4096), (129, 257, 385), (300, 1001, 2200), (257, 4000, 512),
         (1037, 1001, 300), (2500, 2600, 400), (5000, 1100, 256), (700, 9000, 136), (3000, 16, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dtype):
    check(M, N, K, dtype)


# Sizes on both sides of where the cheapest cut into tiles changes: one wave of wide tiles or two
# of narrow ones, and k-blocks shared by 2, 4 or 8 blocks, all of which fit or do not.
CUTS = [(48, 1000, 4000), (65, 1024, 4096), (128, 1000, 4100), (128, 2050, 1920), (96, 6145, 520),
        (100, 12288, 640), (128, 12289, 384), (160, 1024, 4096), (250, 520, 8192), (384, 4096, 300),
        (1024, 4096, 1500), (513, 12288, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", CUTS)
def test_cuts_into_tiles(M, N, K, dtype):
    check(M, N, K, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(8, 256, 512), (40, 384, 300), (300, 500, 700)])
def test_strided_rows_and_outputs(M, N, K):
    a, sa, b, sb, want = check(M, N, K, torch.float32)
    wide_a = torch.zeros(M, 2048, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    wide_a[:, 32:32 + K].copy_(a)
    wide_s = torch.zeros(M, 64, device=DEV)
    wide_s[:, 5:5 + sa.shape[1]] = sa
    wide_o = torch.full((M, N + 21), 9.0, device=DEV)
    out = wide_o[:, 11:11 + N]
    kb.kda_matmul_fp8(wide_a[:, 32:32 + K], wide_s[:, 5:5 + sa.shape[1]], b, sb, out,
                      out_dtype=torch.float32)
    assert torch.equal(out, want)
    assert (wide_o[:, :11] == 9).all() and (wide_o[:, 11 + N:] == 9).all()
    # more leading dimensions
    if M % 4 == 0:
        three = kb.kda_matmul_fp8(wide_a[:, 32:32 + K].unflatten(0, (4, M // 4)),
                                  sa.unflatten(0, (4, M // 4)), b, sb, out_dtype=torch.float32)
        assert torch.equal(three.flatten(0, 1), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 200])
def test_nan_and_infinite_scales_stay_in_their_row(M):
    g = gen(3)
    a, sa = operand(g, M, 256, 1)
    b, sb = operand(g, 300, 256, 128)
    clean = kb.kda_matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)
    raw = a.view(torch.uint8).clone()
    raw[2, 100] = 0x7F                 # e4m3's NaN
    sa2 = sa.clone()
    sa2[4, 1] = float("nan")
    out = kb.kda_matmul_fp8(raw.view(torch.float8_e4m3fn), sa2, b, sb, out_dtype=torch.float32)
    assert out[2].isnan().all() and out[4].isnan().all()
    keep = [m for m in range(M) if m not in (2, 4)]
    assert torch.equal(out[keep], clean[keep])
    sb2 = sb.clone()
    sb2[1, 0] = float("nan")
    out = kb.kda_matmul_fp8(a, sa, b, sb2, out_dtype=torch.float32)
    assert out[:, 128:256].isnan().all() and torch.equal(out[:, :128], clean[:, :128])
    assert torch.equal(out[:, 256:], clean[:, 256:])


@pytest.mark.gpu
def test_same_call_same_bits_and_graph():
    a, sa, b, sb, want = check(20, 700, 3000, torch.bfloat16)
    for _ in range(3):
        assert torch.equal(kb.kda_matmul_fp8(a, sa, b, sb), want)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kb.kda_matmul_fp8(a, sa, b, sb, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_reads_what_the_norm_writes():
    """Rows normalised into 8 bits, times weights: the exact product of the rows within the
    8-bit rounding of the rows (2^-4 of a row's values at most)."""
    g = gen(8)
    x = torch.randn(70, 1000, device=DEV, generator=g).bfloat16()
    w = torch.ones(1000, device=DEV)
    b, sb = operand(g, 200, 1000, 128, 0.01)
    q, s, _ = kb.kda_add_rms_norm_quant(x, w)
    out = kb.kda_matmul_fp8(q, s, b, sb, out_dtype=torch.float32)
    ref, mag = reference(q, s, b, sb)
    assert_near(out, ref, 2.0 ** -24, "out", atol=48 * 2.0 ** -23 * mag)
    x64 = x.double()
    y = x64 / (x64.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    _, b_mag = reference(torch.ones(q.shape, device=DEV).to(q.dtype), torch.ones_like(s), b, sb)
    exact, _ = reference(q, s, b, sb)
    kb_ = torch.arange(1000, device=DEV) // 128
    b64 = b.double() * sb.double()[torch.arange(200, device=DEV) // 128][:, kb_]
    assert ((y @ b64.t() - exact).abs() <= y.abs() @ b64.abs().t() * 2.0 ** -3.9 + 1e-3 * b_mag).all()


# ---- refusals: on the host, before anything is launched
def P(i, off=0):
    return ctypes.c_void_p((1 << 40) + (i << 36) + off)


def call(M=100, N=256, K=256, dtype=0, **over):
    p = dict(a=P(0), ld_a=256, sa=P(1), ld_sa=2, b=P(2), ld_b=256, sb=P(3), ld_sb=2, out=P(4), ld_o=256)
    p.update(over)
    return kb.load().kda_matmul_fp8(p["a"], p["ld_a"], p["sa"], p["ld_sa"], p["b"], p["ld_b"], p["sb"],
                                    p["ld_sb"], p["out"], p["ld_o"], M, N, K, dtype, None)


@pytest.mark.parametrize("over,word", [
    (dict(M=-1), b"M=-1"), (dict(N=-1), b"N=-1"), (dict(K=0), b"K=0"), (dict(dtype=3), b"bf16 or f32"),
    (dict(a=None), b"a is NULL"), (dict(sa=None), b"a_scale is NULL"), (dict(b=None), b"b is NULL"),
    (dict(sb=None), b"b_scale is NULL"), (dict(out=None), b"out is NULL"),
    (dict(a=P(0, 8)), b"a: every row"), (dict(ld_a=264), b"a: every row"),
    (dict(b=P(2, 1)), b"b: every row"), (dict(ld_b=257), b"b: every row"),
    (dict(ld_a=240), b"leading dimension"), (dict(ld_sb=1), b"leading dimension"),
    (dict(ld_o=255), b"leading dimension"), (dict(out=P(4, 1)), b"out is not aligned"),
    (dict(sa=P(1, 2)), b"a_scale is not aligned"), (dict(out=P(2)), b"out overlaps b"),
    (dict(out=P(1, 64)), b"out overlaps a_scale"),
])
def test_refusals(over, word):
    assert call(**over) == 1
    assert word in kb.load().kda_last_error_message()


def test_nothing_to_do():
    assert call(M=0) == 0 and call(N=0) == 0


@pytest.mark.gpu
def test_binding_refusals():
    g = gen(1)
    a, sa = operand(g, 4, 256, 1)
    b, sb = operand(g, 128, 128, 128)
    with pytest.raises(kb.KdaError, match="columns"):
        kb.kda_matmul_fp8(a, sa, b, sb)
    with pytest.raises(kb.KdaError, match="a_scale"):
        kb.kda_matmul_fp8(a[:, :128], sa, b, sb)
    with pytest.raises(kb.KdaError, match="float8"):
        kb.kda_matmul_fp8(a[:, :128].float(), sa[:, :1], b, sb)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 130), (40, 129), (65, 300), (129, 257), (200, 1001), (1037, 100),
                                 (1037, 104), (2600, 2601), (2600, 2600)])
def test_nothing_is_written_past_the_last_row(M, N, dtype):
    """Every tile shape, with rows that a tensor copy may and may not write: the rows behind
    out's last one stay as they were."""
    g = gen(M + N)
    a, sa = operand(g, M, 256, 1)
    b, sb = operand(g, N, 256, 128)
    behind = torch.full((M + 256, N), 5.0, dtype=dtype, device=DEV)
    kb.kda_matmul_fp8(a, sa, b, sb, behind[:M])
    assert (behind[M:] == 5).all()
    assert torch.equal(behind[:M], kb.kda_matmul_fp8(a, sa, b, sb, out_dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [(5, 1, 1), (1, 5, 1), (1, 1, 1), (3, 0)])
def test_reads_what_the_norm_writes_with_dimensions_of_one(lead):
    g = gen(9)
    x = torch.randn(*lead, 2051, device=DEV, generator=g).bfloat16()
    b, sb = operand(g, 200, 2051, 128, 0.01)
    q, s, _ = kb.kda_add_rms_norm_quant(x, torch.ones(2051, device=DEV))
    out = kb.kda_matmul_fp8(q, s, b, sb, out_dtype=torch.float32)
    assert out.shape == (*lead, 200)
    q2, s2, _ = kb.kda_add_rms_norm_quant(x.view(-1, 2051), torch.ones(2051, device=DEV))
    assert torch.equal(out.view(-1, 200), kb.kda_matmul_fp8(q2, s2, b, sb, out_dtype=torch.float32))


def test_loaded_sums_are_used_together_with_what_the_wait_passes_on():
    """A load from tensor memory returns before its registers are written.  Their first use stands
    behind the wait because it also takes a scale that went through the wait; a statement that
    took nothing but the registers (a pairing, a move to another kind) could be moved before it,
    and no result would tell until a compiler does so.  So the source is looked at."""
    import os
    import re
    path = os.path.join(os.path.dirname(kb.__file__), "csrc", "kda_matmul_fp8.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    loads = re.findall(r'tcgen05\.ld\.sync.*?:\s*"r"\(taddr\)', text, re.S)
    assert loads and all('"=f"(r[0])' in x and '"=r"' not in x for x in loads)
    uses = re.findall(r"[^;{}\n]*\bd\[[^;]*;", text)
    assert uses
    for use in uses:
        use = " ".join(use.split())
        assert (re.fullmatch(r"float d\[G::kLoad\];", use)
                or re.fullmatch(r"(lo|hi) = fmaf\(d\[[^]]*\], s[01], \1\);", use)
                or re.fullmatch(r"add_scaled_pair\(lo, hi, d\[j\], d\[j \+ 1\], s0, s1\);", use)), use
    assert re.search(r"const float scale =\s*wait_ld\(", text)
    assert all(re.search(rf"const float {s} = SWAP \? __shfl_sync\(0xffffffffu, scale, .*: scale;", text)
               for s in ("s0", "s1"))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 300), (5, 1), (1, 1)])
def test_a_single_row_through_the_c_entry(M, N):
    """Its only row starts on a 16-byte boundary, whatever the distance to a next one."""
    K = 203
    a, sa, b, sb, want = check(M, N, K, torch.float32)
    out = torch.empty(M, N, device=DEV)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    torch.cuda.synchronize()
    st = kb.load().kda_matmul_fp8(ptr(a), K if M == 1 else a.stride(0), ptr(sa), 2, ptr(b),
                                  K if N == 1 else b.stride(0), ptr(sb), 2, ptr(out), N, M, N, K, 1, None)
    assert st == 0 and kb.kda_get_device_error() == 0
    assert torch.equal(out, want)
