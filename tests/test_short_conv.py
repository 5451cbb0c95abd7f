"""kda_short_conv_fwd and kda_short_conv_step against 64 bits, and their refusals.

Tolerances.  A sum of at most 9 terms in 32 bits: within 9 half ulps of the sum of their
magnitudes (SiLU's slope is at most 1.1); SiLU itself: an exponential within 2 + 1.2 |v| ulps,
a quotient within 2, so at |v| <= 16 under 24 ulps = 3e-6 relative; then the output's own half
ulp.  States are copies: bit for bit."""
import ctypes

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, assert_near, gen, half_ulp, randn, sliced


def reference(x, w, bias, state, lens, silu):
    x64, w64, width = x.double(), w.double(), w.shape[1]
    y, mag = torch.empty_like(x64), torch.empty_like(x64)
    out = torch.zeros(len(lens), width - 1, x.shape[1], dtype=x.dtype, device=x.device)
    at = 0
    for n, length in enumerate(lens):
        before = out[n] if state is None else state[n]
        rows = torch.cat([before, x[at:at + length]])
        r64 = rows.double()
        v = torch.zeros(length, x.shape[1], dtype=torch.float64, device=x.device)
        m = torch.zeros_like(v)
        for j in range(width):
            v += r64[j:j + length] * w64[:, j]
            m += (r64[j:j + length] * w64[:, j]).abs()
        if bias is not None:
            v, m = v + bias.double(), m + bias.double().abs()
        y[at:at + length] = v * torch.sigmoid(v) if silu else v
        mag[at:at + length] = m
        out[n] = rows[length:]
        at += length
    return y, mag, out


def inputs(lens, dim, width, dtype, w_dtype=None, seed=0):
    g = gen(seed + dim + width)
    total = sum(lens)
    return (randn(g, total, dim, dtype=dtype), randn(g, dim, width, std=0.5, dtype=w_dtype or dtype),
            randn(g, dim, std=0.1, dtype=w_dtype or dtype),
            randn(g, len(lens), width - 1, dim, dtype=dtype))


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def near(y, ref, mag, dtype):
    assert_near(y, ref, half_ulp(dtype) + 3e-6, "y", atol=6e-7 * mag)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dim", [1, 24, 130, 1032])
def test_packed_sequences(dim, width, dtype):
    # empty ones first, in the middle, last; shorter than the state; across strips
    lens = [0, 1, 2, 0, 0, 7, 130, 3, 64, 1, 1, 300, 0]
    x, w, b, s = inputs(lens, dim, width, dtype)
    for bias, state, silu in ((b, s, True), (None, None, False)):
        y_ref, mag, s_ref = reference(x, w, bias, state, lens, silu)
        y, out = kb.kda_short_conv_fwd(x, w, bias, state, cu_of(lens), silu=silu)
        near(y, y_ref, mag, dtype)
        assert torch.equal(out, s_ref)
    # a column slice of a wider tensor gives the same bits
    y2, out2 = kb.kda_short_conv_fwd(sliced(x), w, None, None, cu_of(lens), silu=False)
    assert torch.equal(y2, y) and torch.equal(out2, out)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,length,dim", [(1, 1, 4096), (4, 500, 640), (200, 1, 64), (3, 2, 33),
                                          (2, 9000, 264)])
def test_uniform_batches_and_mixed_types(N, length, dim):
    x, w, b, s = inputs([length] * N, dim, 4, torch.bfloat16, torch.float32, seed=N)
    y_ref, mag, s_ref = reference(x, w, b, s, [length] * N, True)
    y, out = kb.kda_short_conv_fwd(x.view(N, length, dim), w, b, s)
    near(y.view(-1, dim), y_ref, mag, torch.bfloat16)
    assert torch.equal(out, s_ref)
    y2, none = kb.kda_short_conv_fwd(x, w, b, s, n_seqs=N, want_state=False)
    assert none is None and torch.equal(y2, y.view(-1, dim))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_state_in_place_continues(dtype):
    lens, dim = [300, 2, 0, 77], 520
    x, w, b, s = inputs(lens, dim, 4, dtype, seed=5)
    y, out = kb.kda_short_conv_fwd(x, w, b, s, cu_of(lens))
    state = s.clone()
    y2, same = kb.kda_short_conv_fwd(x, w, b, state, cu_of(lens), state_out=state)
    assert same is state and torch.equal(state, out) and torch.equal(y2, y)
    # in two halves: the second call starts from the first one's state, bit for bit
    full, _ = kb.kda_short_conv_fwd(x[:300], w, b, s[:1].contiguous(), n_seqs=1)
    part, st = kb.kda_short_conv_fwd(x[:113], w, b, s[:1].contiguous(), n_seqs=1)
    rest, st2 = kb.kda_short_conv_fwd(x[113:300], w, b, st, n_seqs=1)
    assert torch.equal(torch.cat([part, rest]), full) and torch.equal(st2, out[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,dim,width", [(1, 1, 2), (3, 4096, 4), (300, 72, 4), (17, 333, 8),
                                         (5, 1032, 3)])
def test_steps_equal_the_prompt(N, dim, width, dtype):
    x, w, b, s = inputs([5] * N, dim, width, dtype, seed=9)
    want, s_want = kb.kda_short_conv_fwd(x.view(N, 5, dim), w, b, s)
    state = s.clone()
    for t in range(5):
        y = kb.kda_short_conv_step(x.view(N, 5, dim)[:, t], w, state, b)
        assert torch.equal(y, want[:, t])
    assert torch.equal(state, s_want)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_infinities_stay_in_their_window():
    """A row that holds inf or NaN touches the width outputs that read it, in its sequence."""
    lens, dim = [40, 40], 16
    x, w, _, _ = inputs(lens, dim, 3, torch.float32)
    x[20, 3], x[38, 5] = float("nan"), float("inf")
    y, _ = kb.kda_short_conv_fwd(x, w, None, None, cu_of(lens), silu=False)
    bad = ~y.isfinite()
    want = torch.zeros_like(bad)
    want[20:23, 3] = True
    want[38:40, 5] = True
    assert torch.equal(bad, want)


@pytest.mark.gpu
def test_no_tokens_hand_the_state_through():
    _, w, b, s = inputs([1] * 3, 40, 4, torch.bfloat16)
    y, out = kb.kda_short_conv_fwd(torch.empty(0, 40, dtype=torch.bfloat16, device=DEV), w, b, s,
                                   cu_of([0, 0, 0]))
    assert y.shape == (0, 40) and torch.equal(out, s)
    y, out = kb.kda_short_conv_fwd(torch.empty(0, 40, dtype=torch.bfloat16, device=DEV), w, b, None,
                                   n_seqs=2)
    assert (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 50, 20, 100], [5, 50, 60, 100], [0, 50, 60, 90],
                                [0, 50, 60, 1000], [0, -7, 60, 100], [90, 80, 70, 60]])
def test_malformed_cu_seqlens_is_reported(cu):
    x, w, b, s = inputs([100], 40, 4, torch.bfloat16)
    s3 = s.expand(3, 3, 40).contiguous()
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    kb.kda_short_conv_fwd(x, w, b, s3, cu)
    assert kb.kda_get_device_error() == 5
    assert b"cu_seqlens" in kb.load().kda_last_error_message()
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_captured_in_a_graph():
    lens = [100, 31]
    x, w, b, s = inputs(lens, 64, 4, torch.bfloat16)
    cu = cu_of(lens)
    want, s_want = kb.kda_short_conv_fwd(x, w, b, s, cu)
    y, out = torch.empty_like(want), torch.empty_like(s_want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kb.kda_short_conv_fwd(x, w, b, s, cu, y=y, state_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(out, s_want)


# ---- refusals: on the host, before anything is launched
def P(i, off=0):
    return ctypes.c_void_p((1 << 40) + (i << 32) + off)


def call(T=128, N=2, dim=64, width=4, dtype=0, w_dtype=0, **over):
    p = dict(x=P(0), ld_x=dim, w=P(1), b=P(2), s_in=P(3), s_out=P(4), cu=None, y=P(5), ld_y=dim)
    p.update(over)
    return kb.load().kda_short_conv_fwd(p["x"], p["ld_x"], p["w"], p["b"], p["s_in"], p["s_out"],
                                        p["cu"], p["y"], p["ld_y"], T, N, dim, width, 1, dtype,
                                        w_dtype, None)


@pytest.mark.parametrize("status,over,word", [
    (1, dict(T=-1), b"total_tokens"), (1, dict(N=-1), b"n_seqs"), (1, dict(dim=0), b"dim"),
    (2, dict(width=1), b"width"), (2, dict(width=9), b"width"), (1, dict(width=0), b"width"),
    (1, dict(dtype=3), b"bf16 or f32"), (1, dict(w_dtype=2), b"bf16 or f32"),
    (1, dict(T=127), b"multiple"), (1, dict(N=0), b"n_seqs = 0"), (1, dict(x=None), b"x is NULL"),
    (1, dict(w=None), b"weight is NULL"), (1, dict(y=None), b"y is NULL"),
    (1, dict(x=P(0, 1)), b"aligned"), (1, dict(cu=P(6, 2)), b"cu_seqlens is not aligned"),
    (1, dict(ld_x=63), b"leading dimension"), (1, dict(ld_y=1), b"leading dimension"),
    (1, dict(y=P(0)), b"y overlaps x"), (1, dict(s_out=P(3, 64)), b"state_out overlaps state_in"),
    (1, dict(s_out=P(0)), b"state_out overlaps x"), (1, dict(y=P(4)), b"y overlaps state_out"),
    (2, dict(T=1 << 31), b"total_tokens"),
])
def test_refusals(status, over, word):
    assert call(**over) == status
    assert word in kb.load().kda_last_error_message()


def test_nothing_to_do_and_interleaved_slices():
    assert call(T=0, N=0) == 0
    lib = kb.load()
    # x and y as column slices of one buffer do not overlap, but must not share columns
    assert call(ld_x=128, ld_y=128, y=P(0, 2 * 32)) == 1
    assert b"y overlaps x" in lib.kda_last_error_message()
    assert lib.kda_short_conv_step(P(0), 64, P(1), None, None, P(2), 64, 2, 64, 4, 1, 0, 0, None) == 1
    assert b"state is NULL" in lib.kda_last_error_message()
    assert lib.kda_short_conv_step(P(0), 64, P(1), None, P(3), P(2), 64, 0, 64, 4, 1, 0, 0, None) == 0


@pytest.mark.gpu
def test_output_beside_its_input():
    """x and y may be column slices of one buffer."""
    x, w, b, s = inputs([50, 3], 64, 4, torch.bfloat16)
    want, _ = kb.kda_short_conv_fwd(x, w, b, s, cu_of([50, 3]))
    wide = torch.zeros(53, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, :64] = x
    kb.kda_short_conv_fwd(wide[:, :64], w, b, s, cu_of([50, 3]), y=wide[:, 64:])
    assert torch.equal(wide[:, 64:], want) and torch.equal(wide[:, :64], x)


@pytest.mark.gpu
def test_a_uniform_batch_without_tokens_hands_the_state_through():
    _, w, b, s = inputs([1] * 3, 40, 4, torch.bfloat16)
    y, out = kb.kda_short_conv_fwd(torch.empty(3, 0, 40, dtype=torch.bfloat16, device=DEV), w, b, s)
    assert y.shape == (3, 0, 40) and torch.equal(out, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [1, 2, 4])
def test_silu_far_out(dim):
    """Large pre-activations of both signs.  In half ulps: the exponent's rounding and its
    constant's move the exponential by 1.25 |v|; the exponential's own error (2^-22.5 = 2.8), the
    reciprocal's (2^-23 = 2) and the sum's and product's roundings are under 8.  Where the sigmoid
    is below 2^-126 (v < -87.3) the result may be 0."""
    v = torch.cat([torch.linspace(-110, 110, 20001), torch.tensor([-1e-30, 1e-30, -1e-38, 1e30, 3e38, -3e38]),
                   torch.zeros(1)]).to(DEV)
    v = v[:v.numel() // dim * dim]
    x = v.view(-1, dim).contiguous()
    w = torch.tensor([0.0, 1.0], device=DEV).repeat(dim, 1)
    ref = v.double() * torch.sigmoid(v.double())
    atol = 1.25 * v.double().abs().clamp(max=120) * 2.0 ** -24 * ref.abs()
    atol = torch.where(v < -87.3, torch.maximum(atol, ref.abs()), atol)
    for y in (kb.kda_short_conv_fwd(x, w)[0],
              kb.kda_short_conv_step(x, w, torch.zeros(x.shape[0], 1, dim, device=DEV))):
        assert_near(y.flatten(), ref, 8 * 2.0 ** -24, "y", atol=atol)
        assert ((y.flatten() - ref).abs()[v < -87.3] <= 88 * 2.0 ** -126).all()
