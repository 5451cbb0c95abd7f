"""kda_ssm_scan_fwd and kda_ssm_scan_step against the recurrence in 64 bits, and their refusals.

Tolerances, against the recurrence run with magnitudes (m_t = a m_(t-1) + |dt x B|, the sum of
the magnitudes of all terms of h).  Relative to them one step rounds a (the exponent's product
and rate: 2 half ulps of |dt A| log2 e <= 20, the exponential 2 ulps), the product and sum; over
the steps a term survives (the a's fall as the exponents grow: sum of |dt A| over a term's life
is bounded where it still counts, below 20) errors stay under 2^-24 * (2 * 20 + 6 * life), life
<= 1 / (1 - a) capped at the length.  With the rates used here (dt A >= 0.001) life <= 1000:
2^-24 * 6040 = 3.6e-4 as a bound that no rounding can reach; the roundings are independent, so
the tests hold them to 1e-5 of the magnitudes, 16 times the root of that count.  y adds its own
half ulp, softplus and SiLU as in the convolution's tests (3e-6)."""
import ctypes

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, assert_near, gen, half_ulp, randn, sliced


def make(T, N, dim, S, G=1, dtype=torch.bfloat16, softplus=True, seed=0):
    g = gen(seed + T + dim + S)
    step = torch.exp(torch.rand(dim, device=DEV, generator=g) * 4.6 - 6.9)
    d = dict(x=randn(g, T, dim, dtype=dtype), z=randn(g, T, dim, dtype=dtype),
             B=randn(g, T, G, S, dtype=dtype), C=randn(g, T, G, S, dtype=dtype),
             A=-(torch.arange(1, S + 1, device=DEV).float() * (0.9 + 0.2 * torch.rand(dim, S, device=DEV, generator=g))),
             D=randn(g, dim), h0=randn(g, N, dim, S, std=0.3))
    if softplus:
        d["dt"] = randn(g, T, dim, std=0.5, dtype=dtype)
        d["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        d["dt"] = (step * (0.5 + torch.rand(T, dim, device=DEV, generator=g))).to(dtype)
        d["dt_bias"] = None
    return d


def reference(d, lens, softplus=True, gate=True, start=True, skip=True):
    """y, its magnitude, the final states and theirs."""
    N, (T, dim), (G, S) = len(lens), d["x"].shape, d["B"].shape[1:]
    x, dt = d["x"].double(), d["dt"].double()
    if d["dt_bias"] is not None:
        dt = dt + d["dt_bias"].double()
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    B = d["B"].double().repeat_interleave(dim // G, 1)
    C = d["C"].double().repeat_interleave(dim // G, 1)
    A = d["A"].double()
    h = d["h0"].double() if start else torch.zeros(N, dim, S, dtype=torch.float64, device=DEV)
    m = h.abs()
    y, my = torch.zeros_like(x), torch.zeros_like(x)
    firsts = torch.tensor([sum(lens[:n]) for n in range(N)], device=DEV)
    lens_t = torch.tensor(lens, device=DEV)
    for t in range(max(lens) if lens else 0):
        on = (lens_t > t).nonzero().flatten()
        r = firsts[on] + t
        a = torch.exp(dt[r][..., None] * A)
        b = (dt[r] * x[r])[..., None] * B[r]
        h[on] = a * h[on] + b
        m[on] = a * m[on] + b.abs()
        y[r] = (h[on] * C[r]).sum(-1)
        my[r] = (m[on] * C[r].abs()).sum(-1)
    if skip:
        y, my = y + d["D"].double() * x, my + (d["D"].double() * x).abs()
    if gate:
        s = d["z"].double() * torch.sigmoid(d["z"].double())
        y, my = y * s, my * s.abs()
    return y, my, h, m


def cu_of(lens):
    return torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def check(d, lens, dtype, *, packed=True, softplus=True, gate=True, start=True, skip=True, **over):
    args = {k: (sliced(v) if over.get("slices") and k in ("x", "dt", "z") else v) for k, v in d.items()}
    y_ref, my, h_ref, m = reference(d, lens, softplus, gate, start, skip)
    y, h = kb.kda_ssm_scan_fwd(args["x"], args["dt"], d["A"], d["B"], d["C"], d["D"] if skip else None,
                               args["z"] if gate else None, d["dt_bias"], d["h0"] if start else None,
                               cu_of(lens) if packed else None, n_seqs=len(lens), softplus=softplus)
    assert kb.kda_get_device_error() == 0
    assert_near(y, y_ref, half_ulp(dtype) + 3e-6, "y", atol=1e-5 * my)
    assert_near(h, h_ref, 0.0, "h", atol=1e-5 * m + 1e-30)
    return y, h


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,G", [(1, 1), (32, 1), (70, 2), (264, 8)])
def test_packed_sequences(dim, G, S, dtype):
    lens = [0, 1, 2, 0, 0, 5, 130, 4, 64, 1, 16, 33, 300, 0]
    check(make(sum(lens), len(lens), dim, S, G, dtype), lens, dtype, slices=dim == 70)


@pytest.mark.gpu
@pytest.mark.parametrize("softplus,gate,start,skip", [(True, False, False, False),
                                                      (False, True, True, False),
                                                      (False, False, True, True)])
def test_options(softplus, gate, start, skip):
    lens = [77, 0, 400]
    d = make(477, 3, 100, 16, 1, torch.bfloat16, softplus)
    check(d, lens, torch.bfloat16, softplus=softplus, gate=gate, start=start, skip=skip)


@pytest.mark.gpu
@pytest.mark.parametrize("N,length,dim,S", [(1, 1, 4096, 16), (1, 5000, 40, 16), (3, 1000, 96, 32),
                                            (64, 17, 512, 16), (700, 3, 33, 16), (2, 64, 64, 64),
                                            (1, 4099, 8, 128)])
def test_uniform_batches(N, length, dim, S):
    """One launch over whole sequences, and sequences cut into chunks (with their entry states
    chained over many chunks)."""
    check(make(N * length, N, dim, S), [length] * N, torch.bfloat16, packed=False)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[6000], [3000, 1, 2999], [1] * 200 + [5000] + [2] * 100,
                                  [64] * 60, [1024, 0, 0, 1024, 2048]])
def test_long_packed_sequences(lens):
    check(make(sum(lens), len(lens), 48, 16, dtype=torch.float32), lens, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[3000, 10, 0, 500], [40, 40]])
def test_state_in_place(lens):
    d = make(sum(lens), len(lens), 64, 16)
    cu = cu_of(lens)
    call = lambda h0, **k: kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"],
                                               d["dt_bias"], h0, cu, **k)
    y, h = call(d["h0"])
    state = d["h0"].clone()
    y2, same = call(state, h_final=state)
    assert same is state and torch.equal(y2, y) and torch.equal(state, h)
    y3, none = call(d["h0"], want_state=False)
    assert none is None and torch.equal(y3, y)


@pytest.mark.gpu
def test_runs_of_the_same_call_agree_bit_for_bit():
    lens = [2500, 700, 1]
    d = make(sum(lens), 3, 200, 16)
    call = lambda: kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"],
                                       d["dt_bias"], d["h0"], cu_of(lens))
    first = call()
    for _ in range(3):
        again = call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,dim,S,G", [(1, 1, 16, 1), (3, 4096, 16, 1), (40, 66, 32, 2),
                                       (7, 100, 64, 4), (5, 33, 128, 1)])
def test_steps_match_64_bits(N, dim, S, G, dtype):
    """Six steps, one after another, against the recurrence of the same tokens."""
    d = make(6 * N, N, dim, S, G, dtype)
    per = {k: d[k].unflatten(0, (N, 6)) for k in ("x", "dt", "z", "B", "C")}
    y_ref, my, h_ref, m = reference(d, [6] * N)
    h = d["h0"].clone()
    for t in range(6):
        y = kb.kda_ssm_scan_step(per["x"][:, t], per["dt"][:, t], d["A"], per["B"][:, t],
                                 per["C"][:, t], h, d["D"], per["z"][:, t], d["dt_bias"])
        assert_near(y, y_ref.unflatten(0, (N, 6))[:, t], half_ulp(dtype) + 3e-6, "y",
                    atol=1e-5 * my.unflatten(0, (N, 6))[:, t])
    assert_near(h, h_ref, 0.0, "h", atol=1e-5 * m)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_step_without_gate_bias_or_softplus():
    d = make(9, 9, 50, 16, softplus=False, dtype=torch.float32)
    y_ref, my, h_ref, m = reference(d, [1] * 9, softplus=False, gate=False, skip=False)
    h = d["h0"].clone()
    y = kb.kda_ssm_scan_step(sliced(d["x"]), d["dt"], d["A"], d["B"], d["C"], h, softplus=False)
    assert_near(y, y_ref, 4e-6, "y", atol=1e-5 * my)
    assert_near(h, h_ref, 0.0, "h", atol=1e-5 * m)


@pytest.mark.gpu
def test_extreme_step_sizes():
    """A step size of 0 leaves the state, a huge one forgets it; a NaN stays in its channel and
    sequence."""
    lens = [100, 100]
    d = make(200, 2, 32, 16, dtype=torch.float32, softplus=False)
    d["dt"][40:50] = 0.0
    d["dt"][60, 5] = 1e6
    d["x"][60, 5] = 0.0
    d["x"][70, 9] = float("nan")
    y, h = kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], None, None, None, d["h0"],
                               cu_of(lens), softplus=False)
    assert y[60, 5] == 0.0
    bad = y.isnan()
    assert bad[70:100, 9].all() and bad.sum() == 30
    assert h[0, 9].isnan().all() and h.isnan().sum() == 16
    # softplus far out on both sides: the step itself, and none
    d["dt"][:100], d["dt"][100:] = 100.0, -200.0
    d["A"].fill_(-1e-4)
    d["x"] = torch.ones_like(d["x"])
    y, h = kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], None, None, None, d["h0"],
                               cu_of(lens))
    assert h[0].isfinite().all() and torch.equal(h[1], d["h0"][1])


@pytest.mark.gpu
def test_no_tokens_hand_the_state_through():
    d = make(1, 3, 40, 16)
    none = {k: d[k][:0] for k in ("x", "dt", "z", "B", "C")}
    for cu in (cu_of([0, 0, 0]), None):
        y, h = kb.kda_ssm_scan_fwd(none["x"], none["dt"], d["A"], none["B"], none["C"], h0=d["h0"],
                                   cu_seqlens=cu, n_seqs=3)
        assert y.shape == (0, 40) and torch.equal(h, d["h0"])


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 500, 200, 1000], [5, 500, 600, 1000], [0, 500, 600, 900],
                                [0, 500, 600, 10000], [0, -7, 600, 1000], [900, 800, 700, 600]])
def test_malformed_cu_seqlens_is_reported(cu):
    d = make(1000, 3, 40, 16)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], None, d["dt_bias"], d["h0"], cu)
    assert kb.kda_get_device_error() == 5
    assert b"cu_seqlens" in kb.load().kda_last_error_message()
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_captured_in_a_graph_and_on_another_stream():
    lens = [2000, 31]
    d = make(sum(lens), 2, 64, 16)
    cu = cu_of(lens)
    call = lambda **k: kb.kda_ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"],
                                           d["dt_bias"], d["h0"], cu, **k)
    want, h_want = call()
    y, h = torch.empty_like(want), torch.empty_like(h_want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y=y, h_final=h)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, h_want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, h2 = call(stream=side)
    side.synchronize()
    assert torch.equal(y2, want) and torch.equal(h2, h_want)


# ---- refusals: on the host, before anything is launched
def P(i, off=0):
    return ctypes.c_void_p((1 << 40) + (i << 32) + off)


def call(T=128, N=2, dim=64, state=16, groups=1, dtype=0, **over):
    p = dict(x=P(0), ld_x=dim, dt=P(1), A=P(2), B=P(3), ld_b=groups * state, C=P(4), D=P(5), z=P(6),
             bias=P(7), h0=P(8), cu=None, y=P(9), ld_y=dim, h=P(10))
    p.update(over)
    return kb.load().kda_ssm_scan_fwd(p["x"], p["ld_x"], p["dt"], dim, p["A"], p["B"], p["ld_b"], p["C"],
                                      groups * state, p["D"], p["z"], dim, p["bias"], p["h0"], p["cu"],
                                      p["y"], p["ld_y"], p["h"], T, N, dim, state, groups, 1, dtype, None)


@pytest.mark.parametrize("status,over,word", [
    (1, dict(T=-1), b"total_tokens"), (1, dict(N=-1), b"n_seqs"), (1, dict(dim=0), b"dim"),
    (1, dict(groups=0), b"groups"), (1, dict(groups=3), b"multiple of groups"),
    (2, dict(state=24), b"state=24"), (1, dict(dtype=3), b"bf16 or f32"),
    (1, dict(T=127), b"multiple"), (1, dict(N=0), b"n_seqs = 0"), (1, dict(x=None), b"x is NULL"),
    (1, dict(dt=None), b"dt is NULL"), (1, dict(A=None), b"A is NULL"), (1, dict(y=None), b"y is NULL"),
    (1, dict(x=P(0, 1)), b"aligned"), (1, dict(A=P(2, 2)), b"A is not aligned"),
    (1, dict(h0=P(8, 4)), b"h0 is not 16-byte aligned"), (1, dict(h=P(10, 8)), b"16-byte aligned"),
    (1, dict(ld_x=63), b"leading dimension"), (1, dict(ld_b=15), b"leading dimension"),
    (1, dict(y=P(0)), b"y overlaps x"), (1, dict(y=P(6, 64)), b"y overlaps z"),
    (1, dict(h=P(8, 64)), b"h_final overlaps h0"), (1, dict(h=P(2)), b"h_final overlaps A"),
    (1, dict(y=P(10)), b"y overlaps h_final"), (2, dict(T=1 << 31), b"total_tokens"),
])
def test_refusals(status, over, word):
    assert call(**over) == status
    assert word in kb.load().kda_last_error_message()


def test_nothing_to_do():
    assert call(T=0, N=0) == 0
    lib = kb.load()
    step = lambda h, N: lib.kda_ssm_scan_step(P(0), 64, P(1), 64, P(2), P(3), 16, P(4), 16, None, None, 0,
                                              None, h, P(9), 64, N, 64, 16, 1, 1, 0, None)
    assert step(None, 2) == 1 and b"h is NULL" in lib.kda_last_error_message()
    assert step(P(8), 0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G", [2, 8])
def test_one_token_of_several_groups(G, dtype):
    """One sequence's one token, whose groups are all of B and C: as a step, as a packed prompt
    and as a uniform batch; and no token at all."""
    d = make(1, 1, 48, 16, G, dtype)
    y_ref, my, h_ref, m = reference(d, [1])
    check(d, [1], dtype)
    check(d, [1], dtype, packed=False)
    one = {k: d[k][None] for k in ("x", "dt", "z", "B", "C")}
    y, h = kb.kda_ssm_scan_fwd(one["x"], one["dt"], d["A"], one["B"], one["C"], d["D"], one["z"],
                               d["dt_bias"], d["h0"])
    assert_near(y[0], y_ref, half_ulp(dtype) + 3e-6, "y", atol=1e-5 * my)
    assert_near(h, h_ref, 0.0, "h", atol=1e-5 * m)
    h = d["h0"].clone()
    y = kb.kda_ssm_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], h, d["D"], d["z"], d["dt_bias"])
    assert_near(y, y_ref, half_ulp(dtype) + 3e-6, "y", atol=1e-5 * my)
    assert_near(h, h_ref, 0.0, "h", atol=1e-5 * m)
    none = {k: d[k][:0] for k in ("x", "dt", "z", "B", "C")}
    y, h = kb.kda_ssm_scan_fwd(none["x"], none["dt"], d["A"], none["B"], none["C"], h0=d["h0"],
                               cu_seqlens=cu_of([0]))
    assert y.shape == (0, 48) and torch.equal(h, d["h0"])
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 4])
def test_a_uniform_batch_without_tokens_hands_the_state_through(G):
    d = make(3, 3, 40, 16, G)
    none = {k: d[k].unflatten(0, (3, 1))[:, :0] for k in ("x", "dt", "z", "B", "C")}
    y, h = kb.kda_ssm_scan_fwd(none["x"], none["dt"], d["A"], none["B"], none["C"], d["D"], none["z"],
                               d["dt_bias"], d["h0"])
    assert y.shape == (3, 0, 40) and torch.equal(h, d["h0"])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [33, 64])
def test_gate_far_out(dim):
    """y is the gate's SiLU alone (no readout, D x = 1); its tolerance as in the convolution's test
    of the same."""
    z = torch.linspace(-110, 110, 300 * dim, device=DEV).view(300, dim)
    d = make(300, 1, dim, 16, dtype=torch.float32)
    one, none = torch.ones(300, dim, device=DEV), torch.zeros_like(d["C"])
    ref = z.double() * torch.sigmoid(z.double())
    atol = 1.25 * z.double().abs() * 2.0 ** -24 * ref.abs()
    atol = torch.where(z < -87.3, torch.maximum(atol, ref.abs()), atol)
    y, _ = kb.kda_ssm_scan_fwd(one, d["dt"], d["A"], d["B"], none, one[0], z, d["dt_bias"])
    assert_near(y, ref, 8 * 2.0 ** -24, "y", atol=atol)
    h = torch.zeros(300, dim, 16, device=DEV)
    y = kb.kda_ssm_scan_step(one, d["dt"], d["A"], d["B"], none, h, one[0], z, d["dt_bias"])
    assert_near(y, ref, 8 * 2.0 ** -24, "y", atol=atol)


@pytest.mark.gpu
def test_no_tokens_need_no_inputs():
    """T = 0 through the C entry with every input NULL, as the other inputs may be: the states are
    handed through, or zeros."""
    N, dim, S = 3, 40, 16
    h0 = torch.randn(N, dim, S, device=DEV)
    for given, want in ((h0, h0), (None, torch.zeros_like(h0))):
        h = torch.full_like(h0, 7.0)
        torch.cuda.synchronize()
        st = kb.load().kda_ssm_scan_fwd(None, dim, None, dim, None, None, S, None, S, None, None, dim, None,
                                        None if given is None else ctypes.c_void_p(given.data_ptr()), None,
                                        None, dim, ctypes.c_void_p(h.data_ptr()), 0, N, dim, S, 1, 1, 0, None)
        assert st == 0 and kb.kda_get_device_error() == 0
        assert torch.equal(h, want)
