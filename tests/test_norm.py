"""kda_add_rms_norm against 64 bits, and its refusals.

Tolerances.  The kernel makes these 32-bit roundings on the way to a y: the
sum h (1/2 ulp, which moves the mean by at most twice that), a sum of dim
squares (each lane adds at most 8 * 8 terms, then log2 steps; errors of
positive terms: at most 64 + 10 half ulps), a division, a root, a quotient and
two products: under 100 half ulps = 6e-6 relative, plus the output's own half
ulp.  A scale is one quotient more.  An 8-bit value may sit one e4m3 step off
where the unrounded value lies within 1e-5 of the middle between two."""
import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, assert_near, gen, half_ulp, randn, sliced

PATH32 = 6e-6


def reference(x, w, r, eps):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    return h, y


def groups_of(y):
    dim = y.shape[-1]
    g = torch.nn.functional.pad(y, (0, -dim % 128))
    return g.view(*y.shape[:-1], -1, 128)


def check_quant(q, scale, y):
    """q and scale against the exact rows y (64 bits)."""
    want = groups_of(y).abs().amax(-1).clamp(min=2.0 ** -64) / 448
    assert_near(scale, want, 1e-5, "scale")
    unit = groups_of(y) / want[..., None]
    got = groups_of(q.double())
    # half a step of e4m3 at that magnitude (2^-4 relative, 2^-10 below 2^-6), and 1e-5 more
    err = (got - unit).abs()
    bound = unit.abs().clamp(min=2.0 ** -6) * 2.0 ** -4 * (1 + 1e-3)
    assert (err <= bound).all(), (err - bound).max()
    # correctly rounded but for values near the middle of two steps
    near = unit.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    assert (got != near).double().mean() < 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 4096), (3, 7), (5, 128), (4, 256), (401, 264),
                                      (2, 300), (700, 1000), (7, 2051), (3, 8192), (2, 16392),
                                      (400, 32776), (2, 65536), (310, 65535)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_matches_64_bits(rows, dim, dtype, with_residual):
    g = gen(rows * 7 + dim)
    x = randn(g, rows, dim, dtype=dtype)
    r = randn(g, rows, dim, std=3.0, dtype=dtype) if with_residual else None
    w = randn(g, dim, dtype=dtype)
    h_ref, y_ref = reference(x, w, r, 1e-6)
    y, h = kb.kda_add_rms_norm(x, w, r, eps=1e-6)
    assert_near(y, y_ref, half_ulp(dtype) + PATH32, "y")
    assert (h is None) == (r is None)
    if h is not None:
        assert_near(h, h_ref, half_ulp(dtype) + 2.0 ** -23, "h", atol=1e-6)
    q, s, h2 = kb.kda_add_rms_norm_quant(x, w, r, eps=1e-6)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape
    check_quant(q, s, y_ref)
    assert h is None or torch.equal(h, h2)
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,w_dtype", [(torch.bfloat16, torch.float32),
                                           (torch.float32, torch.bfloat16)])
def test_norm_of_strided_rows_and_mixed_types(dtype, w_dtype):
    g = gen(1)
    x, r = randn(g, 33, 515, dtype=dtype), randn(g, 33, 515, dtype=dtype)
    w = randn(g, 515, dtype=w_dtype)
    _, y_ref = reference(x, w, r, 1e-5)
    y, h = kb.kda_add_rms_norm(sliced(x), w, sliced(r), eps=1e-5)
    assert_near(y, y_ref, half_ulp(dtype) + PATH32, "y")
    # outputs into slices, and their neighbours untouched
    wide = torch.full((33, 600), 7.0, dtype=dtype, device=DEV)
    out = wide[:, 40:555]
    kb.kda_add_rms_norm(x, w, r, eps=1e-5, y=out, h=h)
    assert torch.equal(out, y)
    assert (wide[:, :40] == 7).all() and (wide[:, 555:] == 7).all()
    # more leading dimensions
    y3, _ = kb.kda_add_rms_norm(x.view(3, 11, 515), w, r.view(3, 11, 515), eps=1e-5)
    assert torch.equal(y3.view(33, 515), y)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(3, 4096), (500, 1000), (9, 77)])
def test_norm_in_place(rows, dim):
    g = gen(2)
    x, r = (randn(g, rows, dim, dtype=torch.bfloat16) for _ in range(2))
    w = randn(g, dim, dtype=torch.bfloat16)
    y, h = kb.kda_add_rms_norm(x, w, r)
    x2, r2 = x.clone(), r.clone()
    y2, h2 = kb.kda_add_rms_norm(x2, w, r2, y=x2, h=r2)
    assert y2 is x2 and h2 is r2 and torch.equal(x2, y) and torch.equal(r2, h)


@pytest.mark.gpu
def test_norm_of_extreme_rows():
    x = torch.zeros(6, 300, device=DEV)
    x[1, 5] = 1.0                       # two groups of zeros
    x[2] = 1e-30                        # far below eps
    x[3, 4] = float("nan")
    x[4, 200] = float("inf")
    x[5] = 2.0 ** 55                    # squares near the top of 32 bits
    w = torch.ones(300, device=DEV)
    y, _ = kb.kda_add_rms_norm(x, w, eps=1e-6)
    q, s, _ = kb.kda_add_rms_norm_quant(x, w, eps=1e-6)
    assert (y[0] == 0).all() and (q[0].float() == 0).all()
    assert torch.equal(s[0], torch.full((3,), 2.0 ** -64 / 448, device=DEV))
    assert q[1].float()[5] == 448 and (s[1, 1:] == 2.0 ** -64 / 448).all()
    assert_near(y[2], torch.full((300,), 1e-27, device=DEV, dtype=torch.float64), 1e-5, "tiny")
    assert y[3].isnan().all() and q[3].float().isnan().all() and s[3].isnan().all()
    # the root of an infinite mean is infinite: zeros, and NaN where inf / inf stands
    assert y[4].isnan().sum() == 1 and y[4, 200].isnan() and (y[4, :200] == 0).all()
    assert q[4].float()[128:256].isnan().all() and (q[4].float()[:128] == 0).all()
    assert_near(y[5], torch.ones(300, device=DEV, dtype=torch.float64), 1e-5, "large")
    assert kb.kda_get_device_error() == 0


@pytest.mark.gpu
def test_norm_without_rows_and_on_another_stream():
    w = torch.ones(64, device=DEV)
    y, h = kb.kda_add_rms_norm(torch.empty(0, 64, device=DEV), w, torch.empty(0, 64, device=DEV))
    assert y.shape == (0, 64) and h.shape == (0, 64)
    x = randn(gen(4), 2000, 64)
    want, _ = kb.kda_add_rms_norm(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = kb.kda_add_rms_norm(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


# ---- refusals: on the host, before anything is launched
import ctypes  # noqa: E402

BASE = 1 << 40


def P(i, off=0):
    return ctypes.c_void_p(BASE + (i << 32) + off)


def call(rows=4, dim=256, eps=1e-6, dtype=0, w_dtype=0, y_dtype=0, ld=256, **over):
    p = dict(x=P(0), residual=P(1), weight=P(2), h=P(3), y=P(4), scale=None, ld_y=ld, ld_s=2)
    p.update(over)
    return kb.load().kda_add_rms_norm(p["x"], ld, p["residual"], ld, p["weight"], p["h"], ld,
                                      p["y"], p["ld_y"], p["scale"], p["ld_s"], rows, dim, eps,
                                      dtype, w_dtype, y_dtype, None)


@pytest.mark.parametrize("over,word", [
    (dict(rows=-1), b"rows"), (dict(dim=0), b"dim"), (dict(eps=-1.0), b"eps"),
    (dict(eps=float("nan")), b"eps"), (dict(dtype=2), b"bf16 or f32"),
    (dict(w_dtype=3), b"bf16 or f32"), (dict(y_dtype=1), b"x's dtype"),
    (dict(x=None), b"x is NULL"), (dict(weight=None), b"weight is NULL"),
    (dict(y=None), b"y is NULL"), (dict(h=None), b"h is NULL"),
    (dict(y_dtype=3), b"y_scale is NULL"), (dict(scale=P(5)), b"y_scale is given"),
    (dict(x=P(0, 1)), b"x is not aligned"), (dict(ld=255), b"leading dimension"),
    (dict(y_dtype=3, scale=P(5), ld_s=1), b"leading dimension"),
    (dict(y_dtype=3, scale=P(5, 2)), b"y_scale is not aligned"),
    (dict(y=P(3)), b"y overlaps h"), (dict(h=P(0, 64)), b"h overlaps x"),
    (dict(y=P(2)), b"y overlaps weight"), (dict(y_dtype=3, scale=P(5), y=P(0)), b"y overlaps x"),
    (dict(y_dtype=3, scale=P(3)), b"y_scale overlaps h"),
])
def test_norm_refuses(over, word):
    assert call(**over) == 1
    assert word in kb.load().kda_last_error_message()


def test_norm_unsupported_and_empty():
    assert call(dim=65537, ld=65537) == 2
    assert call(rows=1 << 31) == 2
    assert call(rows=0) == 0


def test_norm_binding_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(kb.KdaError, match="CUDA"):
        kb.kda_add_rms_norm(x, torch.zeros(8))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3, 0, 64), (0, 3, 64), (2, 0, 5, 77)])
def test_norm_of_a_batch_without_rows(shape):
    x, w = torch.empty(*shape, device=DEV), torch.ones(shape[-1], device=DEV)
    y, h = kb.kda_add_rms_norm(x, w, x.clone())
    assert y.shape == x.shape and h.shape == x.shape
    q, s, _ = kb.kda_add_rms_norm_quant(x, w)
    assert q.shape == x.shape and s.shape == (*shape[:-1], 1)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(5, 1, 1, 2051), (1, 5, 1, 2051), (1, 1, 1, 2051), (5, 1, 1, 1, 40)])
def test_norm_of_rows_with_dimensions_of_one(shape):
    """Dimensions of one between the rows and their columns, in rows that stand further apart
    than they are long: what the 8-bit form allocates itself, and slices."""
    g = gen(11)
    x = randn(g, *shape, dtype=torch.bfloat16)
    w = randn(g, shape[-1], dtype=torch.bfloat16)
    rows = x.view(-1, shape[-1])
    want, want_s, _ = kb.kda_add_rms_norm_quant(rows, w)
    for given in (x, sliced(x)):
        q, s, _ = kb.kda_add_rms_norm_quant(given, w)
        assert q.shape == x.shape
        assert torch.equal(q.float().view_as(rows), want.float()) and torch.equal(s.view_as(want_s), want_s)
    y, _ = kb.kda_add_rms_norm(sliced(x), w)
    assert torch.equal(y.view_as(rows), kb.kda_add_rms_norm(rows, w)[0])


@pytest.mark.gpu
def test_norm_refuses_rows_at_uneven_distances():
    w = torch.ones(64, device=DEV)
    wide = torch.zeros(4, 6, 64, device=DEV)
    for x in (wide[:, :5], wide.transpose(0, 1), wide[:, None, ::2][:, :, :2]):
        with pytest.raises(kb.KdaError, match="one row stride apart"):
            kb.kda_add_rms_norm(x, w)
