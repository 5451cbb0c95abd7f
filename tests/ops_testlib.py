"""Helpers of the tests of the operators around the layer: tolerances derived
from the roundings each operator makes, and comparisons against 64-bit
references."""
from __future__ import annotations

import torch

DEV = "cuda"
BF16_HALF = 2.0 ** -8   # half a unit of the last place of bf16, relative
F32_HALF = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def half_ulp(dtype):
    return BF16_HALF if dtype == torch.bfloat16 else F32_HALF


def assert_near(got, want, rel, what, atol=0.0):
    """|got - want| <= rel |want| + atol, element by element; NaN and infinities in the same
    places."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = want.isfinite()
    err = (got - want).abs()[ok]
    bound = (rel * want.abs() + atol)[ok]
    if err.numel():
        worst = (err - bound).max().item()
        assert worst <= 0.0, f"{what}: off by {err.max().item():.3e}, {worst:.3e} over its bound"


def sliced(t, left=3, right=5):
    """The same values as some columns of a wider buffer: odd strides and starts."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + left + right, dtype=t.dtype, device=t.device)
    wide[..., left:left + t.shape[-1]] = t
    return wide[..., left:left + t.shape[-1]]
