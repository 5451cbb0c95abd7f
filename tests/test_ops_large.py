"""The operators around the layer where an element's place passes 2^31, with scales that are
infinite, and from two host threads.

Rows far apart: a few rows of every operand, 4.8e9 bytes from one to the next, in one buffer for
the inputs and one for the outputs; the results are those of the same rows side by side, bit for
bit, and what lies between the outputs' rows stays as it was."""
import threading

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb
from ops_testlib import DEV, assert_near, gen, half_ulp, randn

pytestmark = pytest.mark.gpu

PITCH = 4_800_000_000   # bytes: 1.2e9 32-bit, 2.4e9 16-bit elements
ROWS = 3
COLUMNS = 1 << 20       # bytes of each row in use


class Far:
    """Rows PITCH bytes apart, handed out from left to right."""

    def __init__(self):
        self.bytes = torch.empty((ROWS - 1) * PITCH + COLUMNS, dtype=torch.uint8, device=DEV)
        for r in range(ROWS):
            self.bytes[r * PITCH:r * PITCH + COLUMNS] = 0x55
        self.used = 0

    def like(self, shape, dtype):
        """A tensor of that shape, its first dimension the rows."""
        size = torch.empty(0, dtype=dtype).element_size()
        start = self.used // size
        n = 1
        for s in shape[1:]:
            n *= s
        self.used += (n * size + 255) // 256 * 256 + 256
        strides = [1] * len(shape)
        for k in range(len(shape) - 2, 0, -1):
            strides[k] = strides[k + 1] * shape[k + 1]
        return self.bytes.view(dtype).as_strided(shape, [PITCH // size, *strides[1:]], start)

    def put(self, t):
        return self.like(t.shape, t.dtype).copy_(t)

    def untouched(self):
        """The bytes behind the last tensor of each row."""
        return all((self.bytes[r * PITCH + self.used:r * PITCH + COLUMNS] == 0x55).all() for r in range(ROWS))


@pytest.fixture
def far():
    yield Far(), Far()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [256, 301])
def test_norm(far, dim, dtype):
    g = gen(dim)
    x, r, w = randn(g, ROWS, dim, dtype=dtype), randn(g, ROWS, dim, dtype=dtype), randn(g, dim, dtype=dtype)
    ins, outs = far
    y, h, s = outs.like((ROWS, dim), dtype), outs.like((ROWS, dim), dtype), outs.like((ROWS, 3), torch.float32)
    q = outs.like((ROWS, dim), torch.float8_e4m3fn)
    fx, fr = ins.put(x), ins.put(r)
    want, want_h = kb.kda_add_rms_norm(x, w, r)
    kb.kda_add_rms_norm(fx, w, fr, y=y, h=h)
    assert torch.equal(y, want) and torch.equal(h, want_h)
    want, want_s, _ = kb.kda_add_rms_norm_quant(x, w, r)
    n = want_s.shape[1]
    kb.kda_add_rms_norm_quant(fx, w, fr, y=q, y_scale=s[:, :n], h=h)
    assert torch.equal(q.float(), want.float()) and torch.equal(s[:, :n], want_s) and torch.equal(h, want_h)
    assert outs.untouched() and kb.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [8, 300])
def test_matmul(far, N, dtype):
    g = gen(N)
    K = 400
    v = lambda n: (torch.randn(n, K, device=DEV, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    a, sa = v(ROWS), torch.rand(ROWS, 4, device=DEV, generator=g)
    b, sb = v(N), torch.rand(-(-N // 128), 4, device=DEV, generator=g)
    ins, outs = far
    out = outs.like((ROWS, N), dtype)
    want = kb.kda_matmul_fp8(a, sa, b, sb, out_dtype=dtype)
    kb.kda_matmul_fp8(ins.put(a), ins.put(sa), b, sb, out)
    assert torch.equal(out, want)
    # the weights' rows far apart, and so many rows of A that each has a lane
    wide, swide = v(200), torch.rand(200, 4, device=DEV, generator=g)
    want = kb.kda_matmul_fp8(wide, swide, a, sa[:1], out_dtype=dtype)
    assert torch.equal(kb.kda_matmul_fp8(wide, swide, ins.put(a), sa[:1], out_dtype=dtype), want)
    assert outs.untouched() and kb.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 33])
def test_convolution(far, dim, dtype):
    g = gen(dim)
    x, w = randn(g, ROWS, dim, dtype=dtype), randn(g, dim, 4, dtype=dtype)
    ins, outs = far
    y, fx = outs.like((ROWS, dim), dtype), ins.put(x)
    want, want_s = kb.kda_short_conv_fwd(x, w)
    _, s = kb.kda_short_conv_fwd(fx, w, y=y)
    assert torch.equal(y, want) and torch.equal(s, want_s)
    state = randn(g, ROWS, 3, dim, dtype=dtype)
    state2 = state.clone()
    want = kb.kda_short_conv_step(x, w, state)
    kb.kda_short_conv_step(fx, w, state2, y=y)
    assert torch.equal(y, want) and torch.equal(state2, state)
    assert outs.untouched() and kb.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,G", [(64, 2), (33, 1)])
def test_scan(far, dim, G, dtype):
    g = gen(dim)
    S = 16
    x, dt, z = (randn(g, ROWS, dim, dtype=dtype) for _ in range(3))
    B, C = (randn(g, ROWS, G, S, dtype=dtype) for _ in range(2))
    A = -torch.rand(dim, S, device=DEV, generator=g)
    ins, outs = far
    y = outs.like((ROWS, dim), dtype)
    fx, fdt, fz, fB, fC = (ins.put(t) for t in (x, dt, z, B, C))
    want, want_h = kb.kda_ssm_scan_fwd(x, dt, A, B, C, None, z)
    _, h = kb.kda_ssm_scan_fwd(fx, fdt, A, fB, fC, None, fz, y=y)
    assert torch.equal(y, want) and torch.equal(h, want_h)
    h = randn(g, ROWS, dim, S)
    h2 = h.clone()
    want = kb.kda_ssm_scan_step(x, dt, A, B, C, h, None, z)
    kb.kda_ssm_scan_step(fx, fdt, A, fB, fC, h2, None, fz, y=y)
    assert torch.equal(y, want) and torch.equal(h2, h)
    assert outs.untouched() and kb.kda_get_device_error() == 0


def test_states_of_more_than_2_31_values():
    """The last sequences' steps and convolutions, whose states lie behind 2^31 others."""
    g = gen(5)
    N, dim, S = 2100, 8192, 128
    h = torch.zeros(N, dim, S, device=DEV)
    x, dt = randn(g, N, dim, dtype=torch.bfloat16), randn(g, N, dim, dtype=torch.bfloat16)
    B, C = (randn(g, N, 1, S, dtype=torch.bfloat16) for _ in range(2))
    A = -torch.rand(dim, S, device=DEV, generator=g)
    last = slice(N - 2, N)
    h[last] = randn(g, 2, dim, S)
    h2 = h[last].clone()
    y = kb.kda_ssm_scan_step(x, dt, A, B, C, h)
    want = kb.kda_ssm_scan_step(x[last], dt[last], A, B[last], C[last], h2)
    assert torch.equal(y[last], want) and torch.equal(h[last], h2)
    # (the same as one token of each prompt: states read and written whole)
    y2, h3 = kb.kda_ssm_scan_fwd(x, dt, A, B, C, h0=h, n_seqs=N)
    want, h4 = kb.kda_ssm_scan_fwd(x[last], dt[last], A, B[last], C[last], h0=h2, n_seqs=2)
    assert_near(y2[last], want.double(), 2 * half_ulp(torch.bfloat16), "y", atol=1e-4)
    assert_near(h3[last], h4.double(), 1e-6, "h", atol=1e-6)
    del h, h3
    N, dim = 40_000, 8192
    state = torch.zeros(N, 7, dim, dtype=torch.bfloat16, device=DEV)
    x, w = randn(g, N, dim, dtype=torch.bfloat16), randn(g, dim, 8, dtype=torch.bfloat16)
    last = slice(N - 2, N)
    state[last] = randn(g, 2, 7, dim, dtype=torch.bfloat16)
    state2 = state[last].clone()
    y = kb.kda_short_conv_step(x, w, state)
    want = kb.kda_short_conv_step(x[last], w, state2)
    assert torch.equal(y[last], want) and torch.equal(state[last], state2)
    assert kb.kda_get_device_error() == 0
    del state
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [5, 40, 200, 1000])
def test_infinite_scales_stay_in_their_rows(M):
    g = gen(M)
    v = lambda n: (torch.randn(n, 300, device=DEV, generator=g) * 60).clamp(-448, 448)
    wide = torch.zeros(M + 300, 304, dtype=torch.float8_e4m3fn, device=DEV)
    a, b = wide[:M, :300], wide[M:, :300]
    a.copy_(v(M)), b.copy_(v(300))
    sa, sb = torch.rand(M, 3, device=DEV, generator=g) + 0.1, torch.rand(3, 3, device=DEV, generator=g) + 0.1
    clean = kb.kda_matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)
    sa2 = sa.clone()
    sa2[3, 1] = float("inf")
    out = kb.kda_matmul_fp8(a, sa2, b, sb, out_dtype=torch.float32)
    block = a[3:4, 128:256].double() @ b[:, 128:256].double().t()
    want = torch.where(block == 0, float("nan"), block * float("inf"))[0]
    assert torch.equal(out[3].isnan(), want.isnan()) and torch.equal(out[3].nan_to_num(7), want.float().nan_to_num(7))
    keep = [m for m in range(M) if m != 3]
    assert torch.equal(out[keep], clean[keep])
    sb2 = sb.clone()
    sb2[1, 2] = float("inf")
    out = kb.kda_matmul_fp8(a, sa, b, sb2, out_dtype=torch.float32)
    assert not out[:, 128:256].isfinite().any()
    assert torch.equal(out[:, :128], clean[:, :128]) and torch.equal(out[:, 256:], clean[:, 256:])


def test_calls_from_two_host_threads():
    """Each on its own stream, refusals among them: results as from one thread, and each thread's
    own message."""
    g = gen(1)
    x, w = randn(g, 300, 512, dtype=torch.bfloat16), randn(g, 512, dtype=torch.bfloat16)
    cw = randn(g, 512, 4, dtype=torch.bfloat16)
    want = [kb.kda_add_rms_norm(x, w)[0], kb.kda_short_conv_fwd(x, cw)[0]]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        try:
            side = torch.cuda.Stream()
            for _ in range(200):
                got = (kb.kda_add_rms_norm(x, w, stream=side) if k == 0
                       else kb.kda_short_conv_fwd(x, cw, stream=side))[0]
                side.synchronize()
                if not torch.equal(got, want[k]):
                    wrong.append((k, "result"))
                with pytest.raises(kb.KdaError, match="eps" if k == 0 else "width"):
                    if k == 0:
                        kb.kda_add_rms_norm(x, w, eps=-1.0, stream=side)
                    else:
                        kb.kda_short_conv_fwd(x, cw[:, :1].contiguous(), stream=side)
        except BaseException as e:
            wrong.append((k, repr(e)))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert kb.kda_get_device_error() == 0
