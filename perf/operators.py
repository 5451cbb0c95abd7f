"""The operators around the recurrent layer, as cases that can be timed and compared.

Four operators, which a served model runs in this order around a recurrent layer:

* ``norm``    the residual's addition and the root-mean-square norm, with an output in the
  input's type or in 8 bits (e4m3) with a scale for each row and 128 columns;
* ``matmul``  the product of such rows with 8-bit weights that have a scale for each 128 x 128
  block (a projection);
* ``conv``, ``conv_step``  the short causal convolution per channel with its SiLU, for packed
  prompts and for one token of each sequence;
* ``scan``, ``scan_step``  the selective state space scan, for packed prompts and for one token.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end), or, where ``own`` is true, by the library's entry points.
"""
import functools
import math
import random

import torch

own = False

GROUP = 128          # columns (or rows and columns) that share a scale
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -64  # a group's largest magnitude counts as at least this
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@functools.lru_cache(maxsize=None)
def _library():
    from gated_delta_rule_48_gb300 import binding
    return binding


# ------------------------------------------------------------------------------------ cases
def _case(name, op, **sizes):
    return {"name": name, "op": op, **sizes}


def listed():
    return [
        # one sequence decodes one token: a single row between two layers, all latency
        _case("norm_token", "norm", rows=1, dim=4096, dtype="bf16", residual=True, quant=False),
        # a batch of 4 prompts of 4096 tokens, normalised into the 8-bit projection's input
        _case("norm_prompt_8bit", "norm", rows=16384, dim=4096, dtype="bf16", residual=True,
              quant=True),
        # a ragged batch held in 32 bits, a width that is no multiple of a vector or a group
        _case("norm_ragged_f32", "norm", rows=1777, dim=2051, dtype="f32", residual=True,
              quant=True),
        # q, k and v projections of 32 decoding sequences (32 heads of 128): the weights' bytes
        _case("matmul_decode", "matmul", m=32, n=12288, k=4096, out="bf16"),
        # the same projections for a batch of 4 prompts of 4096 tokens: the largest case
        _case("matmul_prompt", "matmul", m=16384, n=12288, k=4096, out="bf16"),
        # a chunk of a prompt into a small odd projection (gates), kept in 32 bits
        _case("matmul_ragged", "matmul", m=1037, n=1001, k=2200, out="f32"),
        # the convolution after those projections, a uniform batch
        _case("conv_prompt", "conv", seqs=4, total=16384, dim=12288, width=4, packed=False,
              dtype="bf16", bias=False, silu=True, state=False, sliced=False),
        # packed prompts of uneven lengths, some empty, continued from a state; a column slice
        _case("conv_packed", "conv", seqs=37, total=20011, dim=2050, width=4, packed=True,
              dtype="bf16", bias=True, silu=True, state=True, sliced=True),
        # one token of each of 256 decoding sequences
        _case("conv_step", "conv_step", seqs=256, dim=12288, width=4, dtype="bf16", bias=True,
              silu=True, sliced=False),
        # a batch of 4 prompts of 4096 tokens through a scan of 4096 channels
        _case("scan_prompt", "scan", seqs=4, total=16384, dim=4096, state=16, groups=1,
              packed=False, dtype="bf16", gate=True, softplus=True, start=False, sliced=True),
        # 65,536 packed tokens in a few long documents, few channels: little to run side by side
        _case("scan_long", "scan", seqs=8, total=65536, dim=2048, state=16, groups=1,
              packed=True, dtype="bf16", gate=True, softplus=True, start=True, sliced=False),
        # one token of each of 256 decoding sequences
        _case("scan_step", "scan_step", seqs=256, dim=4096, state=16, groups=1, dtype="bf16",
              gate=True, softplus=True, sliced=False),
    ]


def _spread(rng, lo, hi):
    """A whole number, spread evenly over the range's logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _groups(rng, dim):
    return rng.choice([g for g in (1, 2, 4, 8) if dim % g == 0])


def draw(rng):
    op = rng.choice(["norm", "matmul", "conv", "conv_step", "scan", "scan_step"])
    flag = lambda: rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        dim = _spread(rng, 32, 16384)
        return dict(op=op, rows=_spread(rng, 1, min(32768, 100_000_000 // dim)), dim=dim,
                    dtype=dtype, residual=flag(), quant=flag())
    if op == "matmul":
        m, n = _spread(rng, 1, 16384), _spread(rng, 16, 16384)
        k = _spread(rng, 16, max(16, min(16384, 800_000_000_000 // (m * n))))
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "conv":
        dim = _spread(rng, 8, 16384)
        total = _spread(rng, 1, min(65536, 200_000_000 // dim))
        seqs = _spread(rng, 1, min(total, 256))
        packed = flag()
        if not packed:
            total = max(1, total // seqs) * seqs
        return dict(op=op, seqs=seqs, total=total, dim=dim, width=rng.choice([2, 3, 4, 4, 5, 8]),
                    packed=packed, dtype=dtype, bias=flag(), silu=flag(), state=flag(),
                    sliced=flag())
    if op == "conv_step":
        return dict(op=op, seqs=_spread(rng, 1, 1024), dim=_spread(rng, 8, 16384),
                    width=rng.choice([2, 3, 4, 4, 5, 8]), dtype=dtype, bias=flag(), silu=flag(),
                    sliced=flag())
    state = rng.choice([16, 16, 32, 64, 128])
    if op == "scan":
        dim = _spread(rng, 8, 8192)
        total = _spread(rng, 1, min(65536, 1_000_000_000 // (dim * state)))
        seqs = _spread(rng, 1, min(total, 128))
        packed = flag()
        if not packed:
            total = max(1, total // seqs) * seqs
        return dict(op=op, seqs=seqs, total=total, dim=dim, state=state, groups=_groups(rng, dim),
                    packed=packed, dtype=dtype, gate=flag(), softplus=flag(), start=flag(),
                    sliced=flag())
    dim = _spread(rng, 8, 8192)
    return dict(op=op, seqs=_spread(rng, 1, min(1024, 100_000_000 // (dim * state))), dim=dim,
                state=state, groups=_groups(rng, dim), dtype=dtype, gate=flag(), softplus=flag(),
                sliced=flag())


# ------------------------------------------------------------------------------------ inputs
def _lengths(total, seqs, packed, seed):
    """The sequences' lengths: equal, or cut at random places (empty ones among them)."""
    if not packed:
        return [total // seqs] * seqs
    rng = random.Random(seed * 7919 + 13)
    cuts = sorted(rng.randint(0, total) for _ in range(seqs - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _rows(rows, dim, dtype, gen, sliced=False, std=1.0):
    """[rows, dim] of normal values; `sliced`: some columns of a wider buffer, as a projection's
    output is cut up."""
    wide = dim + 48 if sliced else dim
    x = (torch.randn(rows, wide, device="cuda", generator=gen) * std).to(dtype)
    return x[:, 16:16 + dim] if sliced else x


def _sequences(case, seed):
    lens = _lengths(case["total"], case["seqs"], case["packed"], seed)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return lens, cu


def _quantise(x, by_rows):
    """Weights or rows in 8 bits: values, and the scales of their blocks (128 x 128, or each row's
    128 columns).  The values' rows start at multiples of 16 bytes."""
    rows, cols = x.shape
    gr, gc = (1 if by_rows else GROUP), GROUP
    pr, pc = -rows % gr, -cols % gc
    p = torch.nn.functional.pad(x, (0, pc, 0, pr))
    blocks = p.view((rows + pr) // gr, gr, (cols + pc) // gc, gc)
    scale = blocks.abs().amax(dim=(1, 3)).clamp(min=AMAX_MIN) / E4M3_MAX
    q = (blocks / scale[:, None, :, None]).view(rows + pr, cols + pc)[:rows, :cols]
    wide = torch.zeros(rows, cols + -cols % 16, dtype=torch.float8_e4m3fn, device=x.device)
    wide[:, :cols].copy_(q.to(torch.float8_e4m3fn))
    return wide[:, :cols], scale.contiguous()


def _ssm_inputs(case, tokens, dtype, gen):
    dim, state, groups, sliced = case["dim"], case["state"], case["groups"], case["sliced"]
    # steps of 0.001 to 0.1, decay rates of 1 to `state`, the usual start of such a layer
    step = torch.exp(torch.rand(dim, device="cuda", generator=gen) * math.log(100.0)
                     + math.log(1e-3))
    s = dict(x=_rows(tokens, dim, dtype, gen, sliced),
             B=_rows(tokens, groups * state, dtype, gen, sliced).unflatten(1, (groups, state)),
             C=_rows(tokens, groups * state, dtype, gen, sliced).unflatten(1, (groups, state)),
             A=-(torch.arange(1, state + 1, device="cuda", dtype=torch.float32)
                 * (0.9 + 0.2 * torch.rand(dim, state, device="cuda", generator=gen))),
             D=torch.ones(dim, device="cuda"),
             z=_rows(tokens, dim, dtype, gen, sliced) if case["gate"] else None)
    if case["softplus"]:
        s["dt"] = _rows(tokens, dim, dtype, gen, sliced, std=0.5)
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        noise = 0.5 + torch.rand(tokens, dim, device="cuda", generator=gen)
        s["dt"] = (step * noise).to(dtype)
        s["dt_bias"] = None
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        dtype = DTYPES[case["dtype"]]
        s["x"] = _rows(case["rows"], case["dim"], dtype, gen)
        s["residual"] = _rows(case["rows"], case["dim"], dtype, gen, std=4.0) \
            if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(case["dim"], device="cuda", generator=gen)) \
            .to(dtype)
    elif op == "matmul":
        a = torch.randn(case["m"], case["k"], device="cuda", generator=gen)
        a *= torch.exp(0.5 * torch.randn(case["m"], 1, device="cuda", generator=gen))
        s["a"], s["a_scale"] = _quantise(a, by_rows=True)
        b = torch.randn(case["n"], case["k"], device="cuda", generator=gen) * 0.02
        s["b"], s["b_scale"] = _quantise(b, by_rows=False)
    elif op in ("conv", "conv_step"):
        dtype = DTYPES[case["dtype"]]
        dim, width, seqs = case["dim"], case["width"], case["seqs"]
        tokens = case["total"] if op == "conv" else seqs
        s["x"] = _rows(tokens, dim, dtype, gen, case["sliced"])
        s["weight"] = (torch.randn(dim, width, device="cuda", generator=gen) * 0.5).to(dtype)
        s["bias"] = (torch.randn(dim, device="cuda", generator=gen) * 0.1).to(dtype) \
            if case["bias"] else None
        s["state"] = torch.randn(seqs, width - 1, dim, device="cuda", generator=gen).to(dtype) \
            if op == "conv_step" or case["state"] else None
        if op == "conv":
            s["lens"], s["cu"] = _sequences(case, seed)
    elif op == "scan":
        s |= _ssm_inputs(case, case["total"], DTYPES[case["dtype"]], gen)
        s["lens"], s["cu"] = _sequences(case, seed)
        s["h0"] = torch.randn(case["seqs"], case["dim"], case["state"], device="cuda",
                              generator=gen) * 0.1 if case["start"] else None
    else:
        s |= _ssm_inputs(case, case["seqs"], DTYPES[case["dtype"]], gen)
        s["h"] = torch.randn(case["seqs"], case["dim"], case["state"], device="cuda",
                             generator=gen) * 0.1
    return s


# ------------------------------------------------------------------------------ the plain forms
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    dtype = s["x"].dtype
    h = x.to(dtype) if s["residual"] is not None else None
    if not s["case"]["quant"]:
        return {"y": y.to(dtype), "h": h}
    rows, dim = y.shape
    groups = torch.nn.functional.pad(y, (0, -dim % GROUP)).view(rows, -1, GROUP)
    scale = groups.abs().amax(-1).clamp(min=AMAX_MIN) / E4M3_MAX
    q = (groups / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :dim]
    return {"y": q.to(torch.float8_e4m3fn), "y_scale": scale, "h": h}


def _spread_scales(scale, gr, gc, rows, cols):
    return scale.repeat_interleave(gr, 0)[:rows].repeat_interleave(gc, 1)[:, :cols]


def _plain_matmul(s):
    (m, k), n = s["a"].shape, s["b"].shape[0]
    a = s["a"].float() * _spread_scales(s["a_scale"], 1, GROUP, m, k)
    b = s["b"].float() * _spread_scales(s["b_scale"], GROUP, GROUP, n, k)
    return {"c": (a @ b.t()).to(DTYPES[s["case"]["out"]])}


def _token_sequences(cu, total):
    """For each token the number of its sequence."""
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(total, device=cu.device),
                              right=True)


def _plain_conv(s):
    x, w, cu = s["x"], s["weight"].float(), s["cu"].long()
    (total, dim), width, seqs = x.shape, w.shape[1], cu.numel() - 1
    back = width - 1
    # every sequence behind its own `back` earlier rows
    rows = torch.zeros(total + seqs * back, dim, device=x.device)
    at = torch.arange(total, device=x.device) + (_token_sequences(cu, total) + 1) * back
    rows[at] = x.float()
    first = cu[:-1] + torch.arange(seqs, device=x.device) * back
    before = first[:, None] + torch.arange(back, device=x.device)
    if s["state"] is not None:
        rows[before] = s["state"].float()
    v = (rows.unfold(0, width, 1) * w).sum(-1)[at - back]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if s["case"]["silu"]:
        v = _silu(v)
    after = before + (cu[1:] - cu[:-1])[:, None]
    return {"y": v.to(x.dtype), "state": rows[after].to(x.dtype)}


def _plain_conv_step(s):
    x, w, state = s["x"], s["weight"].float(), s["state"]
    rows = torch.cat([state, x[:, None]], 1)
    v = (rows.float() * w.t()).sum(1)
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if s["case"]["silu"]:
        v = _silu(v)
    state.copy_(rows[:, 1:])
    return {"y": v.to(x.dtype), "state": state}


def _plain_terms(s):
    """The step sizes, decays and additions of every token, in 32 bits: [tokens, dim, state]."""
    x, dt = s["x"].float(), s["dt"].float()
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"]
    if s["case"]["softplus"]:
        dt = _softplus(dt)
    per = s["case"]["dim"] // s["case"]["groups"]
    b = s["B"].float().repeat_interleave(per, 1)
    c = s["C"].float().repeat_interleave(per, 1)
    return x, c, torch.exp(dt[..., None] * s["A"]), b.mul_((dt * x)[..., None])


def _plain_readout(s, x, y):
    y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype)


def _plain_scan(s):
    x, c, a, b = _plain_terms(s)
    cu, lens = s["cu"].long(), s["lens"]
    total, seqs = x.shape[0], len(lens)
    full = (cu[1:] > cu[:-1]).nonzero().flatten()   # the sequences that are not empty
    if s["h0"] is not None:
        b[cu[full]] += a[cu[full]] * s["h0"][full]
    a[cu[full]] = 0.0                               # nothing passes a sequence's start
    # h_t = a_t h_(t-1) + b_t for all t by doubling: after a step of `reach`, (a, b) stand for
    # 2 * reach tokens
    reach = 1
    while reach < max(lens):
        b[reach:] += a[reach:] * b[:-reach]
        a[reach:] = a[reach:] * a[:-reach]
        reach *= 2
    h = torch.zeros(seqs, *b.shape[1:], device=b.device) if s["h0"] is None else s["h0"].clone()
    h[full] = b[cu[1:][full] - 1]
    return {"y": _plain_readout(s, x, (b * c).sum(-1)), "h": h}


def _plain_scan_step(s):
    x, c, a, b = _plain_terms(s)
    h = s["h"]
    h.mul_(a).add_(b)
    return {"y": _plain_readout(s, x, (h * c).sum(-1)), "h": h}


PLAIN = {"norm": _plain_norm, "matmul": _plain_matmul, "conv": _plain_conv,
         "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step}


# ------------------------------------------------------------------------- the library's calls
def _own(s):
    k, case = _library(), s["case"]
    op = case["op"]
    if op == "norm":
        if case["quant"]:
            y, scale, h = k.kda_add_rms_norm_quant(s["x"], s["weight"], s["residual"], eps=EPS)
            return {"y": y, "y_scale": scale, "h": h}
        y, h = k.kda_add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        return {"y": y, "h": h}
    if op == "matmul":
        return {"c": k.kda_matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"],
                                      out_dtype=DTYPES[case["out"]])}
    if op == "conv":
        y, state = k.kda_short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"],
                                        s["cu"] if case["packed"] else None,
                                        n_seqs=case["seqs"], silu=case["silu"])
        return {"y": y, "state": state}
    if op == "conv_step":
        y = k.kda_short_conv_step(s["x"], s["weight"], s["state"], s["bias"], silu=case["silu"])
        return {"y": y, "state": s["state"]}
    if op == "scan":
        y, h = k.kda_ssm_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                  s["dt_bias"], s["h0"], s["cu"] if case["packed"] else None,
                                  n_seqs=case["seqs"], softplus=case["softplus"])
        return {"y": y, "h": h}
    y = k.kda_ssm_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"], s["D"], s["z"],
                            s["dt_bias"], softplus=case["softplus"])
    return {"y": y, "h": s["h"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "norm":
        n = case["rows"] * case["dim"]
        read = n * e * (2 if case["residual"] else 1) + case["dim"] * e
        write = n * e if case["residual"] else 0
        write += n + 4 * case["rows"] * -(-case["dim"] // GROUP) if case["quant"] else n * e
        return {"bytes": read + write, "flops": 6 * n}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // GROUP)
        return {"bytes": m * k + n * k + 4 * blocks * (m + -(-n // GROUP))
                + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if op in ("conv", "conv_step"):
        dim, width = case["dim"], case["width"]
        tokens = case["total"] if op == "conv" else case["seqs"]
        reads = 2 if op == "conv_step" or case["state"] else 1   # the state in, the state out
        return {"bytes": e * dim * (2 * tokens + width + (1 if case["bias"] else 0)
                                    + reads * case["seqs"] * (width - 1)),
                "flops": tokens * dim * (2 * width + (4 if case["silu"] else 0))}
    tokens = case["total"] if op == "scan" else case["seqs"]
    dim, state = case["dim"], case["state"]
    rows = tokens * (dim * (4 if case["gate"] else 3) + 2 * case["groups"] * state)
    reads = 2 if op == "scan_step" or case["start"] else 1
    return {"bytes": e * rows + 4 * dim * (state + 2) + reads * 4 * case["seqs"] * dim * state,
            "flops": tokens * dim * (7 * state + 12)}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_norm(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double()
    out = {"h": h if s["residual"] is not None else None}
    if not s["case"]["quant"]:
        return out | {"y": y}
    rows, dim = y.shape
    number = torch.arange(dim, device=y.device) // GROUP
    top = torch.full((rows, int(number[-1]) + 1), AMAX_MIN, dtype=torch.float64, device=y.device)
    top.scatter_reduce_(1, number.expand(rows, dim), y.abs(), "amax")
    scale = top / E4M3_MAX
    return out | {"y": y / scale[:, number], "y_scale": scale}


def _exact_matmul(s):
    a, b, sa, sb = s["a"].double(), s["b"].double(), s["a_scale"].double(), s["b_scale"].double()
    k = torch.arange(a.shape[1], device=a.device) // GROUP
    n = torch.arange(b.shape[0], device=a.device) // GROUP
    a *= sa[:, k]
    b *= sb[n][:, k]
    return {"c": torch.matmul(a, b.t())}


def _exact_conv(s):
    x, w = s["x"].double(), s["weight"].double()
    back = w.shape[1] - 1
    v = torch.zeros_like(x)
    state = torch.zeros(len(s["lens"]), back, x.shape[1], dtype=torch.float64, device=x.device)
    if s["state"] is not None:
        state += s["state"].double()
    at = 0
    for n, length in enumerate(s["lens"]):
        rows = torch.cat([state[n], x[at:at + length]])
        for j in range(back + 1):
            v[at:at + length] += rows[j:j + length] * w[:, j]
        state[n] = rows[length:]
        at += length
    return _exact_activation(s, v) | {"state": state}


def _exact_activation(s, v):
    if s["bias"] is not None:
        v = v + s["bias"].double()
    return {"y": v * torch.sigmoid(v) if s["case"]["silu"] else v}


def _exact_conv_step(s):
    x, w, old = s["x"].double(), s["weight"].double(), s["state"].double()
    v = x * w[:, -1]
    for j in range(old.shape[1]):
        v += old[:, j] * w[:, j]
    return _exact_activation(s, v) | {"state": torch.cat([old[:, 1:], x[:, None]], 1)}


def _exact_tokens(s, h, rows):
    """One token of each of some sequences (its row of the inputs in `rows`): new h, and y."""
    case = s["case"]
    dt, x = s["dt"][rows].double(), s["x"][rows].double()
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"].double()
    if case["softplus"]:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    shape = (x.shape[0], case["groups"], -1, case["state"])
    new = h * torch.exp(dt[:, :, None] * s["A"].double())
    new = new.view(shape) + (dt * x).view(*shape[:3], 1) * s["B"][rows].double()[:, :, None]
    y = torch.einsum("ngds,ngs->ngd", new, s["C"][rows].double()).reshape(x.shape)
    y = y + s["D"].double() * x
    if s["z"] is not None:
        z = s["z"][rows].double()
        y = y * z * torch.sigmoid(z)
    return new.view(h.shape), y


def _exact_scan(s):
    lens, cu = s["lens"], s["cu"].tolist()
    if max(lens) > 70000:
        return None
    case = s["case"]
    h = torch.zeros(case["seqs"], case["dim"], case["state"], dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h += s["h0"].double()
    y = torch.zeros(case["total"], case["dim"], dtype=torch.float64, device="cuda")
    # longest first, so that the sequences that still have a token t are the first ones
    order = sorted(range(case["seqs"]), key=lambda n: -lens[n])
    first = torch.tensor([cu[n] for n in order], device="cuda")
    h = h[order]
    live = len(order)
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        rows = first[:live] + t
        h[:live], y[rows] = _exact_tokens(s, h[:live], rows)
    back = torch.empty_like(h)
    back[order] = h
    return {"y": y, "h": back}


def _exact_scan_step(s):
    h, y = _exact_tokens(s, s["h"].double(), torch.arange(s["case"]["seqs"], device="cuda"))
    return {"y": y, "h": h}


EXACT = {"norm": _exact_norm, "matmul": _exact_matmul, "conv": _exact_conv,
         "conv_step": _exact_conv_step, "scan": _exact_scan, "scan_step": _exact_scan_step}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
