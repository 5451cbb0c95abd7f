"""Two recurrent layers of a model, from residual stream to residual stream.

A delta-rule layer and a state space layer, each as it stands in a model that serves prompts
and then tokens:

    residual's addition, RMS norm, 8 bits  ->  8-bit projection  ->  short causal convolution
    ->  recurrence (kda_chunk_fwd_fused, or kda_ssm_scan_fwd)
    ->  RMS norm, 8 bits  ->  8-bit projection back

``prompt`` takes packed prompts and returns each sequence's states; ``step`` takes one token of
each sequence and moves the states on in place.  Run as a program it feeds the same tokens both
ways and compares:

    python examples/recurrent_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_48_gb300 import binding as kda  # noqa: E402

WIDTH = 4  # of the short convolutions


def quantise_weight(w):
    """e4m3 weights [out, in] with a scale for each 128 x 128 block, rows on 16-byte boundaries."""
    n, k = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    blocks = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    scale = blocks.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -64) / 448.0
    q = (blocks / scale[:, None, :, None]).view_as(p)[:n, :k]
    wide = torch.zeros(n, k + -k % 16, dtype=torch.float8_e4m3fn, device=w.device)
    wide[:, :k].copy_(q.to(torch.float8_e4m3fn))
    return wide[:, :k], scale.contiguous()


class Layer:
    """What both layers share: the norms and projections around a recurrence."""

    def __init__(self, dim, inner, columns, gen):
        rand = lambda *s, std: torch.randn(*s, device="cuda", generator=gen) * std
        self.norm_in = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        self.norm_out = torch.ones(inner, dtype=torch.bfloat16, device="cuda")
        self.w_in = quantise_weight(rand(columns, dim, std=dim ** -0.5))
        self.w_out = quantise_weight(rand(dim, inner, std=0.5 * inner ** -0.5))

    def project_in(self, x, residual):
        q, scale, h = kda.kda_add_rms_norm_quant(x, self.norm_in, residual)
        return kda.kda_matmul_fp8(q, scale, *self.w_in), h

    def project_out(self, y):
        q, scale, _ = kda.kda_add_rms_norm_quant(y, self.norm_out)
        return kda.kda_matmul_fp8(q, scale, *self.w_out)


class DeltaRuleLayer(Layer):
    def __init__(self, dim, heads, head_dim, gen):
        self.heads, self.d, self.inner = heads, head_dim, heads * head_dim
        super().__init__(dim, self.inner, 4 * self.inner + heads, gen)
        self.conv = [(torch.randn(self.inner, WIDTH, device="cuda", generator=gen) * 0.5).bfloat16()
                     for _ in range(3)]

    def _split(self, p):
        """q, k, v before their convolutions (columns of the projection), gate logits, beta."""
        n, shape = self.inner, (-1, self.heads, self.d)
        return ([p[:, i * n:(i + 1) * n] for i in range(3)],
                p[:, 3 * n:4 * n].contiguous().view(shape), torch.sigmoid(p[:, 4 * n:].float()))

    def prompt(self, x, residual, cu):
        p, h = self.project_in(x, residual)
        parts, gate, beta = self._split(p)
        convs = [kda.kda_short_conv_fwd(t, w, cu_seqlens=cu) for t, w in zip(parts, self.conv)]
        q, k, v = (y.view(-1, self.heads, self.d) for y, _ in convs)
        o, S = kda.kda_chunk_fwd_fused(q, k, v, gate, beta, cu_seqlens=cu)
        return self.project_out(o.flatten(1)), h, ([s for _, s in convs], S)

    def step(self, x, residual, state):
        p, h = self.project_in(x, residual)
        parts, gate, beta = self._split(p)
        q, k, v = (kda.kda_short_conv_step(t, w, s).view(-1, self.heads, self.d)
                   for t, w, s in zip(parts, self.conv, state[0]))
        o = kda.kda_decode_step_fused(q, k, v, gate, beta, state[1])
        return self.project_out(o.flatten(1)), h


class StateSpaceLayer(Layer):
    def __init__(self, dim, inner, states, gen):
        self.inner, self.states = inner, states
        super().__init__(dim, inner, 3 * inner + 2 * states, gen)
        self.conv = (torch.randn(inner, WIDTH, device="cuda", generator=gen) * 0.5).bfloat16()
        self.A = -torch.arange(1, states + 1, device="cuda").float().repeat(inner, 1)
        self.D = torch.ones(inner, device="cuda")
        self.dt_bias = torch.full((inner,), -4.0, device="cuda")  # steps about 0.02

    def _split(self, p):
        """x, z, dt [tokens, inner], B and C [tokens, 1, states]: columns of the projection."""
        n, s = self.inner, self.states
        return (p[:, :n], p[:, n:2 * n], p[:, 2 * n:3 * n],
                p[:, 3 * n:3 * n + s].unsqueeze(1), p[:, 3 * n + s:].unsqueeze(1))

    def prompt(self, x, residual, cu):
        p, h = self.project_in(x, residual)
        x, z, dt, B, C = self._split(p)
        x, conv = kda.kda_short_conv_fwd(x, self.conv, cu_seqlens=cu)
        y, state = kda.kda_ssm_scan_fwd(x, dt, self.A, B, C, self.D, z, self.dt_bias, cu_seqlens=cu)
        return self.project_out(y), h, (conv, state)

    def step(self, x, residual, state):
        p, h = self.project_in(x, residual)
        x, z, dt, B, C = self._split(p)
        x = kda.kda_short_conv_step(x, self.conv, state[0])
        y = kda.kda_ssm_scan_step(x, dt, self.A, B, C, state[1], self.D, z, self.dt_bias)
        return self.project_out(y), h


class Block:
    """Both layers, and the norm of the stream behind them."""

    def __init__(self, dim=512, heads=4, head_dim=64, inner=512, states=16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.layers = [DeltaRuleLayer(dim, heads, head_dim, gen),
                       StateSpaceLayer(dim, inner, states, gen)]
        self.norm = torch.ones(dim, dtype=torch.bfloat16, device="cuda")

    def prompt(self, x, cu):
        delta, h, states = x, torch.zeros_like(x), []
        for layer in self.layers:
            delta, h, state = layer.prompt(delta, h, cu)
            states.append(state)
        y, _ = kda.kda_add_rms_norm(delta, self.norm, h)
        return y, states

    def step(self, x, states):
        delta, h = x, torch.zeros_like(x)
        for layer, state in zip(self.layers, states):
            delta, h = layer.step(delta, h, state)
        y, _ = kda.kda_add_rms_norm(delta, self.norm, h)
        return y


def compare(lens=(70, 1, 130), new=8, dim=512, seed=0):
    """The last `new` tokens of each sequence, once as part of its prompt and once as steps after
    a shorter prompt: the largest difference of the outputs over their root mean square."""
    block = Block(dim, seed=seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    seqs = [torch.randn(n + new, dim, device="cuda", generator=gen).bfloat16() for n in lens]

    def packed(parts):
        ends = torch.tensor([0] + [len(p) for p in parts]).cumsum(0)
        return torch.cat(parts), ends.to(torch.int32).cuda()

    full, _ = block.prompt(*packed(seqs))
    ends = torch.tensor([n + new for n in lens]).cumsum(0).tolist()
    want = torch.stack([full[e - new:e] for e in ends])           # [sequences, new, dim]
    _, states = block.prompt(*packed([s[:-new] for s in seqs]))
    got = torch.stack([block.step(torch.stack([s[n + t] for s, n in zip(seqs, lens)]), states)
                       for t in range(new)], 1)
    if kda.kda_get_device_error() != 0:
        raise RuntimeError(kda.load().kda_last_error_message().decode())
    want, got = want.float(), got.float()
    return ((got - want).norm() / want.norm()).item(), (got - want).abs().max().item()


def main():
    rel, worst = compare()
    print(f"8 tokens of 3 sequences, as steps against as part of the prompts: "
          f"relative difference {rel:.2e}, largest {worst:.3f}")
    return rel


if __name__ == "__main__":
    main()
