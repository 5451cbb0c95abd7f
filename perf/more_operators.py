"""Full attention and its cache in 4 bits, as cases that can be timed and compared.

A model that interleaves recurrent layers with full-attention ones runs, for those:

* ``attn``       attention over packed or uniform prompts, with grouped heads, where the queries
  may be the last tokens of longer sequences (a prompt's next chunk);
* ``kv4_write``  the keys and values of new tokens, quantised into a paged cache of 4-bit codes,
  and those tokens read back as what they now stand for;
* ``kv4_read``   whole prefixes read back from that cache;
* ``kv4_attn``   one token (or a draft of a few) of each sequence over that cache.

The cache holds, for each token and head, groups of 32 channels: a scale s = bf16(max(max |x|,
2^-64) / 7) and codes n + 8 with n = x / s rounded half to even; a code stands for n s.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end), or, where ``own`` is true, by the library's entry points.
"""
import functools
import math
import random

import torch

own = False

GROUP = 32             # channels of a token and head that share a scale
AMAX_MIN = 2.0 ** -64  # a group's largest magnitude counts as at least this


@functools.lru_cache(maxsize=None)
def _library():
    from gated_delta_rule_48_gb300 import binding
    return binding


# ------------------------------------------------------------------------------------ cases
def _case(name, op, **sizes):
    return {"name": name, "op": op, **sizes}


def listed():
    return [
        # one short question to a model: a single sequence of 100 tokens, all latency
        _case("attn_short", "attn", seqs=1, total=100, context=0, heads=32, kv_heads=8, d=128,
              packed=False, causal=True, lse=False, sliced=True),
        # a batch of 4 prompts of 4096 tokens, 32 query heads in groups of 4
        _case("attn_prompt", "attn", seqs=4, total=16384, context=0, heads=32, kv_heads=8, d=128,
              packed=False, causal=True, lse=False, sliced=True),
        # one document of 32,768 tokens: the largest case
        _case("attn_long", "attn", seqs=1, total=32768, context=0, heads=16, kv_heads=2, d=128,
              packed=False, causal=True, lse=True, sliced=False),
        # packed prompts of uneven lengths, some empty, small heads in groups of 3
        _case("attn_packed", "attn", seqs=37, total=20011, context=0, heads=12, kv_heads=4, d=64,
              packed=True, causal=True, lse=False, sliced=False),
        # the next chunk of 8 prompts, behind some 3900 tokens each that were read back
        _case("attn_chunk", "attn", seqs=8, total=2101, context=31337, heads=32, kv_heads=4,
              d=128, packed=True, causal=True, lse=True, sliced=False),
        # one token of each of 256 decoding sequences into the cache
        _case("kv4_write_step", "kv4_write", seqs=256, total=256, kv_heads=8, d=128, page=64,
              packed=False, behind=True, sliced=True),
        # a batch of 4 prompts of 4096 tokens into the cache
        _case("kv4_write_prompt", "kv4_write", seqs=4, total=16384, kv_heads=8, d=128, page=64,
              packed=False, behind=False, sliced=True),
        # prefixes of 8 sequences, 65,536 tokens in all, read back
        _case("kv4_read_prefix", "kv4_read", seqs=8, total=65536, kv_heads=8, d=128, page=64,
              packed=True, behind=False),
        # ragged prefixes of small heads, not from their first token on
        _case("kv4_read_ragged", "kv4_read", seqs=19, total=3333, kv_heads=3, d=64, page=16,
              packed=True, behind=True),
        # one token of each of 256 decoding sequences of 2048 to 6144 tokens
        _case("kv4_attn_batch", "kv4_attn", seqs=256, total=1048576, tokens=1, heads=32,
              kv_heads=8, d=128, page=64, lse=False),
        # one sequence of 131,072 tokens decodes one token: little to run side by side
        _case("kv4_attn_long", "kv4_attn", seqs=1, total=131072, tokens=1, heads=32, kv_heads=8,
              d=128, page=64, lse=True),
        # drafts of 4 tokens of a few sequences of uneven lengths, small heads
        _case("kv4_attn_draft", "kv4_attn", seqs=5, total=7777, tokens=4, heads=12, kv_heads=4,
              d=64, page=16, lse=False),
    ]


def _spread(rng, lo, hi):
    """A whole number, spread evenly over the range's logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "kv4_write", "kv4_read", "kv4_attn", "kv4_attn"])
    flag = lambda: rng.random() < 0.5
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("attn", "kv4_attn"):
        heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "attn":
        seqs = _spread(rng, 1, 64)
        # no more than 2^32 pairs of a query and a key over all heads
        longest = int(math.sqrt(2 ** 32 * seqs / heads))
        total = _spread(rng, seqs, min(32768, longest))
        context = _spread(rng, 1, 2 * longest) if rng.random() < 0.4 else 0
        context = min(context, 65536, int(2 ** 32 * seqs / heads / total))
        packed = flag()
        if not packed:
            total, context = total // seqs * seqs, context // seqs * seqs
        return dict(op=op, seqs=seqs, total=total, context=context, heads=heads,
                    kv_heads=kv_heads, d=d, packed=packed, causal=rng.random() < 0.8, lse=flag(),
                    sliced=flag())
    if op in ("kv4_write", "kv4_read"):
        seqs = _spread(rng, 1, 256)
        total = _spread(rng, seqs, 65536)
        packed = flag()
        if not packed:
            total = total // seqs * seqs
        case = dict(op=op, seqs=seqs, total=total, kv_heads=kv_heads, d=d, page=page,
                    packed=packed, behind=flag())
        return case | dict(sliced=flag()) if op == "kv4_write" else case
    seqs, tokens = _spread(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 5])
    total = _spread(rng, seqs * 8, min(131072 * seqs, 8_000_000 // kv_heads))
    return dict(op=op, seqs=seqs, total=total, tokens=tokens, heads=heads, kv_heads=kv_heads, d=d,
                page=page, lse=flag())


def _lengths(total, seqs, packed, salt):
    """The sequences' lengths, by the case alone: equal, or cut at random places (empty ones
    among them)."""
    if not packed:
        return [total // seqs] * seqs
    rng = random.Random(total * 7919 + seqs * 31 + salt)
    cuts = sorted(rng.randint(0, total) for _ in range(seqs - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _attn_lengths(case):
    q = _lengths(case["total"], case["seqs"], case["packed"], 0)
    c = _lengths(case["context"], case["seqs"], case["packed"], 1)
    return q, [a + b for a, b in zip(q, c)]


def _cache_lengths(case):
    """kv4_attn: lengths from half to one and a half of the mean, the queries among them."""
    mean = case["total"] / case["seqs"]
    if case["seqs"] == 1:
        return [max(case["tokens"], case["total"])]
    rng = random.Random(case["total"] * 7919 + case["seqs"])
    return [max(case["tokens"], int(mean * rng.uniform(0.5, 1.5))) for _ in range(case["seqs"])]


def _spans(case):
    """kv4_write, kv4_read: each sequence's first position, and its length."""
    lens = _lengths(case["total"], case["seqs"], case["packed"], 0)
    rng = random.Random(case["total"] * 31 + case["seqs"])
    return [rng.randint(0, 600) if case["behind"] else 0 for _ in lens], lens


# ------------------------------------------------------------------------------------ inputs
def _cu(lens):
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    return torch.tensor(starts, dtype=torch.int32, device="cuda")


def _heads(tokens, heads, d, gen, sliced=False, gain=None):
    """[tokens, heads, d] of normal values in bf16; `sliced`: columns of a wider buffer, as a
    projection's output is cut up."""
    n = heads * d
    x = torch.empty(tokens, n + 64 if sliced else n, dtype=torch.bfloat16, device="cuda")
    for at in range(0, tokens, 1 << 15):   # (32-bit values of a part at a time)
        part = torch.randn(min(1 << 15, tokens - at), x.shape[1], device="cuda", generator=gen)
        x[at:at + (1 << 15)] = part
    x = (x[:, 16:16 + n] if sliced else x).unflatten(1, (heads, d))
    return x if gain is None else x.mul_(gain)


def _gain(heads, d, gen):
    """Keys have channels that are larger than others in all tokens."""
    return torch.exp(0.4 * torch.randn(heads, d, device="cuda", generator=gen)).bfloat16()


def _table(case, lens, seed):
    """Pages of each sequence, in no order, a few of the cache left over."""
    counts = [-(-n // case["page"]) for n in lens]
    rng = random.Random(seed)
    pages = list(range(sum(counts) + 3))
    rng.shuffle(pages)
    width, at, rows = max(max(counts), 1), 0, []
    for n in counts:
        rows.append(pages[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), len(pages)


def _cache(case, pages):
    """Codes and scales of keys, then of values."""
    shape = (pages, case["kv_heads"], case["page"])
    new = lambda n, dtype: torch.zeros(*shape, n, dtype=dtype, device="cuda")
    d = case["d"]
    return (new(d // 2, torch.uint8), new(d // GROUP, torch.bfloat16),
            new(d // 2, torch.uint8), new(d // GROUP, torch.bfloat16))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, d, kv_heads = case["op"], case["d"], case["kv_heads"]
    s = dict(case=case, scale=d ** -0.5)
    if op == "attn":
        s["q_lens"], s["k_lens"] = _attn_lengths(case)
        s["cu_q"], s["cu_k"] = _cu(s["q_lens"]), _cu(s["k_lens"])
        keys = sum(s["k_lens"])
        s["q"] = _heads(case["total"], case["heads"], d, gen, case["sliced"])
        s["k"] = _heads(keys, kv_heads, d, gen, case["sliced"], _gain(kv_heads, d, gen))
        s["v"] = _heads(keys, kv_heads, d, gen, case["sliced"])
        return s
    if op == "kv4_write":
        start, s["lens"] = _spans(case)
        s["table"], pages = _table(case, [a + n for a, n in zip(start, s["lens"])], seed)
        s["cache"] = _cache(case, pages)
        s["k"] = _heads(case["total"], kv_heads, d, gen, case["sliced"], _gain(kv_heads, d, gen))
        s["v"] = _heads(case["total"], kv_heads, d, gen, case["sliced"])
    else:  # a cache in which whole sequences lie
        if op == "kv4_read":
            start, s["lens"] = _spans(case)
            held = [a + n for a, n in zip(start, s["lens"])]
        else:
            start, held = None, _cache_lengths(case)
            s["lens"] = held
            s["seq_lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
            shape = (case["seqs"], case["tokens"], case["heads"], d)
            s["q"] = torch.randn(shape, device="cuda", generator=gen).bfloat16()
            if case["tokens"] == 1:
                s["q"] = s["q"][:, 0]
        s["table"], pages = _table(case, held, seed)
        s["cache"] = _cache(case, pages)
        gain = _gain(kv_heads, d, gen)
        slots = pages * case["page"]
        for at in range(0, slots, 1 << 17):   # every slot, in parts
            n = min(1 << 17, slots - at)
            to = torch.arange(at, at + n, device="cuda")
            _store(s["cache"], to, _heads(n, kv_heads, d, gen, gain=gain),
                   _heads(n, kv_heads, d, gen))
    if start is not None:
        s["cu"] = _cu(s["lens"])
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------ the plain forms
def _order(d, keys, device):
    """For each nibble of a row, in order, the channel whose code it holds: a key's 32-bit word
    j G + g holds channels 32 g + 8 j + 0..7, a value's 16-bit word r G + g channels
    32 g + 4 r + 0..3 (G = d / 32 groups)."""
    run = 8 if keys else 4
    c = torch.arange(d, device=device).view(d // GROUP, GROUP // run, run)
    return c.transpose(0, 1).reshape(d)


def _quantise(x):
    """Whole numbers in [-7, 7], and the groups' scales (bf16)."""
    g = x.float().unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1).clamp(min=AMAX_MIN) / 7.0).bfloat16()
    return torch.round(g / scale.float()[..., None]).flatten(-2).to(torch.int8), scale


def _store(cache, slots, k, v):
    """Tokens k, v [T, heads, d] into slots (page * page size + place) of the cache."""
    page, at = slots // cache[0].shape[2], slots % cache[0].shape[2]
    for i, x in ((0, k), (2, v)):
        n, scale = _quantise(x)
        nibbles = (n + 8).to(torch.uint8)[..., _order(x.shape[-1], i == 0, x.device)]
        cache[i][page, :, at] = nibbles[..., 0::2] | nibbles[..., 1::2] << 4
        cache[i + 1][page, :, at] = scale


def _load(cache, slots, keys, dtype=torch.float32):
    """What the slots' codes stand for: [T, heads, d]."""
    codes, scales = cache[0 if keys else 2], cache[1 if keys else 3]
    page, at = slots // codes.shape[2], slots % codes.shape[2]
    c = codes[page, :, at]
    nibbles = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    n = torch.empty(nibbles.shape, dtype=dtype, device=c.device)
    n[..., _order(nibbles.shape[-1], keys, c.device)] = nibbles.to(dtype) - 8
    return (n.unflatten(-1, (-1, GROUP)) * scales[page, :, at].to(dtype)[..., None]).flatten(-2)


def _slots(s):
    """The slots of the tokens of all sequences' spans."""
    cu, page = s["cu"].long(), s["case"]["page"]
    token = torch.arange(s["case"]["total"], device="cuda")
    n = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    position = s["start"].long()[n] + token - cu[n]
    return s["table"].long()[n, position // page] * page + position % page


def _attend(q, k, v, scale, reach):
    """q [Q, heads, d] over k, v [L, kv_heads, d], query i over the first reach[i] keys:
    o [Q, heads, d] and the logarithms of the sums."""
    g = q.shape[1] // k.shape[1]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype, device=q.device)
    step = max(1, (1 << 28) // max(1, g * k.shape[0]))   # queries at a time
    for h in range(k.shape[1]):
        for a in range(0, q.shape[0], step):
            r = reach[a:a + step]
            n = int(r[-1])
            if n <= 0:
                continue
            x = q[a:a + step, h * g:(h + 1) * g].transpose(0, 1) @ k[:n, h].t() * scale
            x = x.masked_fill_(torch.arange(n, device=q.device) >= r[:, None].to(q.device), -math.inf)
            top = x.amax(-1, keepdim=True).clamp(min=-1e30)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            o = (x @ v[:n, h]) / total
            out[a:a + step, h * g:(h + 1) * g] = o.transpose(0, 1).nan_to_num_(nan=0.0) \
                if int(r[0]) <= 0 else o.transpose(0, 1)
            lse[a:a + step, h * g:(h + 1) * g] = (top + total.log()).squeeze(-1).t()
    return out, lse


def _sequences(s):
    """Each sequence's first query and key, their counts, and how many keys each query reaches."""
    q0 = k0 = 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        reach = torch.arange(nq) + (nk - nq + 1) if s["case"]["causal"] else torch.full((nq,), nk)
        yield q0, k0, nq, nk, reach.clamp(0, nk)
        q0, k0 = q0 + nq, k0 + nk


def _all_sequences(s, dtype):
    o = torch.zeros(s["q"].shape, dtype=dtype, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=dtype, device="cuda")
    for q0, k0, nq, nk, reach in _sequences(s):
        if nq and nk:
            o[q0:q0 + nq], lse[q0:q0 + nq] = _attend(
                s["q"][q0:q0 + nq].to(dtype), s["k"][k0:k0 + nk].to(dtype),
                s["v"][k0:k0 + nk].to(dtype), s["scale"], reach)
    return o, lse


def _attn_out(s, o, lse):
    return {"o": o, "lse": lse} if s["case"]["lse"] else {"o": o}


def _plain_attn(s):
    o, lse = _all_sequences(s, torch.float32)
    return _attn_out(s, o.bfloat16(), lse)


def _plain_read(s):
    slots = _slots(s)
    return {"k": _load(s["cache"], slots, True).bfloat16(),
            "v": _load(s["cache"], slots, False).bfloat16()}


def _plain_write(s):
    _store(s["cache"], _slots(s), s["k"], s["v"])
    return _plain_read(s)


def _over_cache(s, dtype):
    case = s["case"]
    page, tokens = case["page"], case["tokens"]
    q = s["q"].to(dtype).view(case["seqs"], tokens, case["heads"], case["d"])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=dtype, device="cuda")
    for n, length in enumerate(s["lens"]):
        position = torch.arange(length, device="cuda")
        slots = s["table"][n].long()[position // page] * page + position % page
        reach = torch.arange(tokens) + (length - tokens + 1)
        o[n], lse[n] = _attend(q[n], _load(s["cache"], slots, True, dtype),
                               _load(s["cache"], slots, False, dtype), s["scale"], reach)
    return o.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _plain_kv4_attn(s):
    o, lse = _over_cache(s, torch.float32)
    return _attn_out(s, o.bfloat16(), lse)


PLAIN = {"attn": _plain_attn, "kv4_write": _plain_write, "kv4_read": _plain_read,
         "kv4_attn": _plain_kv4_attn}


# ------------------------------------------------------------------------- the library's calls
def _own(s):
    lib, case = _library(), s["case"]
    op = case["op"]
    if op == "attn":
        packed = case["packed"]
        o, lse = lib.kda_attention_fwd(s["q"], s["k"], s["v"], s["cu_q"] if packed else None,
                                       s["cu_k"] if packed else None, n_seqs=case["seqs"],
                                       causal=case["causal"], scale=s["scale"],
                                       want_lse=case["lse"])
        return _attn_out(s, o, lse)
    if op == "kv4_attn":
        o, lse = lib.kda_kv4_attention(s["q"], s["cache"], s["table"], s["seq_lens"],
                                       scale=s["scale"], want_lse=case["lse"])
        return _attn_out(s, o, lse)
    cu = s["cu"] if case["packed"] else None
    if op == "kv4_write":
        lib.kda_kv4_write(s["k"], s["v"], s["cache"], s["table"], s["start"], cu,
                          n_seqs=case["seqs"])
    k, v = lib.kda_kv4_read(s["cache"], s["table"], case["total"], s["start"], cu,
                            n_seqs=case["seqs"])
    return {"k": k, "v": v}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------- the work
def _held(case):
    """Bytes of a token's keys and values in the cache."""
    return case["kv_heads"] * (case["d"] + 4 * case["d"] // GROUP)


def work(case):
    op, d, kv = case["op"], case["d"], case["kv_heads"]
    if op == "attn":
        q_lens, k_lens = _attn_lengths(case)
        if case["causal"]:
            pairs = sum(n * (2 * m - n + 1) // 2 for n, m in zip(q_lens, k_lens))
        else:
            pairs = sum(n * m for n, m in zip(q_lens, k_lens))
        rows = case["total"] * case["heads"]
        return {"bytes": 4 * d * (rows + sum(k_lens) * kv) + (4 * rows if case["lse"] else 0),
                "flops": 4 * d * case["heads"] * pairs}
    if op == "kv4_attn":
        lens, t = _cache_lengths(case), case["tokens"]
        rows = case["seqs"] * t * case["heads"]
        pairs = sum(t * n - t * (t - 1) // 2 for n in lens)
        return {"bytes": sum(lens) * _held(case) + 4 * d * rows + (4 * rows if case["lse"] else 0)
                + 4 * sum(-(-n // case["page"]) + 1 for n in lens),
                "flops": 4 * d * case["heads"] * pairs}
    tokens = case["total"]
    both = 2 if op == "kv4_write" else 1   # there and back
    return {"bytes": both * tokens * (_held(case) + 4 * d * kv),
            "flops": both * 4 * d * kv * tokens}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_softmax(q, k, v, scale, reach):
    """One head's queries [Q, d] over its keys, all in 64 bits: o and the logarithms."""
    x = scale * torch.einsum("qd,kd->qk", q, k)
    seen = torch.arange(k.shape[0], device=q.device)[None] < reach[:, None]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None])
    return torch.einsum("qk,kd->qd", p, v), lse


def _exact_attn(s):
    case = s["case"]
    group = case["heads"] // case["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        for h in range(case["heads"] if nk else 0):
            k, v = (s[name][k0:k0 + nk, h // group].double() for name in "kv")
            for a in range(0, nq, 2048):
                rows = torch.arange(a, min(a + 2048, nq), device="cuda")
                reach = rows + 1 + nk - nq if case["causal"] else torch.full_like(rows, nk)
                n = max(0, min(nk, int(reach[-1])))
                o[q0 + rows, h], lse[q0 + rows, h] = _exact_softmax(
                    s["q"][q0 + rows, h].double(), k[:n], v[:n], s["scale"], reach)
        q0, k0 = q0 + nq, k0 + nk
    return _attn_out(s, o, lse)


def _exact_code(x):
    """What x stands for once it has been through the cache, in 64 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[-1], GROUP):
        g = x[..., at:at + GROUP].double()
        s = torch.clamp(g.abs().max(-1, keepdim=True).values, min=AMAX_MIN) / 7
        s = s.to(torch.bfloat16).double()
        out[..., at:at + GROUP] = torch.round(g / s) * s
    return out


def _exact_row(codes, scales, keys):
    """Rows of codes [..., d / 2] and scales to values, group by group, in 64 bits."""
    groups = scales.shape[-1]
    run = 8 if keys else 4     # channels of a group that lie side by side
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    for c in range(out.shape[-1]):
        g, part, i = c // GROUP, c % GROUP // run, c % run
        nibble = (part * groups + g) * run + i
        n = (codes[..., nibble // 2] >> (4 * (nibble % 2))) & 15
        out[..., c] = (n.double() - 8.0) * scales[..., g].double()
    return out


def _exact_span(s, n, first, last):
    """Keys and values of positions [first, last) of sequence n: [tokens, heads, d]."""
    size = s["case"]["page"]
    position = torch.arange(first, last, device="cuda")
    pages = s["table"][n, torch.div(position, size, rounding_mode="floor")].long()
    kc, ks, vc, vs = (t[pages, :, position % size] for t in s["cache"])
    return _exact_row(kc, ks, True), _exact_row(vc, vs, False)


def _exact_write(s):
    return {"k": _exact_code(s["k"]), "v": _exact_code(s["v"])}


def _exact_read(s):
    parts = [_exact_span(s, n, a, a + length)
             for n, (a, length) in enumerate(zip(s["start"].tolist(), s["lens"])) if length]
    return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}


def _exact_kv4_attn(s):
    case = s["case"]
    tokens, group = case["tokens"], case["heads"] // case["kv_heads"]
    q = s["q"].double().reshape(case["seqs"], tokens, case["heads"], case["d"])
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    for n, length in enumerate(s["lens"]):
        k, v = _exact_span(s, n, 0, length)
        reach = length - tokens + 1 + torch.arange(tokens, device="cuda")
        for h in range(case["kv_heads"]):
            for i in range(h * group, (h + 1) * group):
                o[n, :, i], lse[n, :, i] = _exact_softmax(q[n, :, i], k[:, h], v[:, h], s["scale"],
                                                          reach)
    return _attn_out(s, o.view(s["q"].shape), lse.view(s["q"].shape[:-1]))


EXACT = {"attn": _exact_attn, "kv4_write": _exact_write, "kv4_read": _exact_read,
         "kv4_attn": _exact_kv4_attn}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
