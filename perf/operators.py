"""What one attention layer of a serving step does around a quantised paged KV cache.

Four operators, each computed in its plain form (elementary torch operations in 32 bits) or by the framework:

  norm_rope  RMS norm of every query and key head and its position rotation.
  append     the same on the way into the cache: queries out, keys and values of the new tokens quantised to 8 bits
             with one scale per token and kv head and written to their blocks.
  read       a sequence's cached tokens gathered from their blocks and dequantised, packed one sequence after another.
  decode     grouped-query attention of the last token (or the last few, causally) of each sequence over that cache.
"""
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
TYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TINY = 2.0 ** -100  # rows whose largest magnitude is below this are stored as zeros
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a 32-sequence batch: the smallest launch, latency counts
        dict(name="norm_rope_step", op="norm_rope", tokens=32, hq=32, hkv=8, d=128, rotary=128, interleaved=False),
        # a long prompt, an odd number of tokens, half of each head rotated, neighbouring columns paired
        dict(name="norm_rope_prompt", op="norm_rope", tokens=8191, hq=64, hkv=8, d=128, rotary=64, interleaved=True),
        # one decoding step: one new token per sequence enters the cache
        dict(name="append_step", op="append", fmt="e4m3", b=32, hq=32, hkv=8, d=128, bs=16, new=1, lens="u", lo=16, hi=96,
             lens_seed=1, rotary=128, interleaved=False, read=False),
        # ragged prompts of a prefill batch
        dict(name="append_prompts", op="append", fmt="e4m3", b=24, hq=32, hkv=8, d=128, bs=16, new=0, lens="logu", lo=17,
             hi=4096, lens_seed=2, rotary=128, interleaved=False, read=False),
        # drafted tokens of a speculative step with wide heads, written and read back
        dict(name="append_draft_int8", op="append", fmt="int8", b=16, hq=16, hkv=4, d=256, bs=16, new=4, lens="u", lo=4,
             hi=300, lens_seed=3, rotary=128, interleaved=False, read=True),
        # the cached prefixes of a small batch, read back for another kernel
        dict(name="read_1b", op="read", fmt="e4m3", b=8, hq=32, hkv=8, d=64, bs=16, lens="u", lo=512, hi=2048, lens_seed=4),
        # a whole long-context batch moved out of the cache
        dict(name="read_ragged_int8", op="read", fmt="int8", b=64, hq=64, hkv=8, d=128, bs=32, lens="logu", lo=128, hi=32768,
             lens_seed=5),
        # two short sequences: latency
        dict(name="decode_tiny", op="decode", fmt="e4m3", b=2, hq=4, hkv=2, d=64, bs=16, lens="u", lo=37, hi=80, lens_seed=6,
             q_len=1),
        # the 8B-style serving batch
        dict(name="decode_8b", op="decode", fmt="e4m3", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=4096, hi=4096,
             lens_seed=7, q_len=1),
        # wide heads, ragged lengths
        dict(name="decode_wide_int8", op="decode", fmt="int8", b=16, hq=16, hkv=4, d=256, bs=16, lens="u", lo=1024, hi=8192,
             lens_seed=8, q_len=1),
        # long contexts of very different lengths, eight query heads per kv head
        dict(name="decode_ragged", op="decode", fmt="e4m3", b=64, hq=64, hkv=8, d=128, bs=32, lens="logu", lo=128, hi=32768,
             lens_seed=9, q_len=1),
        # four drafted tokens per sequence checked at once
        dict(name="decode_draft", op="decode", fmt="e4m3", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=1000, hi=4096,
             lens_seed=10, q_len=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read", "decode", "decode"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(op=op, hq=hq, hkv=hkv, d=d)
    rotary = rng.choice([d, d, d // 2])
    if op == "norm_rope":
        return dict(c, tokens=_log(rng, 1, min(8191, 75_000_000 // ((hq + hkv) * d))), rotary=rotary, interleaved=rng.random() < 0.5)
    c.update(fmt=rng.choice(["e4m3", "int8"]), bs=rng.choice([8, 16, 32, 64, 16, 32, 1, 4]), lens_seed=rng.randrange(1 << 30))
    if op == "append":
        new = rng.choice([0, 1, 1, 2, 5])
        c.update(b=_log(rng, 1, 64), new=new, lens="logu", lo=1, hi=_log(rng, 8, 1024), rotary=rotary,
                 interleaved=rng.random() < 0.5, read=c["fmt"] == "int8")
        return c
    hi = _log(rng, 16, 32768)
    q_len = rng.choice([1, 1, 1, 2, 4, 7]) if op == "decode" else 1
    most = min(64, 300_000_000 // (hkv * d * q_len * hi))
    c.update(b=_log(rng, 1, max(1, most)), lens=rng.choice(["u", "logu"]), lo=rng.choice([0, 1, hi // 2, hi]), hi=hi)
    if c["lens"] == "logu":
        c["lo"] = max(1, c["lo"])
    if op == "decode":
        c["q_len"] = q_len
    return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    lo, hi = case["lo"], case["hi"]
    lens = [r.randint(lo, hi) if case["lens"] == "u" else _log(r, lo, hi) for _ in range(case["b"])]
    return [max(1, lens[0])] + lens[1:]


def _news(case, lens):
    """New tokens per sequence of an append: `new`, or whole prompts where that is 0."""
    return [min(n, case["new"]) if case["new"] else n for n in lens]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "norm_rope":
        n = case["tokens"]
        return {"bytes": n * (2 * (hq + hkv) * d * 2 + 4), "flops": 10 * n * (hq + hkv) * d}
    lens = _lens(case)
    total = sum(lens)
    kv = 2 * hkv * (d + 4)  # one token's codes and scales
    if case["op"] == "append":
        n = sum(_news(case, lens))
        return {"bytes": n * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + kv) + (total * (kv + 4 * hkv * d) if case["read"] else 0),
                "flops": 14 * n * (hq + 2 * hkv) * d}
    if case["op"] == "read":
        return {"bytes": total * (kv + 4 * hkv * d), "flops": 2 * total * hkv * d}
    return {"bytes": total * kv + 4 * case["b"] * case["q_len"] * hq * d, "flops": 4 * total * case["q_len"] * hq * d}


# ------------------------------------------------------------------ inputs

def _rope_table(n, rotary):
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 1e4 ** (
        -torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _codes(x, fmt):
    """Codes and scales of rows (the last axis), in 32 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    keep = amax >= TINY
    y = torch.where(keep, x * (QMAX[fmt] / amax), 0.0)
    codes = y.to(TYPES[fmt]) if fmt == "e4m3" else y.round().clamp(-127, 127).to(torch.int8)
    return codes, torch.where(keep, amax / QMAX[fmt], 0.0)[..., 0]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    def heads(tokens):
        # the projections' output, one row per token: queries, keys and values side by side
        qkv = normal(tokens, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"], s["k_weight"] = ((1 + 0.1 * normal(d).float()).bfloat16() for _ in range(2))

    if case["op"] == "norm_rope":
        heads(case["tokens"])
        s["cos_sin"] = _rope_table(16384, case["rotary"])
        s["positions"] = torch.randint(0, 16384, (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        return s
    b, bs, fmt = case["b"], case["bs"], case["fmt"]
    lens = _lens(case)
    blocks = [-(-n // bs) for n in lens]
    width, pool = max(1, *blocks), sum(blocks) + 3
    order = torch.randperm(pool, generator=g, device="cuda")
    table = torch.zeros((b, width), dtype=torch.int64, device="cuda")
    used = torch.arange(width, device="cuda")[None] < torch.tensor(blocks, device="cuda")[:, None]
    table[used] = order[:sum(blocks)]
    s["table"] = table.int()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    s["total"] = sum(lens)
    s["scales"] = torch.empty((pool, hkv, 2, bs), device="cuda")
    for i, name in enumerate(("k_pool", "v_pool")):
        s[name], sc = _codes(torch.randn((pool, bs, hkv, d), generator=g, device="cuda").mul_(1.0 if i else 1.5), fmt)
        s["scales"][:, :, i] = sc.transpose(1, 2)
    if case["op"] == "append":
        news = _news(case, lens)
        heads(sum(news))
        s["new_starts"] = torch.tensor([sum(news[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
        s["cos_sin"] = _rope_table(max(1, *lens), case["rotary"])
    if case["op"] == "decode":
        s["q"] = normal(b, case["q_len"], hq, d)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_gqa_decode_05_gb300 as pda
        c = case
        ctx = s["ctx"] = pda.Context(max_seqs=max(1, c.get("b", 1) * c.get("q_len", 1)), num_q_heads=c["hq"],
                                     num_kv_heads=c["hkv"], head_dim=c["d"], block_size=c.get("bs", 16))
        if c["op"] in ("norm_rope", "append"):
            s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
            prep = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, cos_sin=s["cos_sin"],
                        interleaved=c["interleaved"])
        if c["op"] == "norm_rope":
            s["k_out"] = torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda")
            s["call"] = ctx.bind_norm_rope(s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"], **prep)
        if c["op"] == "append":
            s["call"] = ctx.bind_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["lens"], scales=s["scales"],
                                        starts=s["new_starts"], q=s["q"], q_out=s["q_out"], **prep)
        if c["op"] == "read" or c.get("read"):
            s["k_out"], s["v_out"] = (torch.empty((s["total"], c["hkv"], c["d"]), dtype=torch.bfloat16, device="cuda")
                                      for _ in range(2))
        if c["op"] == "decode":
            s["out"] = torch.empty_like(s["q"])
            if c["q_len"] == 1:
                s["call"] = ctx.bind_decode(s["q"][:, 0], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["out"][:, 0],
                                            scales=s["scales"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "norm_rope":
            s["call"]()
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append":
            s["call"]()
            if not case["read"]:
                return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"], "scales": s["scales"]}
        if op == "decode":
            if case["q_len"] == 1:
                s["call"]()
            else:
                s["ctx"].decode_multi(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], scales=s["scales"], out=s["out"])
            return s["out"]
        s["ctx"].read_cache(s["k_pool"], s["v_pool"], s["table"], s["lens"], scales=s["scales"], starts=s["starts"],
                            k_out=s["k_out"], v_out=s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]} if op == "append" else {"k": s["k_out"], "v": s["v_out"]}
    if op == "norm_rope":
        cs = s["cos_sin"][s["positions"].long()][:, None]
        return {"q": _prepared(s["q"], s["q_weight"], cs, case).bfloat16(), "k": _prepared(s["k"], s["k_weight"], cs, case).bfloat16()}
    if op == "append":
        return _append(s)
    if op == "read":
        k, v = _read(s)
        return {"k": k, "v": v}
    return _decode(s)


def _prepared(x, w, cs, case):
    """Norm and rotation in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    r = case["rotary"]
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _new_tokens(s):
    """Position, block and slot in the block of every new token."""
    starts, lens, bs = s["new_starts"].long(), s["lens"].long(), s["case"]["bs"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    at = lens[b] - starts[b + 1] + t
    return at, s["table"].long()[b, at // bs], at % bs


def _append(s):
    case = s["case"]
    at, block, slot = _new_tokens(s)
    cs = s["cos_sin"][at][:, None]
    q = _prepared(s["q"], s["q_weight"], cs, case).bfloat16()
    k, ks = _codes(_prepared(s["k"], s["k_weight"], cs, case), case["fmt"])
    v, vs = _codes(s["v"].float(), case["fmt"])
    s["k_pool"].view(torch.int8)[block, slot] = k.view(torch.int8)
    s["v_pool"].view(torch.int8)[block, slot] = v.view(torch.int8)
    s["scales"][block, :, 0, slot] = ks
    s["scales"][block, :, 1, slot] = vs
    if case["read"]:
        k, v = _read(s)
        return {"q": q, "k": k, "v": v}
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"], "scales": s["scales"]}


def _gathered(s, which, block, slot):
    pool = s[("k_pool", "v_pool")[which]]
    rows = pool.view(torch.int8)[block, slot].view(pool.dtype).float()
    return rows * s["scales"][block, :, which, slot][..., None]


def _read(s):
    starts, bs = s["starts"].long(), s["case"]["bs"]
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    at = t - starts[b]
    block, slot = s["table"].long()[b, at // bs], at % bs
    return _gathered(s, 0, block, slot).bfloat16(), _gathered(s, 1, block, slot).bfloat16()


def _decode(s):
    case = s["case"]
    b, n, hkv, d, bs = case["b"], case["q_len"], case["hkv"], case["d"], case["bs"]
    t = torch.arange(s["table"].shape[1] * bs, device="cuda")
    block, slot = s["table"].long()[:, t // bs], (t % bs).expand(b, -1)
    last = s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")  # the last token that each query sees
    q = s["q"].float().view(b, n, hkv, -1, d)
    scores = torch.einsum("bnhgd,bthd->bhngt", q, _gathered(s, 0, block, slot)) * d ** -0.5
    scores = scores.masked_fill((t > last[..., None])[:, None, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    return torch.einsum("bhngt,bthd->bnhgd", p, _gathered(s, 1, block, slot)).reshape(b, n, -1, d).bfloat16()


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm_rope":
        turn = _turns(s["positions"], case["rotary"], s["cos_sin"])
        return {"q": _exact_heads(s["q"], s["q_weight"], turn, case), "k": _exact_heads(s["k"], s["k_weight"], turn, case)}
    if op == "read":
        k, v = zip(*[_exact_rows(s, i) for i in range(case["b"])])
        return {"k": torch.cat(k), "v": torch.cat(v)}
    if op == "append":
        return _exact_append(s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hkv"]
    for i, n in enumerate(_lens(case)):
        k, v = _exact_rows(s, i)
        for j in range(case["q_len"]):
            m = n - case["q_len"] + j + 1
            if m > 0:
                q = s["q"][i, j].double().reshape(case["hkv"], group, case["d"])
                p = torch.softmax(q @ k[:m].permute(1, 2, 0) / case["d"] ** 0.5, -1)
                out[i, j] = (p @ v[:m].transpose(0, 1)).reshape(case["hq"], case["d"])
    return out


def _turns(positions, rotary, table):
    """The rotations as complex numbers: what the table, an input, holds."""
    row = table.double()[positions.long()]
    return torch.complex(row[:, :rotary // 2], row[:, rotary // 2:])[:, None]


def _exact_heads(x, w, turn, case):
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    r = case["rotary"]
    head = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
    z = torch.view_as_complex((head if case["interleaved"] else head.transpose(-1, -2)).contiguous()) * turn
    z = torch.view_as_real(z)
    x[..., :r] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return x


def _exact_rows(s, i):
    """Sequence i's keys and values, [tokens, kv heads, D]."""
    case = s["case"]
    n, bs = int(s["lens"][i]), case["bs"]
    blocks = s["table"][i, :-(-n // bs)].long()
    got = []
    for which, name in enumerate(("k_pool", "v_pool")):
        codes = s[name].view(torch.uint8)[blocks].view(s[name].dtype).double()
        scales = s["scales"][blocks, :, which].double().transpose(1, 2)[..., None]
        got.append((codes * scales).flatten(0, 1)[:n])
    return got


def _exact_codes(x, fmt):
    """The numbers that the nearest codes stand for (ties to even) over their scales, and the scales."""
    top = x.abs().amax(-1, keepdim=True)
    y = x / top * QMAX[fmt]
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp(min=-5) - 4) if fmt == "e4m3" else torch.ones_like(y)
    return (y / step).round() * step, (top / QMAX[fmt])[..., 0]


def _exact_append(s):
    case = s["case"]
    bs, fmt = case["bs"], case["fmt"]
    lens, starts = s["lens"].tolist(), s["new_starts"].tolist()
    pools = [s[name].double() for name in ("k_pool", "v_pool")]
    scales = s["scales"].double()
    at = torch.cat([torch.arange(n - (e - a), n) for n, a, e in zip(lens, starts, starts[1:])]).cuda()
    of = torch.cat([torch.full((e - a,), i) for i, (a, e) in enumerate(zip(starts, starts[1:]))]).cuda()
    turn = _turns(at, case["rotary"], s["cos_sin"])
    where = (s["table"][of, at // bs].long(), at % bs)
    for i, x in enumerate((_exact_heads(s["k"], s["k_weight"], turn, case), s["v"].double())):
        pools[i][where], scales[where[0], :, i, where[1]] = _exact_codes(x, fmt)
    q = _exact_heads(s["q"], s["q_weight"], turn, case)
    if not case["read"]:
        return {"q": q, "k_pool": pools[0], "v_pool": pools[1], "scales": scales}
    rows = []
    for i in range(2):
        full = pools[i] * scales[:, :, i].transpose(1, 2)[..., None]
        rows.append(torch.cat([full[s["table"][j].long()].flatten(0, 1)[:n] for j, n in enumerate(lens)]))
    return {"q": q, "k": rows[0], "v": rows[1]}
