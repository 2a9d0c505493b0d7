"""Long and shared contexts over a paged KV cache: four operators around the decode.

Each is computed in its plain form (elementary torch operations in 32 bits) or by the framework:

  scored   grouped-query attention of the last token (or the last few, causally) of each sequence whose scores are capped
           by a tanh and / or get a bias proportional to the distance between query and key, a slope per query head.
  weights  the same attention (scores as they are) that also adds the attention weight which every cached token got, summed
           over the query heads of its kv head and over the queries, to a running sum kept beside the cache.
  evict    a sequence's cache cut down to a budget: its first and its last tokens and, of those between, the ones with the
           largest sums stay, per kv head, in their order, at the front of the sequence's blocks (or of other blocks).
  shared   the attention of a batch whose sequences begin with the same blocks, in one or several groups.
"""
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # two short sequences of a model with distance biases: latency
        dict(name="scored_tiny", op="scored", fmt="bf16", b=2, hq=4, hkv=2, d=64, bs=16, lens="u", lo=37, hi=80, lens_seed=1,
             q_len=1, cap=0.0, alibi=True),
        # the 8B-style serving batch, scores capped
        dict(name="scored_8b", op="scored", fmt="bf16", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=4096, hi=4096,
             lens_seed=2, q_len=1, cap=50.0, alibi=False),
        # two drafted tokens per sequence over an 8-bit cache, wide heads, caps and biases
        dict(name="scored_draft_e4m3", op="scored", fmt="e4m3", b=16, hq=16, hkv=4, d=256, bs=16, lens="u", lo=1024, hi=8192,
             lens_seed=3, q_len=2, cap=30.0, alibi=True),
        # one decoding step of a small batch that keeps its sums
        dict(name="weights_1b", op="weights", fmt="bf16", b=8, hq=32, hkv=8, d=64, bs=16, lens="u", lo=512, hi=2048, lens_seed=4,
             q_len=1),
        # the 8B-style serving batch with its sums
        dict(name="weights_8b", op="weights", fmt="bf16", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=4096, hi=4096,
             lens_seed=5, q_len=1),
        # long contexts of very different lengths in 8 bits
        dict(name="weights_ragged_e4m3", op="weights", fmt="e4m3", b=64, hq=64, hkv=8, d=128, bs=32, lens="logu", lo=128,
             hi=32768, lens_seed=6, q_len=1),
        # a small batch cut to a few hundred tokens: latency
        dict(name="evict_small_e4m3", op="evict", fmt="e4m3", b=4, hq=16, hkv=4, d=128, bs=16, lens="u", lo=600, hi=1100, lens_seed=7,
             keep=512, first=4, recent=64, place="out"),
        # the 8B-style batch halved into other blocks
        dict(name="evict_8b", op="evict", fmt="bf16", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=4096, hi=4096, lens_seed=8,
             keep=2048, first=16, recent=256, place="out"),
        # ragged prompts written to the cache and cut down where they are
        dict(name="evict_prompts", op="evict", fmt="bf16", b=24, hq=32, hkv=8, d=128, bs=16, lens="logu", lo=17, hi=8192, lens_seed=9,
             keep=1000, first=4, recent=128, place="in"),
        # a chat batch behind one long system prompt
        dict(name="shared_8b", op="shared", fmt="bf16", b=32, hq=32, hkv=8, d=128, bs=16, lens="u", lo=20, hi=500, lens_seed=10,
             q_len=1, groups=1, prefix=32768, cap=0.0, alibi=False),
        # samples of eight prompts each, few heads and short texts: latency
        dict(name="shared_samples", op="shared", fmt="bf16", b=16, hq=8, hkv=2, d=64, bs=16, lens="u", lo=1, hi=64, lens_seed=11,
             q_len=1, groups=2, prefix=1000, cap=0.0, alibi=True),
        # many sequences of eight query heads per kv head behind one document, 8 bits, scores capped
        dict(name="shared_wide_e4m3", op="shared", fmt="e4m3", b=64, hq=64, hkv=8, d=128, bs=32, lens="u", lo=100, hi=1000, lens_seed=12,
             q_len=1, groups=1, prefix=16384, cap=50.0, alibi=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["scored", "weights", "evict", "shared", "shared"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(op=op, fmt=rng.choice(["bf16", "e4m3", "int8"]), hq=hq, hkv=hkv, d=d, bs=rng.choice([8, 16, 32, 64, 16, 32, 1, 4]),
             lens=rng.choice(["u", "logu"]), lens_seed=rng.randrange(1 << 30))
    q_len = rng.choice([1, 1, 1, 2, 4, 7]) if op != "evict" else 1
    prefix = _log(rng, 30, 20000) if op == "shared" else 0
    hi = _log(rng, 8, 1000 if op == "shared" else 20000)
    most = min(64, 200_000_000 // (hkv * d * q_len * (hi + prefix)))
    c.update(b=_log(rng, 1, max(1, most)), lo=rng.choice([1, max(1, hi // 2), hi]) if c["lens"] == "logu" else
             rng.choice([0, 1, hi // 2, hi]), hi=hi)
    if op == "evict":
        keep = _log(rng, 2, hi + 10)
        c.update(keep=keep, first=rng.choice([0, min(4, keep // 3)]), recent=rng.choice([0, 1, keep // 4, keep // 2]),
                 place=rng.choice(["out", "in"]) if c["fmt"] == "bf16" else "out")
        return c
    c["q_len"] = q_len
    if op != "weights":
        c.update(cap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.4)
    if op == "scored" and not c["cap"]:
        c["alibi"] = True
    if op == "shared":
        c.update(groups=rng.choice([1, 1, 2, 3]), prefix=prefix)
        c["groups"] = min(c["groups"], c["b"])
    return c


def _lens(case):
    """Tokens of each sequence (behind what it shares)."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["lo"], case["hi"]
    lens = [r.randint(lo, hi) if case["lens"] == "u" else _log(r, lo, hi) for _ in range(case["b"])]
    return [max(1, lens[0])] + lens[1:]


def _groups(case):
    """Where each group's sequences start, and how many blocks they share."""
    r = random.Random(case["lens_seed"] + 1)
    g, b = case["groups"], case["b"]
    starts = [0] + sorted(r.sample(range(1, b), g - 1)) + [b]
    return starts, [max(1, (case["prefix"] if i == 0 else r.randint(1, case["prefix"])) // case["bs"]) for i in range(g)]


def _totals(case):
    """All tokens of each sequence."""
    lens = _lens(case)
    if case["op"] != "shared":
        return lens
    starts, shared = _groups(case)
    return [lens[i] + shared[g] * case["bs"] for g in range(case["groups"]) for i in range(starts[g], starts[g + 1])]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = 4 * d if case["fmt"] == "bf16" else 2 * (d + 4)  # a token's key and value, one kv head
    lens = _totals(case)
    if case["op"] == "evict":
        moved = sum(min(n, case["keep"]) for n in lens) * hkv
        written = sum(lens) * hkv * 2 * row if case["place"] == "in" else 0
        return {"bytes": 4 * sum(lens) * hkv + moved * (2 * row + 8) + written, "flops": sum(lens) * hkv}
    total = stored = sum(lens)
    if case["op"] == "shared":
        starts, shared = _groups(case)
        stored -= sum(s * case["bs"] * (b - a - 1) for s, a, b in zip(shared, starts, starts[1:]))
    out = {"bytes": stored * hkv * row + 4 * case["b"] * case["q_len"] * hq * d, "flops": 4 * total * case["q_len"] * hq * d}
    if case["op"] == "weights":
        out["bytes"] += 8 * total * hkv
    return out


# ------------------------------------------------------------------ inputs

def _codes(x, fmt):
    """Codes and scales of rows (the last axis), in 32 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    y = x * (QMAX[fmt] / amax)
    return y.to(TYPES[fmt]) if fmt == "e4m3" else y.round().clamp(-127, 127).to(torch.int8), (amax / QMAX[fmt])[..., 0]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d, b, bs, fmt, op = (case[k] for k in ("hq", "hkv", "d", "b", "bs", "fmt", "op"))
    lens = _totals(case)
    blocks = [-(-n // bs) for n in lens]
    width = max(1, *blocks)
    s = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    table = torch.zeros((b, width), dtype=torch.int64, device="cuda")
    used = torch.arange(width, device="cuda")[None] < torch.tensor(blocks, device="cuda")[:, None]
    if op == "shared":
        starts, shared = _groups(case)
        firsts = torch.zeros((b, width), dtype=torch.int64, device="cuda")
        apart, many = used.clone(), 0
        for a, e, n in zip(starts, starts[1:], shared):
            apart[a:e, :n] = False
            firsts[a:e, :n] = torch.arange(many, many + n, device="cuda")
            many += n
        need = many + int(apart.sum())
        pool = need + 3
        order = torch.randperm(pool, generator=g, device="cuda")
        table = torch.where(used & ~apart, order[firsts], table)
        table[apart] = order[many:need]
        s["shared"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    else:
        kept = -(-case["keep"] // bs) if op == "evict" else 0
        need = sum(blocks)
        pool = need + 3 + b * kept
        order = torch.randperm(pool, generator=g, device="cuda")
        table[used] = order[:need]
        if op == "evict":
            s["out_table"] = order[need:need + b * kept].view(b, kept).int() if case["place"] == "out" else None
    s["table"] = table.int()
    pools = [torch.randn((pool, bs, hkv, d), generator=g, device="cuda").mul_(1.0 if i else 1.5) for i in range(2)]
    s["scales"] = None if fmt == "bf16" else torch.empty((pool, hkv, 2, bs), device="cuda")
    for i, name in enumerate(("k_pool", "v_pool")):
        if fmt == "bf16":
            s[name] = pools[i].bfloat16()
        else:
            s[name], sc = _codes(pools[i], fmt)
            s["scales"][:, :, i] = sc.transpose(1, 2)
    del pools
    if op == "evict":
        # sums over many steps: a few tokens hold most of the weight, some none, some the same
        w = torch.randn((pool, hkv, bs), generator=g, device="cuda").mul_(1.5).exp_()
        even = torch.rand((pool, hkv, bs), generator=g, device="cuda")
        s["weights0"] = torch.where(even < 0.1, torch.floor(4 * w) / 4, w)
        s["weights"] = s["weights0"].clone()
        if case["place"] == "in":
            s["new_starts"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
            for name, scale in (("k", 1.5), ("v", 1.0)):
                s[name] = torch.randn((sum(lens), hkv, d), generator=g, device="cuda").mul_(scale).bfloat16()
        return s
    s["q"] = torch.randn((b, case["q_len"], hq, d), generator=g, device="cuda").bfloat16()
    if op == "weights":
        s["weights0"] = torch.rand((pool, hkv, bs), generator=g, device="cuda")
        s["weights"] = s["weights0"].clone()
    # the usual slopes of distance biases, a geometric sequence over the heads
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if case.get("alibi") else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_gqa_decode_05_gb300 as pda
        c = case
        ctx = s["ctx"] = pda.Context(max_seqs=c["b"] * c.get("q_len", 1), num_q_heads=c["hq"], num_kv_heads=c["hkv"],
                                     head_dim=c["d"], block_size=c["bs"])
        cache = (s["k_pool"], s["v_pool"])
        if c["op"] == "evict":
            s["kept"] = torch.empty((c["b"], c["hkv"], c["keep"]), dtype=torch.int32, device="cuda")
            s["new_lens"] = torch.empty_like(s["lens"])
            if c["place"] == "in":
                s["write"] = ctx.bind_append(s["k"], s["v"], *cache, s["table"], s["lens"], starts=s["new_starts"])
            s["call"] = ctx.bind_evict(*cache, s["weights"], s["table"], s["lens"], c["keep"], first=c["first"],
                                       recent=c["recent"], scales=s["scales"], out_table=s["out_table"], kept=s["kept"],
                                       new_lens=s["new_lens"])
            return s
        s["out"] = torch.empty_like(s["q"])
        single = c["q_len"] == 1
        q, out = (t[:, 0] if single else t for t in (s["q"], s["out"]))
        if c["op"] == "shared":
            s["call"] = ctx.bind_decode_shared(q, *cache, s["table"], s["lens"], s["shared"], out, starts=s["starts"],
                                               scales=s["scales"], softcap=c["cap"], alibi_slopes=s["slopes"])
        elif c["op"] == "scored":
            s["call"] = ctx.bind_decode_scored(q, *cache, s["table"], s["lens"], out, scales=s["scales"], softcap=c["cap"],
                                               alibi_slopes=s["slopes"])
        else:
            s["call"] = ctx.bind_decode_scored(q, *cache, s["table"], s["lens"], out, scales=s["scales"],
                                               weights=s["weights"], weights_from=s["weights0"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "evict":
        if s["case"]["place"] == "in":
            s["weights"].copy_(s["weights0"])  # the sums of this prompt's last queries
            if own:
                s["write"]()
            else:
                _write(s)
        if own:
            s["call"]()
            kept, lens = s["kept"], s["new_lens"]
        else:
            kept, lens = _evict(s)
        out = {"kept": kept, "lens": lens, "k_pool": s["k_pool"], "v_pool": s["v_pool"], "weights": s["weights"]}
        return out if s["scales"] is None else dict(out, scales=s["scales"])
    if own:
        s["call"]()
        out = s["out"]
    else:
        out = _attend(s)
    return {"out": out, "weights": s["weights"]} if op == "weights" else out


def _gathered(s, which, block, slot):
    pool = s[("k_pool", "v_pool")[which]]
    if s["scales"] is None:
        return pool[block, slot].float()
    return pool.view(torch.int8)[block, slot].view(pool.dtype).float() * s["scales"][block, :, which, slot][..., None]


def _attend(s):
    case = s["case"]
    b, n, hq, hkv, d, bs = (case[k] for k in ("b", "q_len", "hq", "hkv", "d", "bs"))
    t = torch.arange(s["table"].shape[1] * bs, device="cuda")
    block, slot = s["table"].long()[:, t // bs], (t % bs).expand(b, -1)
    lens = s["lens"].long()
    last = lens[:, None] - n + torch.arange(n, device="cuda")  # each query's own token, the last one that it sees
    q = s["q"].float().view(b, n, hkv, -1, d)
    x = torch.einsum("bnhgd,bthd->bhngt", q, _gathered(s, 0, block, slot)) * d ** -0.5
    if case.get("cap"):
        x = case["cap"] * torch.tanh(x / case["cap"])
    if case.get("alibi"):
        far = (t - last[..., None]).float()[:, None, :, None]
        x = x + s["slopes"].view(hkv, 1, -1, 1) * far
    x = x.masked_fill((t > last[..., None])[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    if case["op"] == "weights":
        got = p.sum((2, 3)).transpose(1, 2)  # [b, t, hkv]
        seen = t < lens[:, None]
        old = s["weights0"][block, :, slot]
        new = torch.where((t >= lens[:, None] - n)[..., None], 0.0, old) + got  # the queries' own tokens are new
        s["weights"][block[seen], :, slot[seen]] = new[seen]
    return torch.einsum("bhngt,bthd->bnhgd", p, _gathered(s, 1, block, slot)).reshape(b, n, hq, d).bfloat16()


def _write(s):
    starts, lens, bs = s["new_starts"].long(), s["lens"].long(), s["case"]["bs"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    at = lens[b] - starts[b + 1] + t
    block, slot = s["table"].long()[b, at // bs], at % bs
    s["k_pool"][block, slot] = s["k"]
    s["v_pool"][block, slot] = s["v"]


def _evict(s):
    case = s["case"]
    hkv, bs, keep, first, recent = (case[k] for k in ("hkv", "bs", "keep", "first", "recent"))
    lens = s["lens"].long()
    t = torch.arange(s["table"].shape[1] * bs, device="cuda")
    block, slot = s["table"].long()[:, t // bs], (t % bs).expand(len(lens), -1)
    w = s["weights"][block, :, slot].transpose(1, 2)  # [b, hkv, t]
    n = lens[:, None, None]
    w = torch.where((t < first) | (t >= n - recent), float("inf"), w)
    w = torch.where(t < n, w, -float("inf"))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order))
    stays = (t < n) & (rank < keep)
    # the kept tokens in their order
    kept = torch.sort(torch.where(stays, t, t.numel()), dim=-1).values[..., :keep]
    kept = torch.cat([kept, kept.new_full((*kept.shape[:2], keep - kept.shape[-1]), t.numel())], -1)
    kept = torch.where(kept < t.numel(), kept, -1)
    b, h, i = (kept >= 0).nonzero(as_tuple=True)
    at = kept[b, h, i]
    to = s["table"] if s["out_table"] is None else s["out_table"]
    old, new = (s["table"].long()[b, at // bs], at % bs), (to.long()[b, i // bs], i % bs)
    for name in ("k_pool", "v_pool"):
        pool = s[name].view(torch.int8) if s[name].element_size() == 1 else s[name]
        pool[new[0], new[1], h] = pool[old[0], old[1], h]
    s["weights"][new[0], h, new[1]] = s["weights"][old[0], h, old[1]]
    if s["scales"] is not None:
        s["scales"][new[0], h, :, new[1]] = s["scales"][old[0], h, :, old[1]]
    return kept.int(), lens.clamp(max=keep).int()


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_evict(s) if case["op"] == "evict" else _exact_attend(s)


def _exact_rows(s, i, n):
    """Sequence i's keys and values, [tokens, kv heads, D]."""
    blocks = s["table"][i, :-(-n // s["case"]["bs"])].long()
    got = []
    for which, name in enumerate(("k_pool", "v_pool")):
        x = s[name].view(torch.uint8)[blocks].view(s[name].dtype).double()
        if s["scales"] is not None:
            x = x * s["scales"][blocks, :, which].double().transpose(1, 2)[..., None]
        got.append(x.flatten(0, 1)[:n])
    return got


def _exact_attend(s):
    case = s["case"]
    m, hq, hkv, d, bs = (case[k] for k in ("q_len", "hq", "hkv", "d", "bs"))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights0"].double() if case["op"] == "weights" else None
    for i, n in enumerate(_totals(case)):
        if n == 0:
            continue
        k, v = _exact_rows(s, i, n)
        sums = torch.zeros((n, hkv), dtype=torch.float64, device="cuda")
        for j in range(m):
            seen = n - m + j + 1
            if seen <= 0:
                continue
            q = s["q"][i, j].double().reshape(hkv, hq // hkv, d)
            x = q @ k[:seen].permute(1, 2, 0) / d ** 0.5  # [hkv, group, seen]
            if case.get("cap"):
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if case.get("alibi"):
                back = torch.arange(seen - 1, -1, -1, dtype=torch.float64, device="cuda")
                x = x - s["slopes"].double().view(hkv, -1, 1) * back
            p = torch.softmax(x, -1)
            out[i, j] = (p @ v[:seen].transpose(0, 1)).reshape(hq, d)
            sums[:seen] += p.sum(1).T
        if weights is not None:
            at = torch.arange(n, device="cuda")
            block, slot = s["table"][i].long()[at // bs], at % bs
            fresh = at >= n - m
            weights[block[fresh], :, slot[fresh]] = 0.0
            weights[block, :, slot] += sums
    return out if weights is None else {"out": out, "weights": weights}


def _exact_evict(s):
    case = s["case"]
    b, hkv, bs, keep, first, recent = (case[k] for k in ("b", "hkv", "bs", "keep", "first", "recent"))
    lens = _totals(case)
    table = s["table"].tolist()
    out_table = table if s["out_table"] is None else s["out_table"].tolist()
    pools = [s[name].view(torch.uint8).view(s[name].dtype).to(torch.int64 if case["fmt"] == "int8" else torch.float64)
             for name in ("k_pool", "v_pool")]
    weights = s["weights0"].double()
    scales = None if s["scales"] is None else s["scales"].double()
    kept = torch.full((b, hkv, keep), -1, dtype=torch.int64)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        at = torch.arange(n)
        src = torch.tensor(table[i])[at // bs].cuda(), (at % bs).cuda()
        if case["place"] == "in":
            a = sum(lens[:i])
            pools[0][src], pools[1][src] = s["k"][a:a + n].double(), s["v"][a:a + n].double()
        w = weights[src[0], :, src[1]].T.cpu().tolist()  # [hkv][n]
        rows = [p[src] for p in pools]
        sums = weights[src[0], :, src[1]]
        sc = None if scales is None else scales[src[0], :, :, src[1]]
        for h in range(hkv):
            always = [t for t in range(n) if t < first or t >= n - recent] if n > keep else list(range(n))
            chosen = set(always)
            between = sorted((t for t in range(n) if t not in chosen), key=lambda t: (-w[h][t], t))
            stay = sorted(always + between[:max(0, keep - len(always))])
            kept[i, h, :len(stay)] = torch.tensor(stay)
            j = torch.arange(len(stay))
            stay = torch.tensor(stay).cuda()
            dst = torch.tensor(out_table[i])[j // bs].cuda(), (j % bs).cuda()
            for p, r in zip(pools, rows):
                p[dst[0], dst[1], h] = r[stay, h]
            weights[dst[0], h, dst[1]] = sums[stay, h]
            if sc is not None:
                scales[dst[0], h, :, dst[1]] = sc[stay, h]
    out = {"kept": kept, "lens": torch.tensor([min(n, keep) for n in lens]), "k_pool": pools[0], "v_pool": pools[1],
           "weights": weights}
    return out if scales is None else dict(out, scales=scales)
