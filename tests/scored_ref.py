"""fp64 definitions of scored decode, of the sums of attention weights and of eviction, and inputs for their tests."""
from __future__ import annotations

import numpy as np
import torch

import cache_ref as ref

FORMATS = [torch.bfloat16, torch.float8_e4m3fn, torch.int8]


def random_cache(g, num_blocks, bs, hkv, d, dtype):
    """(k_pool, v_pool, scales) of normal values on the CPU, scales None for bfloat16."""
    if dtype is torch.bfloat16:
        return (*(torch.randn((num_blocks, bs, hkv, d), generator=g).bfloat16() for _ in range(2)), None)
    return ref.random_cache(g, num_blocks, bs, hkv, d, dtype)


def scored64(q, k_pool, v_pool, scales, table, lens, bs, scale=None, softcap=0.0, slopes=None):
    """(out, size, sums) of causal decode, q [B, n, Hq, D]: fp64 attention, for each element sum p |v| (and for 8-bit
    pools what fp16 weights flush, see cache_ref.decode64), and per sequence the attention weights [tokens, Hkv]."""
    B, n, hq, d = q.shape
    hkv = k_pool.shape[2]
    G = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros_like(out)
    sums = []
    for b in range(B):
        L = max(int(lens[b]), 0)
        k, v = (ref.rows64(p, scales, i, table[b], L, bs) for i, p in enumerate((k_pool, v_pool)))
        vs = torch.ones(v.shape[:2], dtype=torch.float64) if scales is None else \
            scales[table[b].long(), :, 1].double().transpose(1, 2).flatten(0, 1)[:L]
        code = v.abs() / torch.where(vs == 0, 1.0, vs)[..., None]
        got = torch.zeros((L, hkv), dtype=torch.float64)
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                continue
            s = scale * q[b, i].double().reshape(hkv, G, d) @ k[:m].permute(1, 2, 0)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s + slopes.double().view(hkv, G, 1) * torch.arange(1 - m, 1, dtype=torch.float64)
            p = torch.softmax(s, -1)
            out[b, i] = (p @ v[:m].transpose(0, 1)).reshape(hq, d)
            flushed = 0.0
            if scales is not None:
                top = (p * vs[:m].T[:, None]).amax(-1, keepdim=True)
                flushed = 2.0 ** -21 * top * code[:m].sum(0)[:, None]
            size[b, i] = (p @ v[:m].abs().transpose(0, 1) + flushed).reshape(hq, d)
            got[:m] += p.sum(1).T
        sums.append(got)
    return out, size, sums


def add_sums(weights, sums, table, lens, bs, n):
    """(weights, size): the sums [num_blocks, Hkv, bs] after a decode of n queries each, and what they add; -1 where no
    token is."""
    w = weights.double().clone()
    size = torch.full_like(w, -1.0)
    for b, got in enumerate(sums):
        L = got.shape[0]
        t = torch.arange(L)
        block, slot = table[b].long()[t // bs], t % bs
        old = torch.where((t < L - n)[:, None], weights.double()[block, :, slot], 0.0)
        w[block, :, slot] = old + got
        size[block, :, slot] = got
    return w, size


def evict64(weights, table, lens, bs, keep, first, recent):
    """The kept tokens' former indices, per sequence and kv head."""
    kept = []
    for b, n in enumerate(lens):
        n = max(int(n), 0)
        t = np.arange(n)
        w = weights[table[b].long()[t // bs], :, t % bs].numpy() if n else np.zeros((0, weights.shape[1]))
        heads = []
        for h in range(weights.shape[1]):
            if n <= keep:
                heads.append(list(range(n)))
                continue
            always = [i for i in range(n) if i < first or i >= n - recent]
            rest = [i for i in range(first, n - recent)]
            rest.sort(key=lambda i: (0 if np.isnan(w[i, h]) else 1, 0.0 if np.isnan(w[i, h]) else -float(w[i, h]), i))
            heads.append(sorted(always + rest[:keep - len(always)]))
        kept.append(heads)
    return kept


def shared_table(rng, own, bs, starts, shared, spare=3):
    """(table, lens, pool): sequences of group g begin with the same shared[g] blocks and have own[b] tokens after them."""
    B = len(own)
    group = np.searchsorted(np.asarray(starts), np.arange(B), side="right") - 1
    blocks = [-(-n // bs) for n in own]
    width = max(1, max(shared[g] + nb for g, nb in zip(group, blocks)))
    pool = sum(shared) + sum(blocks) + spare
    order = iter(rng.permutation(pool).astype(np.int32))
    prefixes = [[next(order) for _ in range(n)] for n in shared]
    table = np.full((B, width), pool - 1, dtype=np.int32)
    lens = []
    for b in range(B):
        ids = prefixes[group[b]] + [next(order) for _ in range(blocks[b])]
        table[b, :len(ids)] = ids
        lens.append(shared[group[b]] * bs + own[b])
    return torch.from_numpy(table), lens, pool
