"""fp64 definitions of the operators around the decode, and inputs for their tests."""
from __future__ import annotations

import numpy as np
import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
FORMATS = [torch.float8_e4m3fn, torch.int8]


def norm_rope64(x, weight=None, eps=1e-6, cos_sin=None, positions=None, interleaved=False):
    """(y, size): RMS norm and rotation of heads [T, H, D] in fp64, and for each element the
    magnitude that its rounding errors are relative to (|a| + |b| of its rotation pair)."""
    x = x.double().cpu()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double().cpu()
    y, size = x.clone(), x.abs()
    if cos_sin is not None:
        r = cos_sin.shape[1]
        row = cos_sin.double().cpu()[positions.long().cpu()][:, None]
        c, s = row[..., :r // 2], row[..., r // 2:]
        i = torch.arange(r // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def codes32(x, dtype):
    """Codes and scales of fp32 rows by the documented fp32 arithmetic (exact)."""
    x = x.float().cpu()
    amax = x.abs().amax(-1)
    ok = torch.isfinite(x).all(-1)
    keep = ok & (amax >= 2.0 ** -100)
    m = torch.tensor(QMAX[dtype])
    y = torch.where(keep[..., None], x * (m / amax)[..., None], torch.zeros(()))
    codes = y.to(dtype) if dtype == torch.float8_e4m3fn else y.round().clamp(-127, 127).to(dtype)
    scale = torch.where(keep, amax / m, torch.where(ok, torch.zeros(()), torch.full((), float("nan"))))
    return codes, scale


def half_step(y, dtype):
    """Half the spacing of codes around y (in code units)."""
    if dtype == torch.int8:
        return torch.full_like(y, 0.5)
    e = torch.frexp(y)[1].clamp(min=-5)
    return torch.ldexp(torch.ones_like(y), e - 4) / 2


def place(table, lens, starts, bs):
    """(sequence, position, block, slot, row) of every live new token."""
    out = []
    for b, n in enumerate(lens):
        for row in range(int(starts[b]), int(starts[b + 1])):
            at = n - int(starts[b + 1]) + row
            if at >= 0:
                out.append((b, at, int(table[b, at // bs]), at % bs, row))
    return out


def random_cache(g, num_blocks, bs, hkv, d, dtype):
    """A quantised cache of normal values on the CPU: (k_pool, v_pool, scales)."""
    scales = torch.empty(num_blocks, hkv, 2, bs)
    pools = []
    for i in range(2):
        x = torch.randn((num_blocks, bs, hkv, d), generator=g)
        x *= torch.exp2(torch.randint(-3, 4, (num_blocks, bs, hkv, 1), generator=g).float())
        c, s = codes32(x, dtype)
        pools.append(c)
        scales[:, :, i] = s.transpose(1, 2)
    return pools[0], pools[1], scales


def rows64(pool, scales, which, table_row, n, bs):
    """A sequence's dequantised rows [n, Hkv, D] in fp64."""
    blocks = table_row[:(n + bs - 1) // bs].long()
    x = pool.view(torch.uint8)[blocks].view(pool.dtype).double() if pool.dtype != torch.bfloat16 else pool[blocks].double()
    if scales is not None:
        x = x * scales[blocks, :, which].double().transpose(1, 2)[..., None]
    return x.flatten(0, 1)[:n]


def decode64(q, k_pool, v_pool, scales, table, lens, bs, scale=None):
    """(out, size) of causal decode, q [B, n, Hq, D]: fp64 attention and, for each element,
    what rounding errors of the weights are relative to.

    That is sum p |v| while a weight's error is relative to it.  Weights p vs (vs the row's V
    scale) enter the product as fp16, whose numbers below 2^-14 have an absolute half step of
    2^-25; the largest weight of a column is at least 2^6 there, so a weight's error is at most
    2^-31 of the largest, times its code.  Where the largest weight meets a code of 0, that is
    all there is: an int8 row of D = 64 with p = 1 - 6e-8 and code 0 leaves size 6.5e-8 (weights
    of 1e-6 in fp16) and an error of 6.4e-11 where 2^-10 of the size is 6.3e-11.  So with a
    tolerance of 2^-10, size counts 2^-21 of the largest weight times the sum of |codes| too."""
    B, n, hq, d = q.shape
    hkv = k_pool.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros_like(out)
    for b in range(B):
        L = int(lens[b])
        k, v = (rows64(p, scales, i, table[b], max(L, 0), bs) for i, p in enumerate((k_pool, v_pool)))
        vs = torch.ones(v.shape[:2], dtype=torch.float64) if scales is None else \
            scales[table[b].long(), :, 1].double().transpose(1, 2).flatten(0, 1)[:v.shape[0]]
        code = v.abs() / torch.where(vs == 0, 1.0, vs)[..., None]
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                continue
            qq = q[b, i].double().reshape(hkv, hq // hkv, d)
            p = torch.softmax(scale * qq @ k[:m].permute(1, 2, 0), -1)
            out[b, i] = (p @ v[:m].transpose(0, 1)).reshape(hq, d)
            top = (p * vs[:m].T[:, None]).amax(-1, keepdim=True)
            flushed = 2.0 ** -21 * top * code[:m].sum(0)[:, None]
            size[b, i] = (p @ v[:m].abs().transpose(0, 1) + flushed).reshape(hq, d)
    return out, size


def sequences(rng, lens, bs, spare=2):
    """A shuffled block table (int32, CPU) for lens, and the pool size it needs."""
    blocks = [-(-max(n, 0) // bs) for n in lens]
    pool = sum(blocks) + spare
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(1, *blocks) if blocks else 1), pool - 1, dtype=np.int32)
    at = 0
    for b, nb in enumerate(blocks):
        table[b, :nb] = order[at:at + nb]
        at += nb
    return torch.from_numpy(table), pool
