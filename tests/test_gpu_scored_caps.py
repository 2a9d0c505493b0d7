"""Caps of every size, against fp64 definitions.  Outputs in fp32, whose own rounding hides nothing.

Tolerances are those of the operators' tests.  The cap's share of them: an exponential and a reciprocal that are off by
2^-22 put tanh's definition 1 - 2 / (1 + e) off by 2^-21 of the cap, 2^-14 of a score's unit at a cap of 128; above
that scores within a quarter of the cap come from a series (2^-21 of the score, of 16 or so), the others are off by
2^-19 of themselves, which is 32 steps of fp32, and no more than a score's own error counts, 2^-12.
"""
import numpy as np
import pytest
import torch

import scored_ref as ref
from test_gpu_scored import ctx_of, formats, gen, inputs, product, up, within

pytestmark = pytest.mark.gpu
CAPS = [1e-3, 0.1, 2.0, 100.0, 128.0, 129.0, 1e3, 1e4, 1e5, 1e6]
caps = pytest.mark.parametrize("softcap", CAPS)


@formats
@caps
@pytest.mark.parametrize("hq,hkv,d,bs,n,lens", [  # walks of one query, of 8, 16 and 32 rows
    (8, 2, 128, 16, 1, [1500, 40]), (8, 2, 64, 16, 2, [300, 2]), (8, 2, 128, 16, 3, [700, 65]), (20, 4, 64, 8, 4, [90, 400]),
    (6, 2, 256, 16, 1, [500, 3])])
def test_scored(dtype, softcap, hq, hkv, d, bs, n, lens):
    g, table, pool, cache, q, _ = inputs(d + n, dtype, hq, hkv, d, bs, lens, n)
    old = torch.rand((pool, hkv, bs), generator=g)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq = up(*cache, table, q)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    # (a scale of 2 takes scores of 20 times the usual size, and their errors as far as the cap lets them through)
    for scale in (None, 2.0):
        want, size, sums = ref.scored64(q, *cache, table, lens, bs, scale=scale, softcap=softcap)
        after, added = ref.add_sums(old, sums, table, lens, bs, n)
        w = old.clone().cuda()
        got = ctx.decode_scored(qq, kp, vp, t, ln, softcap=softcap, scale=scale, scales=sc, weights=w, out_dtype=torch.float32)
        wide = 2 * d ** 0.5 if scale else 1
        within(got, want, product(dtype) * size * wide)
        within(w, after, 2.0 ** -10 * added.clamp(min=0) * wide + 2.0 ** -22 * after + hq // hkv * n * 2.0 ** -126)


@formats
@caps
@pytest.mark.parametrize("hq,hkv,d,bs,n,blocks,own,biased", [
    (8, 2, 128, 16, 1, 100, [30, 0, 5], False), (8, 1, 64, 16, 4, 20, [9 + i for i in range(10)], True),
    (8, 2, 256, 8, 1, 60, [1, 7], False)])
def test_shared(dtype, softcap, hq, hkv, d, bs, n, blocks, own, biased):
    g = gen(d + n)
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, [0, len(own)], [blocks])
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(own), n, hq, d), generator=g).bfloat16()
    slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq) if biased else None
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
    ln, sh = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, [blocks]))
    for scale in (None, 2.0):
        want, size, _ = ref.scored64(q, *cache, table, lens, bs, scale=scale, softcap=softcap, slopes=slopes)
        got = ctx.decode_shared(qq, kp, vp, t, ln, sh, softcap=softcap, scale=scale, alibi_slopes=sl, scales=sc,
                                out_dtype=torch.float32)
        within(got, want, product(dtype) * size * (2 * d ** 0.5 if scale else 1))


@pytest.mark.parametrize("softcap", [1e3, 1e6])
def test_infinite_scores(softcap):
    """Scores of plus and minus infinity come out as plus and minus the cap."""
    hq, hkv, d, bs, lens = 4, 2, 64, 16, [40]
    _, table, _, cache, q, _ = inputs(7, torch.bfloat16, hq, hkv, d, bs, lens, 1)
    q[:] = 0
    q[..., 0] = 1
    ctx = ctx_of(hq, hkv, d, bs)
    cache[0][:] = 0
    cache[0][table[0, 0].long(), 3, :, 0] = float("-inf")
    kp, vp, t, qq = up(*cache[:2], table, q)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    want = torch.cat([cache[1][table[0, :3].long()].flatten(0, 1)[:40][i:i + 1] for i in range(40) if i != 3]).double().mean(0)
    for got in (ctx.decode_scored(qq, kp, vp, t, ln, softcap=softcap, out_dtype=torch.float32),
                ctx.decode_shared(qq, kp, vp, t, ln, torch.tensor([2], dtype=torch.int32).cuda(), softcap=softcap,
                                  out_dtype=torch.float32)):
        within(got.view(2, 2, d), want[:, None].expand(2, 2, d), 2.0 ** -10 * want.abs().max() + 2.0 ** -15)
