"""Decode with capped and biased scores, with sums of attention weights, and over shared prefixes, against fp64
definitions.

Tolerances.  A bf16 output is off by at most half a step, 2^-8 of its value.  A score is a sum of up to 256 products in
fp32: off by 256 * 2^-24 of sum |q k| / sqrt(D), which is 16 or so for normal q and k, at most 2^-12, and the cap adds a
few 2^-24 of itself (50: 2^-17).  So a softmax weight is off by 2^-11 of itself, and by what it enters the product
with V as: two bf16 parts (2^-17), or one fp16 part (2^-11): together 2^-10 of sum p |v|, and 2^-9 where the fp16 part is.
Sums of weights are off by 2^-10 of the weights they add, and by fp32's rounding of the sum.
"""
import numpy as np
import pytest
import torch

import paged_gqa_decode_05_gb300 as pda
import scored_ref as ref

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
NAMES = {torch.bfloat16: "bf16", torch.float8_e4m3fn: "e4m3", torch.int8: "int8"}
formats = pytest.mark.parametrize("dtype", ref.FORMATS, ids=NAMES.get)


def product(dtype):
    return 2.0 ** -10 if dtype is torch.bfloat16 else 2.0 ** -9


def ctx_of(hq, hkv, d, bs, max_seqs=64):
    return pda.Context(max_seqs=max_seqs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - tol
    assert off.max() <= 0, f"{off.max()} beyond its tolerance at {np.unravel_index(int(off.argmax()), off.shape)}"


def inputs(seed, dtype, hq, hkv, d, bs, lens, n):
    g = gen(seed)
    table, pool = ref.ref.sequences(np.random.default_rng(seed), lens, bs)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(lens), n, hq, d), generator=g).bfloat16()
    slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq)
    return g, table, pool, cache, q, slopes


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


SHAPES = [  # hq, hkv, d, bs, q_len, lens
    (4, 2, 64, 16, 1, [37, 0, 1, 80]),
    (8, 8, 128, 16, 1, [129, 64, 17]),
    (32, 4, 128, 32, 1, [1, 700, 33, 31, 0, 2000]),
    (5, 1, 256, 8, 1, [300, 8, 9]),
    (12, 4, 128, 64, 3, [65, 2, 190]),
    (16, 2, 64, 1, 2, [5, 130, 0]),
    (6, 2, 256, 4, 5, [77, 3, 4, 260]),
    (3, 1, 128, 2, 7, [40, 9]),
]


@formats
@pytest.mark.parametrize("hq,hkv,d,bs,n,lens", SHAPES)
@pytest.mark.parametrize("softcap,biased", [(0.0, True), (5.0, False), (50.0, True), (0.0, False)])
def test_scored(dtype, hq, hkv, d, bs, n, lens, softcap, biased):
    _, table, _, cache, q, slopes = inputs(d + bs, dtype, hq, hkv, d, bs, lens, n)
    want, size, _ = ref.scored64(q, *cache, table, lens, bs, softcap=softcap, slopes=slopes if biased else None)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    for out_dtype in (torch.bfloat16, torch.float32):
        got = ctx.decode_scored(qq, kp, vp, t, ln, softcap=softcap, alibi_slopes=sl if biased else None, scales=sc,
                                out_dtype=out_dtype)
        within(got, want, (BF16 * want.abs() if out_dtype is torch.bfloat16 else 0) + product(dtype) * size)
    if n == 1:
        one = ctx.decode_scored(qq[:, 0], kp, vp, t, ln, softcap=softcap, alibi_slopes=sl if biased else None, scales=sc,
                                out_dtype=torch.float32)
        assert torch.equal(one, got[:, 0])
    assert ctx.read_device_errors() == 0


@formats
def test_scored_scales_and_strides(dtype):
    """Negative, zero and large scales; pools in the slot layout."""
    hq, hkv, d, bs, lens = 8, 2, 128, 16, [200, 31]
    _, table, pool, cache, q, slopes = inputs(5, dtype, hq, hkv, d, bs, lens, 2)
    ctx = ctx_of(hq, hkv, d, bs)
    strides = pda.slot_strides(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)
    slots = torch.zeros((pool, 2, hkv, bs, d), dtype=cache[0].dtype)
    for i in range(2):
        raw = cache[i].view(torch.int8) if dtype is not torch.bfloat16 else cache[i]
        (slots.view(torch.int8) if dtype is not torch.bfloat16 else slots)[:, i].copy_(raw.transpose(1, 2))
    slots, sc, t, qq, sl = up(slots, cache[2], table, q, slopes)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    flat = slots.view(-1)
    for scale in (-0.3, 0.0, 2.0, None):
        want, size, _ = ref.scored64(q, *cache, table, lens, bs, scale=scale, softcap=3.0, slopes=slopes)
        got = ctx.decode_scored(qq, flat, flat[hkv * bs * d:], t, ln, softcap=3.0, alibi_slopes=sl, scales=sc, scale=scale,
                                strides=strides, num_blocks=pool)
        # (a scale of 2 takes 16 times the usual scores: their errors, too, before a cap of 3 shrinks them)
        within(got, want, BF16 * want.abs() + product(dtype) * size * (16 if scale == 2.0 else 1))


@formats
@pytest.mark.parametrize("hq,hkv,d,bs,n,lens", SHAPES + [(24, 8, 64, 16, 1, [3000, 500]), (8, 1, 128, 16, 20, [300, 10])])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_weights(dtype, hq, hkv, d, bs, n, lens, softcap):
    g, table, pool, cache, q, slopes = inputs(d + bs + 1, dtype, hq, hkv, d, bs, lens, n)
    old = torch.rand((pool, hkv, bs), generator=g) * 3
    want, size, sums = ref.scored64(q, *cache, table, lens, bs, softcap=softcap, slopes=slopes if softcap else None)
    after, added = ref.add_sums(old, sums, table, lens, bs, n)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq, sl, before = up(*cache, table, q, slopes, old)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    w = before.clone()
    kw = dict(softcap=softcap, alibi_slopes=sl if softcap else None, scales=sc)
    got = ctx.decode_scored(qq, kp, vp, t, ln, weights=w, **kw)
    within(got, want, BF16 * want.abs() + product(dtype) * size)
    seen = (added >= 0).cuda()
    within(w, after, 2.0 ** -10 * added.clamp(min=0) + 2.0 ** -22 * after)
    assert torch.equal(w[~seen], before[~seen])
    # the sums of another buffer, and the same bits again
    other = before + 1.0
    assert torch.equal(ctx.decode_scored(qq, kp, vp, t, ln, weights=other, weights_from=before, **kw), got)
    assert torch.equal(other[seen], w[seen]) and torch.equal(other[~seen], before[~seen] + 1.0)
    # without sums the output is the same
    assert torch.equal(ctx.decode_scored(qq, kp, vp, t, ln, **kw), got)
    assert ctx.read_device_errors() == 0


@formats
def test_weights_of_new_tokens_ignore_what_was_there(dtype):
    hq, hkv, d, bs, lens, n = 8, 2, 64, 16, [33, 5], 3
    g, table, pool, cache, q, _ = inputs(9, dtype, hq, hkv, d, bs, lens, n)
    kp, vp, sc, t, qq = up(*cache, table, q)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    clean, dirty = ctx.new_weights(pool), ctx.new_weights(pool)
    for b, L in enumerate(lens):
        for at in range(L - n, L):
            dirty[table[b, at // bs], :, at % bs] = float("nan")
    a = ctx.decode_scored(qq, kp, vp, t, ln, weights=clean, scales=sc)
    b = ctx.decode_scored(qq, kp, vp, t, ln, weights=dirty, scales=sc)
    assert torch.equal(a, b) and torch.equal(clean, dirty)


GROUPS = [  # hq, hkv, d, bs, q_len, starts, shared blocks, own tokens
    (4, 2, 64, 16, 1, [0, 4], [10], [1, 20, 33, 16]),
    (32, 8, 128, 16, 1, [0, 9], [67], [5, 100, 0, 17, 16, 31, 1, 64, 300]),
    (8, 2, 128, 32, 1, [0, 2, 3, 3, 6], [5, 40, 3, 0], [7, 90, 1, 2, 300, 11]),
    (16, 4, 256, 8, 1, [0, 3], [90], [1, 2, 50]),
    (24, 8, 64, 64, 2, [0, 1, 5], [2, 9], [64, 3, 70, 2, 5]),
    (8, 1, 128, 16, 4, [0, 12], [20], [4 + 3 * i for i in range(12)]),     # 384 q rows: three tiles
    (8, 1, 256, 4, 3, [0, 8], [33], [3 + i for i in range(8)]),            # 192 q rows, one stream
    (5, 1, 64, 1, 1, [0, 30], [137], [1 + i for i in range(30)]),          # 150 q rows of five heads
    (40, 8, 128, 2, 1, [0, 3], [500], [9, 1, 30]),
    (64, 8, 128, 16, 1, [0, 40], [300], [1 + 7 * i for i in range(40)]),   # 320 q rows, long
]


@formats
@pytest.mark.parametrize("hq,hkv,d,bs,n,starts,shared,own", GROUPS)
@pytest.mark.parametrize("softcap,biased", [(0.0, False), (10.0, True)])
def test_shared(dtype, hq, hkv, d, bs, n, starts, shared, own, softcap, biased):
    g = gen(len(own) + d)
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, starts, shared)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(own), n, hq, d), generator=g).bfloat16()
    slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq)
    want, size, _ = ref.scored64(q, *cache, table, lens, bs, softcap=softcap, slopes=slopes if biased else None)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
    ln, st, sh = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, starts, shared))
    kw = dict(softcap=softcap, alibi_slopes=sl if biased else None, scales=sc)
    for out_dtype in (torch.bfloat16, torch.float32):
        got = ctx.decode_shared(qq, kp, vp, t, ln, sh, starts=st, out_dtype=out_dtype, **kw)
        assert ctx.read_device_errors() == 0
        within(got, want, (BF16 * want.abs() if out_dtype is torch.bfloat16 else 0) + product(dtype) * size)
    again = ctx.decode_shared(qq, kp, vp, t, ln, sh, starts=st, out_dtype=out_dtype, **kw)
    assert torch.equal(again, got)
    if len(shared) == 1:
        assert torch.equal(ctx.decode_shared(qq, kp, vp, t, ln, sh, out_dtype=out_dtype, **kw), got)
        if n == 1:
            assert torch.equal(ctx.decode_shared(qq[:, 0], kp, vp, t, ln, sh, out_dtype=out_dtype, **kw), got[:, 0])


@formats
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_with_sequences_that_end_in_the_prefix(dtype, d):
    """Lengths of zero, inside the prefix, at its end and past it; sequences of no group; no shared blocks at all."""
    hq, hkv, bs, n = 6, 2, 16, 2
    starts, shared, own = [1, 6], [20], [40, 0, 0, 0, 30, 18, 3]
    g = gen(d)
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, [0, 7], shared)
    lens = [lens[0], 0, 100, 320, lens[4], 1, lens[6]]
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((7, n, hq, d), generator=g).bfloat16()
    want, size, _ = ref.scored64(q, *cache, table, lens, bs)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq = up(*cache, table, q)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    for st, sh in ((starts, shared), ([0, 7], [0]), ([3, 3], [20]), ([0, 0, 7, 7], [20, 20, 20])):
        st, sh = (torch.tensor(x, dtype=torch.int32).cuda() for x in (st, sh))
        got = ctx.decode_shared(qq, kp, vp, t, ln, sh, starts=st, scales=sc)
        within(got, want, BF16 * want.abs() + product(dtype) * size)
    assert ctx.read_device_errors() == 0


def test_shared_plans_that_are_no_plans():
    """Starts that decrease or leave the batch and impossible block counts are clamped and flagged; the output stays
    that of the sequences whose prefix is what the tables say."""
    hq, hkv, d, bs = 4, 2, 64, 16
    own = [5, 9, 30]
    table, lens, pool = ref.shared_table(np.random.default_rng(1), own, bs, [0, 3], [4])
    g = gen(1)
    cache = ref.random_cache(g, pool, bs, hkv, d, torch.bfloat16)
    q = torch.randn((3, 1, hq, d), generator=g).bfloat16()
    want, size, _ = ref.scored64(q, *cache, table, lens, bs)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, t, qq = up(*cache[:2], table, q)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    for st, sh in (([0, 5], [4]), ([-3, 3], [4]), ([0, 2, 1], [4, 4]), ([2, 0, 3], [4, 4]), ([0, 3], [-1])):
        got = ctx.decode_shared(qq, kp, vp, t, ln, torch.tensor(sh, dtype=torch.int32).cuda(),
                                starts=torch.tensor(st, dtype=torch.int32).cuda())
        within(got, want, BF16 * want.abs() + 2.0 ** -10 * size)
        assert ctx.read_device_errors() == pda.DEVERR_BAD_LENGTH
    ctx.decode_shared(qq, kp, vp, t, ln, torch.tensor([1000], dtype=torch.int32).cuda())
    assert ctx.read_device_errors() & pda.DEVERR_BAD_LENGTH


@formats
def test_bad_blocks_read_as_zeros_in_the_prefix(dtype):
    hq, hkv, d, bs = 8, 2, 128, 16
    own = [5, 40]
    table, lens, pool = ref.shared_table(np.random.default_rng(2), own, bs, [0, 2], [30])
    g = gen(2)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((2, 1, hq, d), generator=g).bfloat16()
    bad = table.clone()
    zero = int(table[0, 3])
    bad[:, 3] = pool + 7
    raw = [c.view(torch.int8) if c.element_size() == 1 else c for c in cache[:2]]
    for c in raw:
        c[zero] = 0
    want, size, _ = ref.scored64(q, *cache, table, lens, bs)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, qq = up(*cache, bad, q)
    got = ctx.decode_shared(qq, kp, vp, t, torch.tensor(lens, dtype=torch.int32).cuda(),
                            torch.tensor([30], dtype=torch.int32).cuda(), scales=sc)
    within(got, want, BF16 * want.abs() + product(dtype) * size)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_BLOCK_ID
