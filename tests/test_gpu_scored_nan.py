"""NaN in scored decode, in sums of attention weights and behind a shared prefix: a query that is NaN, or that sees NaN
keys only, gets NaN, and nobody else notices.  What is not NaN is equal to the bit to the same call without NaN: rows of
q, and tokens of a sum, are computed apart."""
import numpy as np
import pytest
import torch

import scored_ref as ref
from test_gpu_scored import ctx_of, formats, gen, inputs, up

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


FORMS = [  # hq, hkv, d, bs, q_len, lens: walks of one query, of 8, 16 and 32 rows, of several launch rows; units in pieces
    (4, 2, 64, 16, 1, [3000, 37, 1]),
    (8, 1, 128, 16, 1, [5000]),
    (8, 2, 128, 16, 2, [2500, 40]),
    (8, 2, 128, 16, 3, [1500, 50]),
    (40, 8, 64, 16, 4, [2100, 30]),
    (8, 2, 256, 8, 2, [900, 45]),
    (3, 1, 128, 2, 7, [1200, 9]),
    (8, 2, 64, 16, 11, [700, 20]),
]
forms = pytest.mark.parametrize("hq,hkv,d,bs,n,lens", FORMS)


def poison_keys(cache, table, b, tokens, bs, head):
    """NaN keys of one sequence and kv head: values in bf16, scales in 8 bits."""
    for t in tokens:
        block, slot = int(table[b, t // bs]), t % bs
        if cache[2] is None:
            cache[0][block, slot, head] = NAN
        else:
            cache[2][block, head, 0, slot] = NAN


@formats
@forms
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_a_nan_query_gives_nan(dtype, hq, hkv, d, bs, n, lens, softcap):
    _, table, pool, cache, q, slopes = inputs(d + n, dtype, hq, hkv, d, bs, lens, n)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t, sl = up(*cache, table, slopes)
    kw = dict(softcap=softcap, alibi_slopes=sl if softcap else None, scales=sc)
    for out_dtype in (torch.bfloat16, torch.float32):
        clean = ctx.decode_scored(q.cuda(), kp, vp, t, i32(lens), out_dtype=out_dtype, **kw)
        for b in range(len(lens)):
            bad, i, h = q.clone(), n // 2, hq - 1
            bad[b, i, h, 5] = NAN
            out = ctx.decode_scored(bad.cuda(), kp, vp, t, i32(lens), out_dtype=out_dtype, **kw)
            rest = torch.ones(q.shape[:3], dtype=torch.bool)
            rest[b, i, h] = lens[b] - n + i < 0  # (a query in front of the sequence sees nothing)
            assert torch.isnan(out[~rest.cuda()]).all()
            assert torch.equal(out[rest.cuda()], clean[rest.cuda()])
    assert ctx.read_device_errors() == 0


@formats
@forms
def test_nan_keys_of_a_whole_piece_give_nan(dtype, hq, hkv, d, bs, n, lens):
    """The middle half of a sequence, one that several CTAs share, and all of it."""
    _, table, pool, cache, q, _ = inputs(d + n, dtype, hq, hkv, d, bs, lens, n)
    ctx = ctx_of(hq, hkv, d, bs)
    G, L = hq // hkv, lens[0]
    kp, vp, sc, t, qq = up(*cache, table, q)
    clean = ctx.decode_scored(qq, kp, vp, t, i32(lens), scales=sc)
    for tokens in (range(L // 4, 3 * L // 4), range(L)):
        bad = [None if c is None else c.clone() for c in cache]
        poison_keys(bad, table, 0, tokens, bs, hkv - 1)
        kp, vp, sc = up(*bad)
        out = ctx.decode_scored(qq, kp, vp, t, i32(lens), scales=sc)
        assert torch.isnan(out[0, :, -G:]).all()
        assert torch.equal(out[0, :, :-G], clean[0, :, :-G]) and torch.equal(out[1:], clean[1:])


@formats
@forms
def test_a_nan_query_reaches_the_sums_of_what_it_sees_only(dtype, hq, hkv, d, bs, n, lens):
    """The tokens behind it, which later queries of its launch row see, keep their sums."""
    g, table, pool, cache, q, _ = inputs(d + n, dtype, hq, hkv, d, bs, lens, n)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t = up(*cache, table)
    old = torch.rand((pool, hkv, bs), generator=g).cuda()
    clean = old.clone()
    ctx.decode_scored(q.cuda(), kp, vp, t, i32(lens), weights=clean, scales=sc)
    assert torch.isfinite(clean).all()
    for b, L in enumerate(lens):
        for i in {0, n // 2, n - 1}:
            bad, seen = q.clone(), max(0, L - n + i + 1)
            bad[b, i, hq - 1, 5] = NAN
            sums = old.clone()
            ctx.decode_scored(bad.cuda(), kp, vp, t, i32(lens), weights=sums, scales=sc)
            want = clean.clone()
            at = torch.arange(seen)
            want[table[b].long()[at // bs].cuda(), hkv - 1, (at % bs).cuda()] = NAN
            assert torch.equal(torch.isnan(sums), torch.isnan(want))
            assert torch.equal(sums.nan_to_num(-1.0), want.nan_to_num(-1.0))
    assert ctx.read_device_errors() == 0


SHARED = [  # hq, hkv, d, bs, q_len, shared blocks, own tokens: pieces on many CTAs and on one, one stream and two
    (8, 2, 128, 16, 1, 200, [0, 30, 0, 5]),
    (4, 2, 64, 16, 1, 4, [3, 0]),
    (16, 4, 256, 8, 1, 300, [0, 9, 1]),
    (32, 8, 128, 16, 2, 700, [2 + i for i in range(24)]),
    (64, 8, 128, 32, 1, 40, [0] * 40),
]
shapes = pytest.mark.parametrize("hq,hkv,d,bs,n,blocks,own", SHARED)


def shared_rig(dtype, hq, hkv, d, bs, n, blocks, own):
    g = gen(d + n)
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, [0, len(own)], [blocks])
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(own), n, hq, d), generator=g).bfloat16()
    return table, lens, cache, q


@formats
@shapes
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_a_nan_query_behind_a_prefix(dtype, hq, hkv, d, bs, n, blocks, own, softcap):
    table, lens, cache, q = shared_rig(dtype, hq, hkv, d, bs, n, blocks, own)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, sc, t = up(*cache, table)
    run = lambda x: ctx.decode_shared(x.cuda(), kp, vp, t, i32(lens), i32([blocks]), softcap=softcap, scales=sc)  # noqa: E731
    clean = run(q)
    assert torch.isfinite(clean).all()
    for b in {0, 1, len(own) - 1}:
        bad = q.clone()
        bad[b, n // 2, hq - 1, 5] = NAN
        out = run(bad)
        rest = torch.ones(q.shape[:3], dtype=torch.bool)
        rest[b, n // 2, hq - 1] = False
        assert torch.isnan(out[~rest.cuda()]).all()
        assert torch.equal(out[rest.cuda()], clean[rest.cuda()])
    assert ctx.read_device_errors() == 0


@formats
@shapes
def test_nan_keys_all_over_a_prefix(dtype, hq, hkv, d, bs, n, blocks, own):
    """Its second quarter, and all of it: pieces without a score that is a number."""
    table, lens, cache, q = shared_rig(dtype, hq, hkv, d, bs, n, blocks, own)
    ctx = ctx_of(hq, hkv, d, bs)
    G, L = hq // hkv, blocks * bs
    kp, vp, sc, t, qq = up(*cache, table, q)
    clean = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32([blocks]), scales=sc)
    for tokens in (range(L // 4, L // 2), range(L)):
        bad = [None if c is None else c.clone() for c in cache]
        poison_keys(bad, table, 0, tokens, bs, hkv - 1)
        kp, vp, sc = up(*bad)
        out = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32([blocks]), scales=sc)
        assert torch.isnan(out[:, :, -G:]).all()
        assert torch.equal(out[:, :, :-G], clean[:, :, :-G])
