"""Norm and rotation of q / k heads, cache writes, read-backs and decode over
8-bit caches against fp64 definitions.

Tolerances.  A bf16 output is off by at most half a step (2^-8 of its value)
plus what fp32 arithmetic adds: a norm and a rotation are about ten roundings
of 2^-24 and a reciprocal square root of 2^-22, under 2^-20 of |a| + |b| of the
rotation pair.  A code is off by half the spacing of codes, and by 2^-20 of the
largest code for that arithmetic.  Decode weights enter the products as fp16
(2^-11 each at most); scores, exponentials and sums in fp32 stay below another
2^-11 of sum p |v| for scores of this size.
"""
import numpy as np
import pytest
import torch

import cache_ref as ref
import paged_gqa_decode_05_gb300 as pda

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
DECODE = 2.0 ** -10


def ctx_of(hq, hkv, d, bs, max_seqs=64):
    return pda.Context(max_seqs=max_seqs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - tol
    assert off.max() <= 0, f"{off.max()} beyond its tolerance at {np.unravel_index(int(off.argmax()), off.shape)}"


def qkv_of(g, tokens, hq, hkv, d):
    return torch.randn((tokens, hq + 2 * hkv, d), generator=g).bfloat16().cuda()


# ------------------------------------------------------------------ norm_rope

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rotary,tokens", [
    (4, 2, 64, 64, 1), (32, 8, 128, 128, 33), (5, 1, 128, 64, 257), (16, 4, 256, 256, 7), (3, 3, 64, 8, 100),
    (8, 8, 256, 24, 65), (64, 8, 128, 120, 19),
    # enough tokens for the streaming form, and (rotary 24) for the other at that size
    (32, 8, 128, 128, 1500), (12, 4, 64, 32, 5111), (16, 4, 256, 128, 1024), (8, 1, 128, 128, 4001), (48, 16, 256, 64, 257),
    (2, 1, 64, 24, 23000)])
def test_norm_rope(hq, hkv, d, rotary, tokens, interleaved):
    g = gen(tokens)
    ctx = ctx_of(hq, hkv, d, 16)
    qkv = qkv_of(g, tokens, hq, hkv, d)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    table = pda.rope_table(9000, rotary)
    pos = torch.randint(0, 9000, (tokens,), generator=g, dtype=torch.int32).cuda()
    for dtype in (torch.bfloat16, torch.float32):
        wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
        got = ctx.norm_rope(q, k, pos, q_weight=wq, k_weight=wk, cos_sin=table, interleaved=interleaved)
        for y, x, w in zip(got, (q, k), (wq, wk)):
            want, size = ref.norm_rope64(x, w, cos_sin=table, positions=pos, interleaved=interleaved)
            within(y, want, BF16 * want.abs() + 2.0 ** -20 * size)
    assert ctx.read_device_errors() == 0


def test_norm_rope_parts_alone():
    """Norm without rotation, rotation without norm, q or k alone, and in place."""
    g = gen(3)
    ctx = ctx_of(8, 2, 128, 16)
    qkv = qkv_of(g, 21, 8, 2, 128)
    q, k = qkv[:, :8], qkv[:, 8:10]
    w = torch.rand(128, generator=g).cuda() + 0.5
    table, pos = pda.rope_table(64, 128), torch.arange(21, dtype=torch.int32).cuda()
    want, _ = ref.norm_rope64(q, w, eps=1e-2)
    a, none = ctx.norm_rope(q, None, q_weight=w, eps=1e-2)
    assert none is None
    within(a, want, (BF16 + 2.0 ** -20) * want.abs())
    want, size = ref.norm_rope64(k, cos_sin=table, positions=pos)
    none, b = ctx.norm_rope(None, k, pos, cos_sin=table)
    assert none is None
    within(b, want, BF16 * want.abs() + 2.0 ** -20 * size)
    before = qkv.clone()
    apart = ctx.norm_rope(q, k, pos, q_weight=w, cos_sin=table)
    ctx.norm_rope(q, k, pos, q_weight=w, cos_sin=table, q_out=q, k_out=k)
    assert torch.equal(qkv[:, :8], apart[0]) and torch.equal(qkv[:, 8:10], apart[1])
    assert torch.equal(qkv[:, 10:], before[:, 10:])


def test_norm_rope_bad_positions_are_flagged():
    ctx = ctx_of(4, 2, 64, 16)
    qkv = qkv_of(gen(4), 5, 4, 2, 64)
    table = pda.rope_table(8, 64)
    pos = torch.tensor([0, 8, 3, -1, 7], dtype=torch.int32).cuda()
    q, _ = ctx.norm_rope(qkv[:, :4], qkv[:, 4:6], pos, cos_sin=table)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_POSITION
    want, size = ref.norm_rope64(qkv[:, :4], cos_sin=table, positions=pos.clamp(0, 7))
    within(q, want, BF16 * want.abs() + 2.0 ** -20 * size)


# ------------------------------------------------------------------ append and read_cache

def check_written(pool, scales, which, codes_in, want, size, places, bs):
    """The rows that `places` lists hold `want` [tokens, Hkv, D] quantised; every other row is as before."""
    dtype = pool.dtype
    untouched = torch.ones(pool.shape[:2], dtype=torch.bool)
    for _, _, blk, slot, row in places:
        untouched[blk, slot] = False
        y = want[row]
        amax = y.abs().amax(-1)
        s = scales[blk, :, which, slot].double()
        assert ((s - amax / ref.QMAX[dtype]).abs() <= 2.0 ** -20 * s).all()
        code = pool.view(torch.uint8)[blk, slot].view(dtype).double()
        exact = y / amax[:, None] * ref.QMAX[dtype]
        tol = ref.half_step(exact, dtype) + 2.0 ** -20 * ref.QMAX[dtype] * (1 + size[row] / amax[:, None])
        assert ((code - exact).abs() <= tol).all()
    raw = pool.view(torch.uint8)
    assert torch.equal(raw[untouched], codes_in.view(torch.uint8)[untouched])


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,bs,lens,news", [
    (32, 8, 128, 16, [5, 16, 17, 300], [1, 1, 1, 1]),
    (4, 2, 64, 1, [3, 1, 9], [3, 1, 2]),
    (8, 1, 256, 4, [40, 0, 7], [40, 0, 5]),
    (6, 2, 128, 64, [100] * 40, [2] * 40),
    (16, 16, 64, 8, [33], [33]),
])
def test_append(dtype, hq, hkv, d, bs, lens, news):
    rng, g = np.random.default_rng(len(lens)), gen(d)
    table, pool = ref.sequences(rng, lens, bs)
    k0, v0, s0 = ref.random_cache(g, pool, bs, hkv, d, dtype)
    ctx = ctx_of(hq, hkv, d, bs)
    starts = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32)
    qkv = qkv_of(g, int(starts[-1]), hq, hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    wk = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda()
    cs = pda.rope_table(max(1, *lens) if len(lens) > 1 else lens[0], d)
    kp, vp, sc = k0.cuda(), v0.cuda(), s0.cuda()
    out = ctx.append(k, v, kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scales=sc,
                     starts=starts.cuda(), q=q, k_weight=wk, cos_sin=cs)
    assert ctx.read_device_errors() == 0
    places = ref.place(table, lens, starts, bs)
    pos = torch.zeros(k.shape[0], dtype=torch.int64)
    for _, at, _, _, row in places:
        pos[row] = at
    want, size = ref.norm_rope64(q, cos_sin=cs, positions=pos)
    within(out, want, BF16 * want.abs() + 2.0 ** -20 * size)
    want, size = ref.norm_rope64(k, wk, cos_sin=cs, positions=pos)
    check_written(kp.cpu(), sc.cpu(), 0, k0, want, size, places, bs)
    # values are quantised from bf16 as they are: every bit is fixed by the fp32 arithmetic
    codes, scale = ref.codes32(v, dtype)
    vc, ss = vp.cpu(), sc.cpu()
    want_v, want_s = v0.clone(), s0.clone()
    for _, _, blk, slot, row in places:
        want_v.view(torch.uint8)[blk, slot] = codes.view(torch.uint8)[row]
        want_s[blk, :, 1, slot] = scale[row]
    assert torch.equal(vc.view(torch.uint8), want_v.view(torch.uint8))
    assert torch.equal(ss[:, :, 1], want_s[:, :, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16] + ref.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,bs,rotary,times", [
    (32, 8, 128, 16, 128, 1), (4, 4, 64, 32, 16, 5), (2, 1, 256, 64, 0, 4), (5, 1, 64, 1, 64, 8), (12, 2, 64, 16, 64, 4), (10, 2, 128, 16, 0, 3)])
def test_append_prompts(dtype, hq, hkv, d, bs, rotary, times):
    """Prompts of a prefill batch, streamed: empty sequences, a block that does not exist, a table too narrow, padding
    behind the last sequence; and the same bits as the tokens appended a few at a time."""
    g, rng = gen(31), np.random.default_rng(31)
    lens = [600 * times, 0, 1, 411 * times, 0, 37 * times, 250 * times]
    table, pool = ref.sequences(rng, lens, bs)
    bad = table.clone()
    bad[5, 0] = pool + 4  # sequence 5's first block
    width = -(-411 * times // bs)  # sequence 0 does not fit
    bad = bad[:, :width].contiguous()
    total = sum(lens)
    starts = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    qkv = qkv_of(g, total + 70, hq, hkv, d)
    ctx = ctx_of(hq, hkv, d, bs)
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    cs = pda.rope_table(600 * times, rotary) if rotary else None
    prep = dict(q_weight=wq, k_weight=wk, cos_sin=cs)
    caches = [ctx.new_cache(pool, dtype) for _ in range(2)]
    outs = [torch.full((total + 70, hq, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    kp, vp, sc = caches[0]
    ctx.append(k, v, kp, vp, bad.cuda(), lens_d, scales=sc, starts=starts.cuda(), q=q, q_out=outs[0], **prep)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_POSITION | pda.DEVERR_BAD_BLOCK_ID
    assert (outs[0][total:] == 3).all()
    kp, vp, sc = caches[1]
    for b, n in enumerate(lens):  # one sequence at a time, 500 tokens at most: the other form of the kernel
        for at in range(0, n, 500):
            m, lo = min(500, n - at), int(starts[b]) + at
            rows = slice(lo, lo + m)
            ctx.append(k[rows], v[rows], kp, vp, bad[b:b + 1].cuda(), torch.tensor([at + m], dtype=torch.int32).cuda(),
                       scales=sc, q=q[rows], q_out=outs[1][rows], **prep)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_POSITION | pda.DEVERR_BAD_BLOCK_ID
    # the sum of squares is taken in another order: a bf16 or code step apart here and there
    assert (outs[0].float() - outs[1].float()).abs().max() <= 2.0 ** -7 * outs[1].float().abs().max()
    for x, y in zip(caches[0][:2], caches[1][:2]):
        x, y = x.float(), y.float()
        assert torch.equal(x.abs().sum((2, 3)) > 0, y.abs().sum((2, 3)) > 0)
        assert (x != y).float().mean() < 1e-3
    assert torch.equal(caches[0][1].view(torch.uint8), caches[1][1].view(torch.uint8))
    # against the definition, where everything is in place
    kp, vp, sc = ctx.new_cache(pool, dtype)
    before = kp.cpu()
    out = ctx.append(k, v, kp, vp, table.cuda(), lens_d, scales=sc, starts=starts.cuda(), q=q, **prep)
    assert ctx.read_device_errors() == 0
    places = ref.place(table, lens, starts, bs)
    pos = torch.zeros(total, dtype=torch.int64)
    for _, at, _, _, row in places:
        pos[row] = at
    want, size = ref.norm_rope64(q[:total], wq, cos_sin=cs, positions=pos)
    within(out[:total], want, BF16 * want.abs() + 2.0 ** -20 * size)
    want, size = ref.norm_rope64(k[:total], wk, cos_sin=cs, positions=pos)
    if dtype == torch.bfloat16:
        got = torch.stack([kp[blk, slot] for _, _, blk, slot, _ in places])
        rows = torch.tensor([row for *_, row in places])
        within(got, want[rows], BF16 * want[rows].abs() + 2.0 ** -20 * size[rows])
    else:
        check_written(kp.cpu(), sc.cpu(), 0, before, want, size, places, bs)


@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 64, 65, 100, 1000])
def test_append_then_read_any_batch(batch):
    """Whole prompts of 0 to 9 tokens written and read back: every token of every sequence in its row."""
    rng, g = np.random.default_rng(batch), gen(batch)
    hkv, d, bs = 2, 64, 4
    for lens in (rng.integers(0, 10, batch), np.where(rng.random(batch) < 0.8, 0, 7), np.ones(batch, dtype=int)):
        lens = [int(n) for n in lens]
        table, pool = ref.sequences(rng, lens, bs)
        total = sum(lens)
        kv = qkv_of(g, total + 3, 0, hkv, d)
        ctx = ctx_of(2, hkv, d, bs, max_seqs=batch)
        kp, vp, _ = ctx.new_cache(pool, torch.bfloat16)
        starts = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
        lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
        ctx.append(kv[:, :hkv], kv[:, hkv:], kp, vp, table.cuda(), lens_d, starts=starts)
        k, v = (torch.full((total + 3, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ctx.read_cache(kp, vp, table.cuda(), lens_d, starts=starts, k_out=k, v_out=v)
        assert ctx.read_device_errors() == 0
        assert torch.equal(k[:total], kv[:total, :hkv]) and torch.equal(v[:total], kv[:total, hkv:])
        assert (k[total:] == 3).all() and (v[total:] == 3).all()
        used = sum(int(p.float().abs().sum((2, 3)).count_nonzero()) for p in (kp, vp))
        assert used == 2 * total


@pytest.mark.parametrize("dtype", ref.FORMATS)
def test_append_without_starts_and_with_positions(dtype):
    """Equal shares per sequence; an explicit rotation position; a sequence shorter than its share."""
    g, rng = gen(9), np.random.default_rng(9)
    lens, bs, hkv, d = [20, 2, 31], 8, 2, 128
    table, pool = ref.sequences(rng, lens, bs)
    ctx = ctx_of(4, hkv, d, bs)
    kv = qkv_of(g, 12, 0, hkv, d)
    kp, vp, sc = ctx.new_cache(pool, dtype)
    before = kp.cpu()
    cs = pda.rope_table(500, 64)
    pos = torch.randint(0, 500, (12,), generator=g, dtype=torch.int32)
    assert ctx.append(kv[:, :hkv], kv[:, hkv:], kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      scales=sc, positions=pos.cuda(), cos_sin=cs) is None
    assert ctx.read_device_errors() == 0
    places = ref.place(table, lens, [0, 4, 8, 12], bs)
    assert len(places) == 10  # two of the second sequence's four rows are padding
    want, size = ref.norm_rope64(kv[:, :hkv], cos_sin=cs, positions=pos)
    check_written(kp.cpu(), sc.cpu(), 0, before, want, size, places, bs)


def test_append_strange_rows():
    """Zero rows, rows too small to scale, infinities and NaN: the documented codes and scales, and what decode
    and read_cache make of them."""
    ctx = ctx_of(2, 1, 64, 8)
    x = torch.randn((6, 1, 64), generator=gen(1)).bfloat16()
    x[1] = 0
    x[2] = 2.0 ** -110
    x[3, 0, 5] = float("inf")
    x[4, 0, 7] = float("nan")
    x[5] *= 2.0 ** 90
    x = x.cuda()
    table, lens = torch.zeros((1, 1), dtype=torch.int32).cuda(), torch.tensor([6], dtype=torch.int32).cuda()
    for dtype in ref.FORMATS:
        kp, vp, sc = ctx.new_cache(1, dtype)
        ctx.append(x, x, kp, vp, table, lens, scales=sc)
        codes, scale = ref.codes32(x, dtype)
        for which, pool in enumerate((kp, vp)):
            assert torch.equal(pool.cpu().view(torch.uint8)[0, :6], codes.view(torch.uint8))
            assert torch.equal(sc.cpu()[0, 0, which, :6].nan_to_num(-1), scale[:, 0].nan_to_num(-1))
        k, v = ctx.read_cache(kp, vp, table, lens, scales=sc, out_dtype=torch.float32)
        assert (k[0, 1:3] == 0).all() and torch.isnan(k[0, 3:5]).all() and torch.isfinite(k[0, 5]).all()
        assert torch.equal(k.nan_to_num(7), v.nan_to_num(7)) and (k[0, 6:] == 0).all()
        q = torch.randn((1, 2, 64), generator=gen(2)).bfloat16().cuda()
        # rows behind the sequence's end may hold anything
        short = torch.tensor([3], dtype=torch.int32).cuda()
        out = ctx.decode(q, kp, vp, table, short, scales=sc, out_dtype=torch.float32)
        want, size = ref.decode64(q[:, None].cpu(), kp.cpu(), vp.cpu(), sc.cpu(), table.cpu(), [3], 8)
        within(out, want[:, 0], DECODE * size[:, 0])
        assert torch.isnan(ctx.decode(q, kp, vp, table, lens, scales=sc)).all()


def test_append_padding_and_bad_places():
    """Rows from starts[batch] on, tokens past the table and bad block ids write nothing."""
    ctx = ctx_of(4, 2, 64, 16)
    kv = qkv_of(gen(6), 9, 0, 2, 64)
    q = torch.randn((9, 4, 64), generator=gen(7)).bfloat16().cuda()
    table = torch.tensor([[1, 2], [9, 0]], dtype=torch.int32).cuda()
    starts = torch.tensor([0, 3, 6], dtype=torch.int32).cuda()
    for dtype in [torch.bfloat16] + ref.FORMATS:
        def cache():
            return ctx.new_cache(4, dtype)
        q_out = torch.full_like(q, 3.0)
        # sequence 0 ends past its two blocks (token 32 and on); sequence 1's first block does not exist
        kp, vp, sc = cache()
        ctx.append(kv[:, :2], kv[:, 2:], kp, vp, table, torch.tensor([34, 18], dtype=torch.int32).cuda(), scales=sc,
                   starts=starts, q=q, q_out=q_out)
        assert ctx.read_device_errors() == pda.DEVERR_BAD_POSITION | pda.DEVERR_BAD_BLOCK_ID
        assert torch.equal(q_out[:6], q[:6]) and (q_out[6:] == 3).all()
        rows = (kp.float().abs().sum((2, 3)) > 0).nonzero().tolist()
        assert rows == [[0, 0], [0, 1], [2, 15]]


@pytest.mark.parametrize("dtype", [torch.bfloat16] + ref.FORMATS)
@pytest.mark.parametrize("d,hkv,bs,lens", [(128, 8, 16, [37, 80, 0, 1]), (64, 2, 1, [5, 3]), (256, 1, 32, [65]),
                                           (64, 3, 4, list(range(40)))])
def test_read_cache(dtype, d, hkv, bs, lens):
    rng, g = np.random.default_rng(5), gen(5)
    table, pool = ref.sequences(rng, lens, bs)
    if dtype == torch.bfloat16:
        kp, vp = (torch.randn((pool, bs, hkv, d), generator=g).bfloat16() for _ in range(2))
        sc = None
    else:
        kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    ctx = ctx_of(hkv, hkv, d, bs)
    args = (kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    kw = dict(scales=None if sc is None else sc.cuda())
    want = [torch.cat([ref.rows64(p, sc, i, table[b], n, bs) for b, n in enumerate(lens)]) for i, p in enumerate((kp, vp))]
    total = sum(lens)
    starts = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
    for out_dtype, tol in ((torch.bfloat16, BF16), (torch.float32, 2.0 ** -24)):
        k, v = (torch.full((total + 3, hkv, d), 7.0, dtype=out_dtype, device="cuda") for _ in range(2))
        ctx.read_cache(*args, starts=starts, k_out=k, v_out=v, **kw)
        for got, w in zip((k, v), want):
            within(got[:total], w, tol * w.abs())
            assert (got[total:] == 7).all()
        k2, none = ctx.read_cache(*args, starts=starts, k_out=torch.zeros_like(k), **kw)
        assert none is None and torch.equal(k2[:total], k[:total])
        k4, v4 = ctx.read_cache(*args, out_dtype=out_dtype, **kw)
        assert k4.shape == (len(lens), table.shape[1] * bs, hkv, d)
        for b, n in enumerate(lens):
            lo = int(starts[b])
            assert torch.equal(k4[b, :n], k[lo:lo + n]) and torch.equal(v4[b, :n], v[lo:lo + n])
            assert (k4[b, n:] == 0).all()
    assert ctx.read_device_errors() == 0


def test_read_cache_bad_pages():
    ctx = ctx_of(2, 2, 64, 8)
    kp, vp, sc = (t.cuda() for t in ref.random_cache(gen(2), 3, 8, 2, 64, torch.int8))
    table = torch.tensor([[2, 5]], dtype=torch.int32).cuda()
    k, v = ctx.read_cache(kp, vp, table, torch.tensor([12], dtype=torch.int32).cuda(), scales=sc)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_BLOCK_ID
    assert (k[0, 8:] == 0).all() and (k[0, :8].abs().sum((1, 2)) > 0).all()
    k, v = (torch.full((40, 2, 64), 5.0, device="cuda") for _ in range(2))
    starts = torch.tensor([0, 40], dtype=torch.int32).cuda()
    table = torch.tensor([[2, 1]], dtype=torch.int32).cuda()
    ctx.read_cache(kp, vp, table, torch.tensor([40], dtype=torch.int32).cuda(), scales=sc, starts=starts, k_out=k, v_out=v)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_LENGTH
    assert (k[16:] == 5).all()


# ------------------------------------------------------------------ decode

LENS = {"tiny": [37, 80], "edges": [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129], "long": [4000, 3, 9001],
        "many": [(37 * i) % 200 for i in range(60)], "few": [943, 0, 2000], "one": [9001]}


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("hq,hkv,d,bs,lens", [
    (4, 2, 64, 16, "tiny"), (8, 2, 128, 16, "edges"), (16, 2, 256, 16, "edges"), (8, 1, 64, 8, "edges"),
    (5, 1, 128, 32, "long"), (12, 4, 128, 1, "edges"), (2, 2, 64, 2, "edges"), (8, 4, 256, 4, "edges"),
    (3, 1, 256, 64, "long"), (16, 8, 128, 16, "many"), (8, 8, 128, 4, "edges"),
    # few units, in many pieces each
    (8, 1, 128, 16, "few"), (4, 1, 256, 4, "few"), (8, 1, 64, 16, "few"), (5, 1, 128, 1, "few"), (8, 1, 128, 16, "one"),
    # many sequences
    (12, 6, 64, 32, "many"), (16, 4, 256, 8, "many"), (8, 8, 64, 64, "many"), (32, 4, 128, 32, "many"),
    (8, 4, 256, 4, "many"), (4, 4, 128, 4, "many"), (6, 2, 128, 64, "many")])
def test_decode(dtype, q_len, hq, hkv, d, bs, lens):
    lens = LENS[lens]
    rng, g = np.random.default_rng(d + bs), gen(d + bs)
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=len(lens) * q_len)
    args = (kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
    scales = sc.cuda()
    if q_len == 1:
        out = ctx.decode(q[:, 0].cuda(), *args, scales=scales, out_dtype=torch.float32)
        within(out, want[:, 0], DECODE * size[:, 0])
    else:
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        ctx.decode_multi(q.cuda(), *args, scales=scales, out=out)
        within(out, want, DECODE * size)
    out = ctx.decode_multi(q.cuda(), *args, scales=scales)
    within(out, want, BF16 * want.abs() + 2 * DECODE * size)
    assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("dtype", ref.FORMATS)
def test_decode_other_strides(dtype):
    """The slot layout (K and V of a block side by side) and a padded pool give the dense pool's bits."""
    g, rng = gen(8), np.random.default_rng(8)
    hq, hkv, d, bs, lens = 8, 2, 128, 16, [37, 200, 64]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((3, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    rest = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    want = ctx.decode(q, kp.cuda(), vp.cuda(), *rest, scales=sc.cuda())
    slot = torch.stack([kp.view(torch.int8).transpose(1, 2), vp.view(torch.int8).transpose(1, 2)], 1).contiguous().cuda()
    slot = slot.view(dtype).flatten()
    strides = pda.slot_strides(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)
    got = ctx.decode(q, slot, slot[hkv * bs * d:], *rest, scales=sc.cuda(), strides=strides, num_blocks=pool)
    assert torch.equal(got, want)
    wide = torch.zeros((pool, bs, hkv, d + 48), dtype=torch.int8)
    pads = []
    for p in (kp, vp):
        w = wide.clone()
        w[..., :d] = p.view(torch.int8)
        pads.append(w.cuda().view(dtype).flatten())
    got = ctx.decode(q, *pads, *rest, scales=sc.cuda(), strides=(bs * hkv * (d + 48), hkv * (d + 48), d + 48),
                     num_blocks=pool)
    assert torch.equal(got, want)


def test_decode_garbage_behind_the_end():
    """Codes and scales past a sequence's end (NaN codes, NaN and infinite scales) do not reach its output."""
    g, rng = gen(12), np.random.default_rng(12)
    hq, hkv, d, bs, lens = 8, 2, 128, 16, [37, 81, 130, 7]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.float8_e4m3fn)
    q = torch.randn((4, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    rest = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    want = ctx.decode(q, kp.cuda(), vp.cuda(), *rest, scales=sc.cuda())
    for b, n in enumerate(lens):
        blk = int(table[b, n // bs])
        for p in (kp, vp):
            p.view(torch.uint8)[blk, n % bs:] = 0x7f
        sc[blk, :, 0, n % bs:] = float("nan")
        sc[blk, :, 1, n % bs:] = float("inf")
    assert torch.equal(ctx.decode(q, kp.cuda(), vp.cuda(), *rest, scales=sc.cuda()), want)


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("bs,d", [(16, 128), (1, 64), (4, 256)])
def test_decode_bad_pages_are_flagged(bs, d, q_len):
    """Block ids outside the pool and lengths past the table raise their flag; the other sequences are as without them."""
    g, rng = gen(43), np.random.default_rng(43)
    hq, hkv, lens = 4, 1, [70, 33, 64]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.int8)
    q = torch.randn((3, q_len, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=3 * q_len)
    cache = [x.cuda() for x in (kp, vp)]

    def run(table, lens):
        lens = torch.tensor(lens, dtype=torch.int32).cuda()
        return ctx.decode_multi(q, *cache, table.cuda(), lens, scales=sc.cuda())

    want = run(table, lens)
    assert ctx.read_device_errors() == 0
    for bad in (-1, pool, 2 ** 31 - 1):
        broken = table.clone()
        broken[1, 0] = bad
        out = run(broken, lens)
        assert ctx.read_device_errors() == pda.DEVERR_BAD_BLOCK_ID
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    for bad in (-5, table.shape[1] * bs + 1, 2 ** 31 - 1):
        out = run(table, [lens[0], bad, lens[2]])
        assert ctx.read_device_errors() == pda.DEVERR_BAD_LENGTH
        within(out[::2], want[::2].double().cpu(), 4 * BF16 * (1 + want[::2].double().cpu().abs()))


def test_captured_decodes_of_split_units_replay():
    """Two graphs of one context with units in many pieces, whose lengths change between replays."""
    g, rng = gen(44), np.random.default_rng(44)
    hq, hkv, d, bs = 8, 1, 128, 16
    table, pool = ref.sequences(rng, [4000], bs)
    kp, vp, sc = (x.cuda() for x in ref.random_cache(g, pool, bs, hkv, d, torch.float8_e4m3fn))
    table = table.cuda()
    q = torch.randn((1, 3, hq, d), generator=g).bfloat16().cuda()
    ctx, other = (ctx_of(hq, hkv, d, bs, max_seqs=3) for _ in range(2))
    lens = torch.tensor([3999], dtype=torch.int32).cuda()
    outs = [torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    last = q[:, 2].contiguous()
    with torch.cuda.graph(graphs[0], stream=side):
        ctx.decode(last, kp, vp, table, lens, scales=sc, out=outs[0])
    with torch.cuda.graph(graphs[1], stream=side):
        ctx.decode_multi(q, kp, vp, table, lens, scales=sc, out=outs[1])
    for n in (3999, 4000, 0, 1, 700, 2500):
        lens.fill_(n)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for i in (0, 1, 0, 1, 1, 0):
                graphs[i].replay()
        side.synchronize()
        assert torch.equal(outs[0], other.decode(last, kp, vp, table, lens, scales=sc))
        assert torch.equal(outs[1], other.decode_multi(q, kp, vp, table, lens, scales=sc))
        want, size = ref.decode64(q.cpu(), kp.cpu(), vp.cpu(), sc.cpu(), table.cpu(), [n], bs)
        within(outs[1], want, BF16 * want.abs() + 2 * DECODE * size)
    assert ctx.read_device_errors() == 0 and other.read_device_errors() == 0


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("hq,d", [(4, 64), (8, 128)])
def test_decode_after_thousands_of_zero_values(dtype, hq, d):
    """Rows of scale 0 count in the softmax's sum and add nothing, however many there are before the first value: every
    unit whole in one CTA, whose weights of thousands of such rows add up."""
    g, rng = gen(41), np.random.default_rng(41)
    batch, hkv, bs, n = 400, 1, 16, 6000
    table, pool = ref.sequences(rng, [n], bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    blocks = table[0].long()
    vp.view(torch.uint8)[blocks[:-8]] = 0
    sc[blocks[:-8], :, 1] = 0
    # scores 0 for 256 tokens, then 5.4 (7.8 in base 2): the weights after the first stages stay short of a new reference
    q = torch.ones((1, hq, d), dtype=torch.bfloat16)
    kp[:] = torch.ones((), dtype=torch.float32).to(dtype)
    sc[blocks, :, 0] = 5.4 / d ** 0.5
    sc[blocks[:16], :, 0] = 0
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=batch)
    out = ctx.decode(q.repeat(batch, 1, 1).cuda(), kp.cuda(), vp.cuda(), table.repeat(batch, 1).cuda(),
                     torch.full((batch,), n, dtype=torch.int32).cuda(), scales=sc.cuda(), out_dtype=torch.float32)
    want, size = ref.decode64(q[:, None], kp, vp, sc, table, [n], bs)
    for b in range(0, batch, 57):
        within(out[b:b + 1], want[:, 0], DECODE * size[:, 0])
    assert ctx.read_device_errors() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [torch.bfloat16] + ref.FORMATS)
def test_a_layer_step_by_step(dtype):
    """A prompt appended, decoded token by token with the cache growing, and read back: the same as attention over
    everything that was written."""
    g = gen(20)
    B, hq, hkv, d, bs, steps = 3, 8, 2, 128, 16, 4
    prompts = [5, 33, 16]
    ctx = ctx_of(hq, hkv, d, bs)
    width = 4
    table = torch.randperm(B * width, generator=g).int().reshape(B, width).cuda()
    kp, vp, sc = ctx.new_cache(B * width, dtype)
    cs = pda.rope_table(width * bs, d)
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    prep = dict(q_weight=wq, k_weight=wk, cos_sin=cs)
    starts = torch.tensor([0] + list(np.cumsum(prompts)), dtype=torch.int32).cuda()
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    qkv = qkv_of(g, sum(prompts), hq, hkv, d)
    ctx.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, table, lens, scales=sc, starts=starts, **prep)
    for _ in range(steps):
        lens += 1
        qkv = qkv_of(g, B, hq, hkv, d)
        q = ctx.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, table, lens, scales=sc, q=qkv[:, :hq], **prep)
        out = ctx.decode(q, kp, vp, table, lens, scales=sc)
    assert ctx.read_device_errors() == 0
    want, size = ref.decode64(q[:, None].cpu(), kp.cpu(), vp.cpu(), None if sc is None else sc.cpu(), table.cpu(),
                              lens.tolist(), bs)
    within(out, want[:, 0], BF16 * want[:, 0].abs() + 2 * DECODE * size[:, 0])
    k, v = ctx.read_cache(kp, vp, table, lens, scales=sc)
    again = ctx.decode_contiguous(q, k, v, lens)
    # read-back rounds to bf16: 2^-8 of every value, and scores off by 2^-8 |q||k| at most
    assert (again.float() - out.float()).abs().max() < 0.05


@pytest.mark.parametrize("dtype", ref.FORMATS)
def test_a_captured_step_replays(dtype):
    """Append and decode captured into one graph: replays read the buffers' contents of the moment and repeat to the
    bit, beside eager calls of another context on another stream."""
    g = gen(40)
    B, hq, hkv, d, bs = 5, 8, 2, 128, 16
    ctx, other = (ctx_of(hq, hkv, d, bs) for _ in range(2))
    table = torch.randperm(B * 3, generator=g).int().reshape(B, 3).cuda()
    caches = [ctx.new_cache(B * 3, dtype) for _ in range(2)]
    for kp, vp, sc in caches:  # the same contents
        k0, v0, s0 = ref.random_cache(gen(41), B * 3, bs, hkv, d, dtype)
        kp.copy_(k0), vp.copy_(v0), sc.copy_(s0)
    qkv = qkv_of(g, B, hq, hkv, d)
    cs = pda.rope_table(48, d)
    lens = torch.tensor([7, 17, 30, 1, 45], dtype=torch.int32).cuda()
    q_out, out = (torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(c, cache, stream=None):
        kp, vp, sc = cache
        c.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, table, lens, scales=sc, q=qkv[:, :hq], q_out=q_out,
                 cos_sin=cs, stream=stream)
        return c.decode(q_out, kp, vp, table, lens, scales=sc, out=out, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ctx, caches[0])
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(ctx, caches[0])
    for i in range(3):
        qkv.copy_(qkv_of(g, B, hq, hkv, d))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
            first = out.clone()
            graph.replay()
        side.synchronize()
        assert torch.equal(out, first)
        replayed = out.clone()
        out.zero_()
        assert torch.equal(step(other, caches[1]), replayed)
        assert torch.equal(caches[0][0].view(torch.uint8), caches[1][0].view(torch.uint8))
        lens += 1
    assert ctx.read_device_errors() == 0 and other.read_device_errors() == 0


def test_decode_more_rows_than_a_launch_holds():
    """1100 sequences (two launches), and 300 of 5 queries each."""
    g, rng = gen(50), np.random.default_rng(50)
    hq, hkv, d, bs = 4, 2, 64, 8
    for B, q_len in ((1100, 1), (300, 5)):
        lens = [int(x) for x in rng.integers(0, 40, B)]
        table, pool = ref.sequences(rng, lens, bs)
        kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.float8_e4m3fn)
        q = torch.randn((B, q_len, hq, d), generator=g).bfloat16()
        ctx = ctx_of(hq, hkv, d, bs, max_seqs=B * q_len)
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        args = (kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
        if q_len == 1:
            ctx.decode(q[:, 0].cuda(), *args, scales=sc.cuda(), out=out[:, 0])
        else:
            ctx.decode_multi(q.cuda(), *args, scales=sc.cuda(), out=out)
        want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
        within(out, want, DECODE * size)
        assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_values_before_keys(d):
    """V's pool below K's in memory, and K and V in one pool, give the same bits as any other placement."""
    g, rng = gen(60), np.random.default_rng(60)
    hq, hkv, bs, lens = 4, 2, 16, [100, 33, 5]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.int8)
    q = torch.randn((3, hq, d), generator=g).bfloat16().cuda()
    rest = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    ctx = ctx_of(hq, hkv, d, bs)
    both = torch.stack([kp, vp]).cuda()
    want = ctx.decode(q, both[0], both[1], *rest, scales=sc.cuda())
    both = torch.stack([vp, kp]).cuda()
    assert torch.equal(ctx.decode(q, both[1], both[0], *rest, scales=sc.cuda()), want)
    same = sc.clone()
    same[:, :, 0] = sc[:, :, 1]
    got = ctx.decode(q, both[0], both[0], *rest, scales=same.cuda(), out_dtype=torch.float32)
    ref_out, size = ref.decode64(q[:, None].cpu(), vp, vp, same, table, lens, bs)
    within(got, ref_out[:, 0], DECODE * size[:, 0])


@pytest.mark.parametrize("dtype", ref.FORMATS)
def test_offsets_past_32_bits(dtype):
    """A pool whose last blocks lie past 2^31 elements: written, decoded and read back there."""
    hq, hkv, d, bs = 4, 8, 128, 16
    blocks = (1 << 31) // (bs * hkv * d) + 3
    ctx = ctx_of(8, hkv, d, bs)
    kp, vp, sc = ctx.new_cache(blocks, dtype)
    g = gen(70)
    qkv = qkv_of(g, 40, 8, hkv, d)
    table = torch.tensor([[blocks - 1, 0, blocks - 3]], dtype=torch.int32).cuda()
    lens = torch.tensor([40], dtype=torch.int32).cuda()
    q = ctx.append(qkv[:, 8:16], qkv[:, 16:], kp, vp, table, lens, scales=sc, q=qkv[:, :8])
    k, v = ctx.read_cache(kp, vp, table, lens, scales=sc, out_dtype=torch.float32)
    codes, scale = ref.codes32(qkv[:, 16:], dtype)
    assert torch.equal(v[0, :40].cpu(), codes.float() * scale[..., None])
    out = ctx.decode(q[-1:].contiguous(), kp, vp, table, lens, scales=sc, out_dtype=torch.float32)
    near = [t.cpu()[:, [0]] for t in (k, v)]
    small = [pool[[blocks - 1, 0, blocks - 3]].cpu() if dtype == torch.int8 else
             pool.view(torch.uint8)[[blocks - 1, 0, blocks - 3]].cpu().view(dtype) for pool in (kp, vp)]
    want, size = ref.decode64(q[-1:][:, None].cpu(), *small, sc[[blocks - 1, 0, blocks - 3]].cpu(),
                              torch.tensor([[0, 1, 2]]), [40], bs)
    within(out, want[:, 0], DECODE * size[:, 0])
    assert ctx.read_device_errors() == 0 and near


def test_bound_calls_and_closed_contexts():
    ctx = ctx_of(4, 2, 64, 16)
    kp, vp, sc = ctx.new_cache(2, torch.int8)
    qkv = qkv_of(gen(80), 2, 4, 2, 64)
    table, lens = torch.tensor([[0], [1]], dtype=torch.int32).cuda(), torch.tensor([3, 9], dtype=torch.int32).cuda()
    put = ctx.bind_append(qkv[:, 4:6], qkv[:, 6:], kp, vp, table, lens, scales=sc, q=qkv[:, :4])
    q = put()
    run = ctx.bind_decode(q, kp, vp, table, lens, torch.empty_like(q), scales=sc)
    assert torch.equal(run(), ctx.decode(q, kp, vp, table, lens, scales=sc))
    for bad in (dict(scales=None), dict(scales=sc[:1]), dict(scales=sc.double()), dict(scales=sc.cpu())):
        with pytest.raises(ValueError):
            ctx.decode(q, kp, vp, table, lens, **bad)
    with pytest.raises(ValueError):
        ctx.decode(q, kp.float(), vp.float(), table, lens, scales=sc)
    with pytest.raises(ValueError):
        ctx.append(qkv[:, 4:6], qkv[:, 6:], kp, vp.view(torch.uint8), table, lens, scales=sc)
    with pytest.raises(ValueError):
        ctx.norm_rope(qkv[:, :4], qkv[:, 4:6], cos_sin=pda.rope_table(4, 64))
    with pytest.raises(ValueError):
        ctx.read_cache(kp, vp, table, lens, scales=sc, starts=torch.zeros(3, dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        ctx.new_cache(1, torch.float16)
    ctx.close()
    with pytest.raises(pda.PdaError):
        run()
    with pytest.raises(pda.PdaError):
        put()
