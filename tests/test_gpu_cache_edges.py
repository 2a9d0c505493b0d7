"""Operators around the decode at the edges of what their documentation allows: other streams, scales and rows of any
size, masked places that hold NaN, against fp64 definitions."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import paged_gqa_decode_05_gb300 as pda

pytestmark = pytest.mark.gpu


def ctx_of(hq, hkv, d, bs, max_seqs=64):
    return pda.Context(max_seqs=max_seqs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)


def gen(seed):
    return torch.Generator().manual_seed(seed)


BF16 = 2.0 ** -8
DECODE = 2.0 ** -10  # of sum p |v|: rounded weights and what fp32 arithmetic adds


def within(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - tol
    assert off.max() <= 0, f"{off.max()} beyond its tolerance at {np.unravel_index(int(off.argmax()), off.shape)}"


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("handle", [False, True])
def test_calls_on_another_stream_make_their_outputs_there(handle):
    """Work queued on the current stream does not touch what a call on another stream returned: rows read back stay,
    and rows of no token stay zero."""
    rng, g = np.random.default_rng(1), gen(1)
    hq, hkv, d, bs, lens = 4, 2, 64, 16, [37, 0, 20]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = (t.cuda() for t in ref.random_cache(g, pool, bs, hkv, d, torch.int8))
    table, lens_d = table.cuda(), i32(lens)
    q = torch.randn((3, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    want = ctx.read_cache(kp, vp, table, lens_d, scales=sc)
    want_o = ctx.decode(q, kp, vp, table, lens_d, scales=sc)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # what comes behind this on the current stream comes late
    stream = side.cuda_stream if handle else side
    got = ctx.read_cache(kp, vp, table, lens_d, scales=sc, stream=stream)
    out = ctx.decode(q, kp, vp, table, lens_d, scales=sc, stream=stream)
    side.synchronize()
    for _ in range(2):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(out, want_o)
        torch.cuda.synchronize()
    assert ctx.read_device_errors() == 0


def test_calls_on_the_default_streams_handle():
    """stream=0 is the default stream, also for what the call makes itself, while another stream is current."""
    g = gen(1)
    ctx = ctx_of(4, 2, 64, 16)
    kp, vp, sc = (t.cuda() for t in ref.random_cache(g, 4, 16, 2, 64, torch.int8))
    table, lens = i32([[0, 1], [2, 3]]), i32([20, 9])
    want = ctx.read_cache(kp, vp, table, lens, scales=sc)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20_000_000)
        got = ctx.read_cache(kp, vp, table, lens, scales=sc, stream=0)
    torch.cuda.default_stream().synchronize()
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        torch.cuda.synchronize()


# ------------------------------------------------------------------ NaN that a query does not see

SHAPES = [(4, 2, 64, 16), (8, 2, 128, 16), (8, 1, 128, 4), (4, 1, 256, 32), (16, 2, 64, 1), (8, 1, 128, 64)]


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("q_len", [2, 3, 4])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("which", [0, 1])
def test_a_later_tokens_nan_row_stays_with_the_queries_that_see_it(dtype, q_len, hq, hkv, d, bs, which):
    """A drafted token whose key or value holds an infinity (a row of scale NaN): the queries before it keep their
    bits, the query that sees it is NaN."""
    rng, g = np.random.default_rng(q_len), gen(d + bs)
    lens = [q_len, 41, 128, 300, 1000]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = (t.cuda() for t in ref.random_cache(g, pool, bs, hkv, d, dtype))
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    rest = (table.cuda(), i32(lens))
    want = ctx.decode_multi(q, kp, vp, *rest, scales=sc)
    rows = torch.randn((2, len(lens), hkv, d), generator=g).bfloat16().cuda()
    rows[which, :, :, 5] = float("inf")
    ctx.append(rows[0], rows[1], kp, vp, *rest, scales=sc)
    got = ctx.decode_multi(q, kp, vp, *rest, scales=sc)
    assert torch.equal(got[:, :-1], want[:, :-1]) and torch.isfinite(got[:, :-1]).all()
    assert torch.isnan(got[:, -1]).all()
    assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("q_len", [2, 4, 7])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_a_later_tokens_nan_codes_stay_with_the_queries_that_see_it(q_len, hq, hkv, d, bs):
    """e4m3 codes that read as NaN in some columns of drafted tokens' values: NaN in those columns of the queries that
    see the token, and nowhere else."""
    rng, g = np.random.default_rng(q_len), gen(d + bs)
    lens = [q_len, 41, 128, 300, 1000]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.float8_e4m3fn)
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    rest = (table.cuda(), i32(lens))
    want = ctx.decode_multi(q, kp.cuda(), vp.cuda(), *rest, scales=sc.cuda())
    nan = torch.zeros((len(lens), q_len, hkv, d), dtype=torch.bool)
    for b, n in enumerate(lens):
        for back in (1, 2):  # the last token's columns 3 and d - 1, the one before's column 8
            at = n - back
            cols = [3, d - 1] if back == 1 else [8]
            vp.view(torch.uint8)[table[b, at // bs].long(), at % bs, :, cols] = 0x7f if back == 1 else 0xff
            nan[b, q_len - back:, :, cols] = True
    got = ctx.decode_multi(q, kp.cuda(), vp.cuda(), *rest, scales=sc.cuda())
    nan = nan.repeat_interleave(hq // hkv, 2).cuda()
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ rows of very different size

@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,bs,q_len", [(8, 2, 128, 16, 1), (4, 4, 64, 8, 3), (4, 1, 256, 16, 1), (8, 2, 128, 16, 4)])
@pytest.mark.parametrize("times", [2.0 ** 10, 2.0 ** 12, 2.0 ** 14])
def test_q_with_one_large_element(dtype, hq, hkv, d, bs, q_len, times):
    """A q element `times` the others, on a channel where every key is zero: the others still make the scores.  With
    an e4m3 cache q elements below 2^-14 of the row's largest are off by 2^-22 of it at most, which moves a score by
    scale sum |dq| |k| and a weight by twice the largest such move; else q is as exact as it came."""
    rng, g = np.random.default_rng(3), gen(d)
    lens = [37, 200, 64]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((3, q_len, hq, d), generator=g)
    at = torch.randint(0, d, (3, q_len, hq), generator=g)
    q.scatter_(3, at[..., None], times)
    kp.view(torch.uint8)[...] = torch.where(torch.zeros(d).scatter_(0, at.flatten(), 1.0).bool(), 0, kp.view(torch.uint8))
    q = q.bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    ctx.decode_multi(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(lens), scales=sc.cuda(), out=out)
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
    top = q.double().abs().amax(-1, keepdim=True)
    dq = torch.where(q.double().abs() < 2.0 ** -14 * top, 2.0 ** -22 * top, 0.0)
    moved = torch.zeros(q.shape[:3] + (1,), dtype=torch.float64)
    if dtype == torch.float8_e4m3fn:
        for b, n in enumerate(lens):
            k = ref.rows64(kp, sc, 0, table[b], n, bs).abs().amax(0).repeat_interleave(hq // hkv, 0)
            moved[b] = 2 * d ** -0.5 * (dq[b] * k).sum(-1, keepdim=True)
    within(out, want, (DECODE + moved) * size)
    assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,bs,lens", [
    (8, 2, 128, 16, [2, 37, 200, 5000]), (4, 1, 256, 16, [2, 300, 4000]), (2, 2, 64, 1, [2, 90]), (8, 1, 64, 16, [9001])])
@pytest.mark.parametrize("kind", ["zeros and 2^90", "2^90 and zeros", "any"])
@pytest.mark.parametrize("q_len", [1, 2])
def test_values_of_any_size(dtype, hq, hkv, d, bs, lens, kind, q_len):
    """Value rows of zeros beside rows of 2^90, and of any size from 2^-40 to 2^115: every row counts in the sum of
    weights, whatever its V scale, in whole units and in units of many pieces."""
    rng, g = np.random.default_rng(7), gen(d + len(lens))
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    for b, n in enumerate(lens):
        if kind == "any":
            e = torch.randint(-40, 116, (n, hkv), generator=g)
        else:
            e = torch.where(((torch.arange(n) < (n + 1) // 2) == (kind == "zeros and 2^90"))[:, None], -1000, 90).expand(n, hkv)
        v = torch.randn((n, hkv, d), generator=g).clamp(-4, 4) * torch.exp2(e.double())[..., None].float()
        codes, scale = ref.codes32(v, dtype)
        for at in range(n):
            blk, slot = int(table[b, at // bs]), at % bs
            vp.view(torch.uint8)[blk, slot] = codes.view(torch.uint8)[at]
            sc[blk, :, 1, slot] = scale[at]
    q = 0.3 * torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    ctx.decode_multi(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(lens), scales=sc.cuda(), out=out)
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
    within(out, want, DECODE * size)
    assert ctx.read_device_errors() == 0


# ------------------------------------------------------------------ fp32 outputs

# Of sum p |v|: weights in two fp16 parts 2^-22; the two exponentials of a weight, their arguments (below 2^5, three
# roundings of 2^-24 of them) and log2 of its V scale 2^-18; scores of up to 2^5 in base 2, summed in fp32 over at most
# 16 products' partial sums, 2^-16.  What fp16 flushes is 2^-31 of the largest weight for every code.
FINE = 2.0 ** -15


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,bs,q_len", [(8, 2, 128, 16, 1), (8, 1, 128, 16, 2), (4, 1, 256, 4, 1), (8, 2, 64, 1, 1),
                                               (4, 2, 64, 64, 4)])
@pytest.mark.parametrize("lens", [[2, 3, 5, 9], [33, 64, 100], [5000]])
def test_fp32_outputs_are_unrounded(dtype, hq, hkv, d, bs, q_len, lens):
    rng, g = np.random.default_rng(2), gen(d + q_len)
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    args = (kp.cuda(), vp.cuda(), table.cuda(), i32(lens))
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    ctx.decode_multi(q.cuda(), *args, scales=sc.cuda(), out=out)
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
    heavy = ref.decode64(q, kp, (vp.float().abs()).to(dtype), sc, table, lens, bs)[0]  # sum p |v|
    within(out, want, FINE * heavy + 2.0 ** -10 * (size - heavy))
    # and the bf16 output is its rounding, up to what bf16 outputs' weights lose
    rounded = ctx.decode_multi(q.cuda(), *args, scales=sc.cuda())
    within(rounded, want, BF16 * want.abs() + 2.0 ** -9 * size)


# ------------------------------------------------------------------ timing events

@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("dtype", ref.FORMATS)
def test_timing_events_are_recorded(dtype, q_len):
    """set_timing_events times decodes over 8-bit caches as it does others, one launch or several."""
    g, rng = gen(5), np.random.default_rng(5)
    hq, hkv, d, bs, B = 4, 2, 64, 16, 1100 // q_len
    table, pool = ref.sequences(rng, [40] * B, bs)
    kp, vp, sc = (t.cuda() for t in ref.random_cache(g, pool, bs, hkv, d, dtype))
    q = torch.randn((B, q_len, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=B * q_len)
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in evs:
        e.record()  # creates the underlying events
    torch.cuda.synchronize()
    around = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ctx.set_timing_events(*evs)
    around[0].record()
    ctx.decode_multi(q, kp, vp, table.cuda(), i32([40] * B), scales=sc)
    around[1].record()
    torch.cuda.synchronize()
    assert 0 < evs[0].elapsed_time(evs[1]) <= evs[0].elapsed_time(evs[2]) <= around[0].elapsed_time(around[1])
    assert 0 <= around[0].elapsed_time(evs[0])
    ctx.set_timing_events()


# ------------------------------------------------------------------ one call, any format and layout

def slots_of(kp, vp):
    """The pools as one, [slot, K | V, Hkv, bs, D] (slot_strides)."""
    raw = [p.view(torch.int8 if p.element_size() == 1 else torch.int16).transpose(1, 2) for p in (kp, vp)]
    return torch.stack(raw, 1).contiguous().view(kp.dtype).flatten().cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16] + ref.FORMATS)
@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 128, 16), (4, 4, 64, 4), (4, 1, 256, 8)])
def test_decode_multi_of_other_strides(dtype, q_len, hq, hkv, d, bs):
    """Several queries over the slot layout give the dense pools' bits, in every format; fp32 outputs."""
    rng, g = np.random.default_rng(9), gen(d)
    lens = [37, 200, 3, 0]
    table, pool = ref.sequences(rng, lens, bs)
    if dtype == torch.bfloat16:
        kp, vp = (torch.randn((pool, bs, hkv, d), generator=g).bfloat16() for _ in range(2))
        sc = None
    else:
        kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    scales = None if sc is None else sc.cuda()
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    rest = (table.cuda(), i32(lens))
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs)
    dense = ctx.decode_multi(q.cuda(), kp.cuda(), vp.cuda(), *rest, scales=scales)
    within(dense, want, BF16 * want.abs() + 2 * DECODE * size)
    both = slots_of(kp, vp)
    layout = dict(strides=pda.slot_strides(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs), num_blocks=pool)
    assert torch.equal(ctx.decode_multi(q.cuda(), both, both[hkv * bs * d:], *rest, scales=scales, **layout), dense)
    if dtype == torch.bfloat16 and q_len > 1:
        with pytest.raises(pda.PdaError) as e:
            ctx.decode_multi(q.cuda(), both, both[hkv * bs * d:], *rest, out_dtype=torch.float32, **layout)
        assert e.value.status == pda.ERR_UNSUPPORTED
        return
    fine = ctx.decode_multi(q.cuda(), both, both[hkv * bs * d:], *rest, scales=scales, out_dtype=torch.float32, **layout)
    assert fine.dtype == torch.float32
    within(fine, want, DECODE * size)
    if q_len == 1:
        one = ctx.decode(q[:, 0].contiguous().cuda(), kp.cuda(), vp.cuda(), *rest, scales=scales, out_dtype=torch.float32)
        assert torch.equal(fine[:, 0], one)
    assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("scale", [0.0, 0.3, -0.05, 1.0])
def test_scales_of_the_scores(dtype, scale):
    """A softmax scale other than the default; 0 takes the mean of the values."""
    rng, g = np.random.default_rng(10), gen(10)
    hq, hkv, d, bs, lens = 8, 2, 128, 16, [37, 200, 3, 2000]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = 0.2 * torch.randn((len(lens), 2, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    got = ctx.decode_multi(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(lens), scales=sc.cuda(), scale=scale,
                           out_dtype=torch.float32)
    want, size = ref.decode64(q, kp, vp, sc, table, lens, bs, scale=scale)
    within(got, want, DECODE * size)


# ------------------------------------------------------------------ read_cache

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16] + ref.FORMATS)
def test_read_cache_flags_bad_lengths(dtype, packed):
    """A negative length and one past the table raise their flag, as in decode, and the rest is read."""
    hkv, d, bs = 2, 64, 8
    ctx = ctx_of(2, hkv, d, bs)
    kp, vp, sc = ctx.new_cache(4, dtype)
    kv = torch.randn((32, 2 * hkv, d), generator=gen(3)).bfloat16().cuda()
    table = i32([[0, 1], [2, 3]])
    ctx.append(kv[:, :hkv], kv[:, hkv:], kp, vp, table, i32([16, 16]), scales=sc)
    kw = dict(scales=sc)
    if packed:  # 16 rows each: none asks for more than the table holds
        kw.update(starts=i32([0, 16, 32]))

    def read(lens):
        if packed:
            kw.update({k: torch.full((32, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for k in ("k_out", "v_out")})
        return [x.reshape(2, 16, hkv, d) for x in ctx.read_cache(kp, vp, table, i32(lens), **kw)]

    want = read([16, 16])
    assert ctx.read_device_errors() == 0
    for bad in (-1, -2 ** 31, 17, 2 ** 31 - 1):
        got = read([16, bad])
        assert ctx.read_device_errors() == pda.DEVERR_BAD_LENGTH, bad
        for x, w in zip(got, want):
            assert torch.equal(x[0], w[0])
            assert torch.equal(x[1], w[1] if bad > 0 else torch.full_like(w[1], 3.0 if packed else 0.0))
    read([0, 16])
    assert ctx.read_device_errors() == 0


# ------------------------------------------------------------------ garbage

@pytest.mark.parametrize("dtype", ref.FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bs", [1, 4, 16, 64])
@pytest.mark.parametrize("hq,q_len", [(8, 1), (8, 4), (1, 4)])
@pytest.mark.parametrize("apart", [False, True])
def test_garbage_outside_the_sequences(dtype, d, bs, hq, q_len, apart):
    """NaN codes, NaN and infinite scales behind every end and in blocks of no sequence, ids of no block in the table
    past a sequence's blocks: the output's bits do not change, whichever way the pools load (as one, or each alone)."""
    hkv = 1
    rng, g = np.random.default_rng(bs), gen(d)
    lens = [37, 0, 81, 130, q_len, 64, 1000]
    table, pool = ref.sequences(rng, lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(lens), q_len, hq, d), generator=g).bfloat16().cuda()
    ctx = ctx_of(hq, hkv, d, bs)

    def run(table):
        pools = [p.cuda() for p in (kp, vp)]
        if apart:  # rows wider than the head: no joined loads at head size 256
            wide = torch.zeros((2, pool, bs, hkv, d + 16), dtype=torch.int8, device="cuda")
            for w, p in zip(wide, pools):
                w[..., :d] = p.view(torch.int8)
            pools = [w.view(dtype).flatten() for w in wide]
        return ctx.decode_multi(q, *pools, table.cuda(), i32(lens), scales=sc.cuda(), out_dtype=torch.float32,
                                strides=[s * (d + 16 * apart) for s in (bs * hkv, hkv, 1)], num_blocks=pool)

    want = run(table)
    assert torch.isfinite(want).all()
    live = torch.zeros((pool, bs), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            live[int(table[b, t // bs]), t % bs] = True
        table[b, -(-n // bs):] = torch.tensor([-1, 2 ** 31 - 1, pool]).repeat(table.shape[1])[:table.shape[1] - -(-n // bs)]
    for p in (kp, vp):
        p.view(torch.uint8)[~live] = 0x7f
    sc.permute(0, 3, 1, 2)[~live] = torch.tensor([float("nan"), float("inf")])
    assert torch.equal(run(table), want)
    assert ctx.read_device_errors() == 0
