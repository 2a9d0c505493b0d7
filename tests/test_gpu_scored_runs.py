"""Scored decode, shared prefixes and eviction as a server runs them: captured and replayed, on other streams, beside
another context, in batches of several launches, and with NaN and infinity where nobody may look.  Tolerances are those
of the operators' own tests; two runs of the same call agree to the bit."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_05_gb300 as pda
import scored_ref as ref
from test_gpu_scored import BF16, ctx_of, formats, gen, inputs, product, up, within

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


# ------------------------------------------------------------------ captured

def rig(dtype, seed=3):
    """Five sequences that share 6 blocks, decoded with 2 queries, and a call of each operator over them."""
    hq, hkv, d, bs, n = 8, 2, 128, 16, 2
    own = [40, 2, 17, 30, 9]
    table, lens, pool = ref.shared_table(np.random.default_rng(seed), own, bs, [0, 5], [6])
    g = gen(seed)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((5, n, hq, d), generator=g).bfloat16()
    slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq)
    return hq, hkv, d, bs, n, table, lens, pool, cache, q, slopes


@formats
@pytest.mark.parametrize("op", ["scored", "weights", "shared"])
def test_captured_decodes_replay(dtype, op):
    """Two graphs of one context and one scratch, whose inputs change between replays, beside eager calls of another
    context on another stream."""
    hq, hkv, d, bs, n, table, lens, pool, cache, q, slopes = rig(dtype)
    ctx, other = (ctx_of(hq, hkv, d, bs) for _ in range(2))
    kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
    ln, sh = i32(lens), i32([6])
    # (sums of tokens that no two sequences share: the shared blocks are copied for them)
    if op == "weights":
        width = t.shape[1]
        big = [x.new_zeros((5 * width, *x.shape[1:])) for x in (raw(kp), raw(vp))]
        bsc = None if sc is None else sc.new_zeros((5 * width, *sc.shape[1:]))
        for b in range(5):
            for x, y in zip((raw(kp), raw(vp)), big):
                y[b * width:(b + 1) * width] = x[t[b].long()]
            if sc is not None:
                bsc[b * width:(b + 1) * width] = sc[t[b].long()]
        kp, vp = (x.view(c.dtype) for x, c in zip(big, (kp, vp)))
        sc, pool = bsc, 5 * width
        t = torch.arange(pool, dtype=torch.int32, device="cuda").view(5, width)
    start = torch.rand((pool, hkv, bs), generator=gen(1)).cuda()
    kw = dict(softcap=8.0, alibi_slopes=sl, scales=sc)

    def bind(c, x, out, weights, scratch, stream=None):
        if op == "shared":
            return c.bind_decode_shared(x, kp, vp, t, ln, sh, out, scratch=scratch, stream=stream, **kw)
        if op == "weights":
            return c.bind_decode_scored(x, kp, vp, t, ln, out, weights=weights, weights_from=start, scratch=scratch,
                                        stream=stream, **kw)
        return c.bind_decode_scored(x, kp, vp, t, ln, out, stream=stream, **kw)

    side = torch.cuda.Stream()
    scratch = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    q1 = qq[:, 1].contiguous()
    outs = [torch.empty_like(q1), torch.empty_like(qq)]
    sums = [start.clone() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, x, out, w in zip(graphs, (q1, qq), outs, sums):
        with torch.cuda.graph(graph, stream=side):
            bind(ctx, x, out, w, scratch)()
    eager = [torch.empty_like(o) for o in outs]
    esums = [torch.empty_like(start) for _ in range(2)]
    calls = [bind(other, x, out, w, None) for x, out, w in zip((q1, qq), eager, esums)]
    for step in range(4):
        ln.copy_(i32([max(0, L - 7 * step * (i + 1)) for i, L in enumerate(lens)]))
        sh.fill_([6, 4, 0, 6][step])
        qq.copy_(torch.randn(qq.shape, generator=gen(10 + step)))
        q1.copy_(qq[:, 1])
        start.copy_(torch.rand(start.shape, generator=gen(step)))
        for w in sums + esums:
            w.copy_(start)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for i in (0, 1, 0, 1, 1, 0):
                graphs[i].replay()
        for call in calls:
            call()
        torch.cuda.synchronize()
        for a, b in zip(outs + sums, eager + esums):
            assert torch.equal(a, b)
        want, size, _ = ref.scored64(qq.cpu(), *(None if c is None else c.cpu() for c in (kp, vp, sc)), t.cpu(), ln.tolist(),
                                     bs, softcap=8.0, slopes=slopes)
        within(outs[1], want, BF16 * want.abs() + product(dtype) * size)
    assert ctx.read_device_errors() == 0 and other.read_device_errors() == 0


@formats
@pytest.mark.parametrize("place", ["in", "out"])
def test_captured_evictions_replay(dtype, place):
    hkv, d, bs, lens, keep = 2, 128, 16, [300, 40, 129], 64
    most = [300, 100, 129]  # of the steps below
    table, pool = ref.ref.sequences(np.random.default_rng(0), most, bs, spare=12)
    used = set(int(table[b, j]) for b, n in enumerate(most) for j in range(-(-n // bs)))
    ot = torch.tensor([i for i in range(pool) if i not in used][:12], dtype=torch.int32).view(3, 4).cuda()
    ctx, other = (ctx_of(hkv, hkv, d, bs) for _ in range(2))
    t, ln, side = table.cuda(), i32(lens), torch.cuda.Stream()
    bufs = []
    for _ in range(2):
        bufs.append(tuple(up(*ref.random_cache(gen(0), pool, bs, hkv, d, dtype), torch.zeros((pool, hkv, bs)))))

    def run(c, buf, kept, new):
        kp, vp, sc, w = buf
        return c.evict(kp, vp, w, t, ln, keep, first=2, recent=8, scales=sc, out_table=ot if place == "out" else None,
                       kept=kept, new_lens=new)

    kept, new = torch.empty((3, hkv, keep), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(ctx, bufs[0], kept, new)
    for step in range(3):
        fresh = up(*ref.random_cache(gen(step), pool, bs, hkv, d, dtype), torch.rand((pool, hkv, bs), generator=gen(step)))
        for buf in bufs:
            for x, y in zip(buf, fresh):
                if x is not None:
                    raw(x).copy_(raw(y))
        ln.copy_(i32([300 - 100 * step, 40 + 30 * step, 129 - 64 * step]))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        new2, kept2 = run(other, bufs[1], None, None)
        torch.cuda.synchronize()
        assert torch.equal(kept, kept2) and torch.equal(new, new2)
        for x, y in zip(*bufs):
            assert x is None or torch.equal(raw(x), raw(y))
        want = ref.evict64(fresh[3].cpu(), table, ln.tolist(), bs, keep, 2, 8)
        assert [[[i for i in h if i >= 0] for h in b] for b in kept.tolist()] == want
    assert ctx.read_device_errors() == 0 and other.read_device_errors() == 0


def test_calls_of_a_stream_follow_each_other():
    """A long row of calls without a synchronisation between them, every one reading what the one before wrote."""
    hq, hkv, d, bs, lens = 8, 2, 64, 16, [500, 70, 260]
    _, table, pool, cache, q, _ = inputs(4, torch.bfloat16, hq, hkv, d, bs, lens, 1)
    kp, vp, _, t, qq = up(*cache, table, q)
    outcome = []
    for stream in (None, torch.cuda.Stream()):
        ctx = ctx_of(hq, hkv, d, bs)
        k, v, w = kp.clone(), vp.clone(), ctx.new_weights(pool)
        ln, x = i32(lens), qq.clone()
        torch.cuda.synchronize()
        for keep in (200, 120, 60, 59):
            for _ in range(3):
                out = ctx.decode_scored(x, k, v, t, ln, weights=w, softcap=10.0, stream=stream)
            with torch.cuda.stream(stream or torch.cuda.current_stream()):
                x = out
            ln, _ = ctx.evict(k, v, w, t, ln, keep, first=1, recent=5, stream=stream)
            one = ctx.decode_shared(x, k, v, t, ln, i32([0]), stream=stream)
            if stream:
                stream.synchronize()
        torch.cuda.synchronize()
        assert ctx.read_device_errors() == 0
        outcome.append((one.cpu(), w.cpu(), ln.cpu(), k.cpu()))
    for a, b in zip(*outcome):
        assert torch.equal(a, b)


def test_timing_events_stand_around_each_decode():
    hq, hkv, d, bs, lens = 8, 2, 64, 16, [100, 7]
    _, table, pool, cache, q, _ = inputs(4, torch.bfloat16, hq, hkv, d, bs, lens, 1)
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, _, t, qq = up(*cache, table, q)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    ctx.set_timing_events(*ev)
    for call in (lambda: ctx.decode_scored(qq, kp, vp, t, i32(lens), weights=ctx.new_weights(pool)),
                 lambda: ctx.decode_shared(qq, kp, vp, t, i32(lens), i32([0]))):
        call()
        torch.cuda.synchronize()
        assert 0 < ev[0].elapsed_time(ev[1]) and ev[0].elapsed_time(ev[1]) <= ev[0].elapsed_time(ev[2]) < 1000
    ctx.set_timing_events()


# ------------------------------------------------------------------ several launches

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("B,n,G", [(1500, 1, 2), (150, 20, 4), (90, 37, 5), (600, 2, 8), (1100, 3, 8)])
def test_batches_of_several_launches(dtype, B, n, G):
    hkv, d, bs = 2, 64, 16
    hq = G * hkv
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 60, B)]
    _, table, pool, cache, q, slopes = inputs(B, dtype, hq, hkv, d, bs, lens, n)
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=B * n)
    kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
    w = ctx.new_weights(pool)
    got = ctx.decode_scored(qq, kp, vp, t, i32(lens), weights=w, alibi_slopes=sl, scales=sc)
    want, size, sums = ref.scored64(q, *cache, table, lens, bs, slopes=slopes)
    within(got, want, BF16 * want.abs() + product(dtype) * size)
    after, added = ref.add_sums(torch.zeros(w.shape), sums, table, lens, bs, n)
    within(w, after, 2.0 ** -10 * added.clamp(min=0) + 2.0 ** -22 * after)
    assert ctx.read_device_errors() == 0


@formats
@pytest.mark.parametrize("B,n,groups", [(1300, 1, 3), (120, 20, 40), (70, 1, 70), (600, 2, 1)])
def test_groups_across_launches(dtype, B, n, groups):
    """Groups that a launch's end divides, more groups than a plan in shared memory holds, groups of one sequence."""
    hq, hkv, d, bs = 8, 2, 64, 16
    rng = np.random.default_rng(B)
    own = [int(x) for x in rng.integers(n, n + 40, B)]
    starts = [0] + sorted(int(x) for x in rng.integers(0, B + 1, groups - 1)) + [B]
    shared = [int(x) for x in rng.integers(0, 9, groups)]
    if groups == B:
        starts = list(range(B + 1))
    table, lens, pool = ref.shared_table(rng, own, bs, starts, shared)
    g = gen(B)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((B, n, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=B * n)
    kp, vp, sc, t, qq = up(*cache, table, q)
    want, size, _ = ref.scored64(q, *cache, table, lens, bs)
    got = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32(shared), starts=i32(starts), scales=sc)
    within(got, want, BF16 * want.abs() + product(dtype) * size)
    assert ctx.read_device_errors() == 0


# ------------------------------------------------------------------ what nobody may look at

@formats
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (256, 8), (128, 2)])
def test_nan_behind_every_length(dtype, d, bs):
    """NaN and infinity (8-bit: NaN scales, and codes where there are such) in every slot that holds no token, and in
    blocks of no sequence."""
    hq, hkv, n = 6, 2, 2
    own = [5, 40, 3, 19]
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, [0, 4], [9])
    g = gen(d)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    if dtype is torch.bfloat16:
        dirty = [c.clone().fill_(x) for c, x in zip(cache, (float("nan"), float("inf")))] + [None]
    else:
        dirty = [raw(c).clone().fill_(0x7f).view(dtype) for c in cache[:2]] + [torch.full_like(cache[2], float("nan"))]
    for b, L in enumerate(lens):
        at = torch.arange(L)
        block = table[b].long()[at // bs]
        for x, y in zip(cache[:2], dirty):
            raw(y)[block, at % bs] = raw(x)[block, at % bs]
        if cache[2] is not None:
            dirty[2][block, :, :, at % bs] = cache[2][block, :, :, at % bs]
    q = torch.randn((4, n, hq, d), generator=g).bfloat16()
    got = []
    for kp, vp, sc in (up(*cache), up(*dirty)):
        ctx = ctx_of(hq, hkv, d, bs)
        t, qq = up(table, q)
        got.append((ctx.decode_shared(qq, kp, vp, t, i32(lens), i32([9]), softcap=5.0, scales=sc),
                    ctx.decode_scored(qq, kp, vp, t, i32(lens), softcap=5.0, scales=sc)))
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_reaches_only_those_who_see_it(d):
    """A NaN key and an infinite value late in a shared prefix: sequences that end before them, and other groups, do not
    notice; the others get NaN, as alone."""
    hq, hkv, bs, n = 8, 2, 16, 1
    own = [5, 40, 3, 19, 8, 1]
    starts, shared = [0, 4, 6], [20, 7]
    table, lens, pool = ref.shared_table(np.random.default_rng(d), own, bs, starts, shared)
    lens[1], lens[2] = 250, 0  # (end before token 300)
    g = gen(d)
    cache = ref.random_cache(g, pool, bs, hkv, d, torch.bfloat16)
    q = torch.randn((6, hq, d), generator=g).bfloat16()
    ctx = ctx_of(hq, hkv, d, bs)
    kp, vp, t, qq = up(*cache[:2], table, q)
    clean = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32(shared), starts=i32(starts))
    kp[table[0, 18].long(), 12, 0, 3] = float("nan")   # token 300, kv head 0
    vp[table[0, 19].long(), 1, 1, 5] = float("inf")    # token 305, kv head 1
    out = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32(shared), starts=i32(starts))
    for b in (1, 2, 4, 5):
        assert torch.equal(out[b], clean[b])
    for b in (0, 3):
        assert torch.isnan(out[b, :hq // 2]).all()
        assert not torch.isfinite(out[b, hq // 2:, 5]).any()
        rest = [i for i in range(d) if i != 5]
        assert torch.equal(out[b, hq // 2:, rest], clean[b, hq // 2:, rest])
    alone = ctx.decode_scored(qq, kp, vp, t, i32(lens))
    assert bool((torch.isfinite(alone) == torch.isfinite(out)).all())


def test_a_context_serves_several_shapes():
    """One context, caches of every format in turn, the same outputs each time round."""
    hq, hkv, d, bs, lens = 8, 2, 128, 16, [200, 31]
    ctx = ctx_of(hq, hkv, d, bs)
    seen = {}
    for turn in range(2):
        for dtype in ref.FORMATS:
            _, table, pool, cache, q, slopes = inputs(5, dtype, hq, hkv, d, bs, lens, 2)
            kp, vp, sc, t, qq, sl = up(*cache, table, q, slopes)
            for k in (1, 2):
                out = (ctx.decode_scored(qq[:, :k].contiguous(), kp, vp, t, i32(lens), softcap=4.0, alibi_slopes=sl, scales=sc),
                       ctx.decode_shared(qq[:, :k].contiguous(), kp, vp, t, i32(lens), i32([0, 0]), scales=sc))
                if turn:
                    assert all(torch.equal(a, b) for a, b in zip(out, seen[dtype, k]))
                seen[dtype, k] = out
    assert ctx.read_device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_long_prefix_again_and_again(dtype):
    """One q tile for both of the prefix kernel's streams, over caches that do not fit L2 together: thousands of calls, all
    alike (a copy that lands late must not be taken for one that has)."""
    hq, hkv, d, bs = 32, 8, 128, 16
    own, prefix = [17, 40, 5, 100], 1024  # blocks
    runs = []
    for seed in range(2):
        table, lens, pool = ref.shared_table(np.random.default_rng(seed), own, bs, [0, 4], [prefix])
        ctx = ctx_of(hq, hkv, d, bs)
        g = torch.Generator("cuda").manual_seed(seed)
        kp, vp, sc = ctx.new_cache(pool, dtype)
        for x in (kp, vp):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if sc is not None:
            sc.copy_(torch.rand(sc.shape, generator=g, device="cuda") + 0.5)
        q = torch.randn((4, hq, d), generator=g, device="cuda").bfloat16()
        out = torch.empty_like(q)
        runs.append((ctx, ctx.bind_decode_shared(q, kp, vp, table.cuda(), i32(lens), i32([prefix]), out, scales=sc), out,
                     ctx.decode_scored(q, kp, vp, table.cuda(), i32(lens), scales=sc)))
    first = [call().clone() for _, call, _, _ in runs]
    for (_, _, _, alone), x in zip(runs, first):
        assert torch.isfinite(x).all() and (x.float() - alone.float()).abs().max() < 0.05
    for _ in range(20):
        for _ in range(150):
            for _, call, _, _ in runs:
                call()
        for (ctx, _, out, _), x in zip(runs, first):
            assert torch.equal(out, x)
    assert all(ctx.read_device_errors() == 0 for ctx, _, _, _ in runs)


def test_calls_at_once():
    """Three contexts on three streams at once, each with scratch of its own: the outputs of each alone."""
    hq, hkv, d, bs = 16, 4, 128, 16
    own = [30, 200, 7, 90, 64, 11]
    jobs = []
    for i, dtype in enumerate((torch.bfloat16, torch.float8_e4m3fn, torch.bfloat16)):
        table, lens, pool = ref.shared_table(np.random.default_rng(i), own, bs, [0, 6], [200])
        ctx = ctx_of(hq, hkv, d, bs)
        kp, vp, sc = up(*ref.random_cache(gen(i), pool, bs, hkv, d, dtype))
        q = torch.randn((6, hq, d), generator=gen(i)).bfloat16().cuda()
        t, ln, out = table.cuda(), i32(lens), torch.empty_like(q)
        stream = torch.cuda.Stream()
        if i < 2:
            args, bind = (q, kp, vp, t, ln, i32([200]), out), ctx.bind_decode_shared
        else:
            args, bind = (q, kp, vp, t, ln, out), ctx.bind_decode_scored
        alone = bind(*args, scales=sc, softcap=20.0)().clone()
        torch.cuda.synchronize()
        jobs.append((ctx, bind(*args, scales=sc, softcap=20.0, stream=stream), out, alone))
    for _ in range(10):
        for _ in range(50):
            for _, call, _, _ in jobs:
                call()
        torch.cuda.synchronize()
        for ctx, _, out, alone in jobs:
            assert torch.equal(out, alone) and ctx.read_device_errors() == 0
            out.zero_()
        torch.cuda.synchronize()
