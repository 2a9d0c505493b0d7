"""Eviction by sums of attention weights: exact against its definition, and the operators together."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_05_gb300 as pda
import scored_ref as ref
from test_gpu_scored import BF16, ctx_of, formats, gen, product, up, within

pytestmark = pytest.mark.gpu


def check(dtype, hkv, d, bs, lens, keep, first, recent, place, seed=0, weights=None, strided=False):
    g = gen(seed)
    rng = np.random.default_rng(seed)
    kept_blocks = -(-keep // bs)
    table, pool = ref.ref.sequences(rng, lens, bs, spare=3 + len(lens) * kept_blocks)
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    if weights is None:
        w = torch.rand((pool, hkv, bs), generator=g) * 4
        w = torch.where(torch.rand(w.shape, generator=g) < 0.3, torch.floor(w), w)  # ties, zeros
    else:
        w = weights(torch.rand((pool, hkv, bs), generator=g))
    out_table = None
    if place == "out":
        used = set(int(table[b, j]) for b, n in enumerate(lens) for j in range(-(-max(n, 0) // bs)))
        free = [i for i in rng.permutation(pool) if i not in used]
        out_table = torch.tensor(np.array(free[:len(lens) * kept_blocks]).reshape(len(lens), -1), dtype=torch.int32)
    kept = ref.evict64(w, table, lens, bs, keep, first, recent)
    raw = [c.view(torch.int8) if c.element_size() == 1 else c for c in cache[:2]]
    want = [c.clone() for c in raw] + [w.clone()] + ([] if cache[2] is None else [cache[2].clone()])
    to = table if out_table is None else out_table
    for b, heads in enumerate(kept):
        for h, old in enumerate(heads):
            t, i = torch.tensor(old, dtype=torch.long), torch.arange(len(old))
            src, dst = (table[b].long()[t // bs], t % bs), (to[b].long()[i // bs], i % bs)
            for y, x in zip(want[:2], raw):
                y[dst[0], dst[1], h] = x[src[0], src[1], h]
            want[2][dst[0], h, dst[1]] = w[src[0], h, src[1]]
            if cache[2] is not None:
                want[3][dst[0], h, :, dst[1]] = cache[2][src[0], h, :, src[1]]
    ctx = ctx_of(hkv, hkv, d, bs)
    kp, vp, sc, t, ot, ww = up(*cache, table, out_table, w)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    new, got = ctx.evict(kp, vp, ww, t, ln, keep, first=first, recent=recent, scales=sc, out_table=ot)
    assert ctx.read_device_errors() == 0
    assert new.tolist() == [min(max(n, 0), keep) for n in lens]
    for b, heads in enumerate(kept):
        for h, old in enumerate(heads):
            assert got[b, h].tolist() == old + [-1] * (keep - len(old)), (b, h)
    have = [c.view(torch.int8) if c.element_size() == 1 else c for c in (kp, vp)] + [ww] + ([] if sc is None else [sc])
    for y, x in zip(have, want):
        assert torch.equal(y.cpu().view(torch.int8), x.view(torch.int8))


@formats
@pytest.mark.parametrize("place", ["in", "out"])
@pytest.mark.parametrize("hkv,d,bs,lens,keep,first,recent", [
    (2, 64, 16, [100, 0, 1, 33, 32, 34], 33, 4, 8),
    (8, 128, 16, [700, 129, 600, 64], 128, 0, 0),
    (1, 256, 8, [513, 77], 64, 3, 61),
    (3, 128, 64, [1000, 65, 999], 200, 16, 50),
    (4, 64, 1, [300, 40, 41], 40, 1, 0),
    (2, 128, 4, [90, 8, 7], 7, 0, 7),
    (5, 256, 2, [50, 1, 2], 1, 0, 0),
    (1, 128, 32, [9000, 5], 4000, 4, 100),      # the larger form of the choice
    (2, 64, 16, [60, 61], 1000, 10, 10),        # nothing to cut
])
def test_evict(dtype, place, hkv, d, bs, lens, keep, first, recent):
    check(dtype, hkv, d, bs, lens, keep, first, recent, place, seed=d + keep)


@pytest.mark.parametrize("place", ["in", "out"])
@pytest.mark.parametrize("weights", [
    lambda u: torch.zeros_like(u), lambda u: torch.full_like(u, float("nan")), lambda u: -u,
    lambda u: torch.where(u < 0.3, float("nan"), torch.where(u < 0.5, float("inf"), torch.where(u < 0.7, -0.0, 0.0))),
    lambda u: u * 1e-42, lambda u: torch.where(u < 0.5, -1e30, 1e30) * (u * 8).floor(), lambda u: (u * 1000).floor()],
    ids=["zeros", "nan", "negative", "special", "subnormal", "signs", "ties"])
def test_evict_weights_of_all_kinds(weights, place):
    check(torch.bfloat16, 3, 64, 16, [400, 211, 300], 100, 2, 10, place, seed=7, weights=weights)


def test_evict_more_tokens_than_shared_memory_holds():
    check(torch.int8, 1, 64, 64, [70000, 50000, 3], 30000, 4, 1000, "in", seed=3)
    check(torch.float8_e4m3fn, 2, 64, 64, [60001], 20000, 0, 0, "out", seed=4)


def test_evict_in_place_of_many_units():
    """Units enough for whole rows to a CTA."""
    check(torch.bfloat16, 16, 128, 16, [300 + 13 * i for i in range(20)], 250, 4, 32, "in", seed=5)


def test_evict_bad_blocks_and_lengths():
    ctx = ctx_of(2, 2, 64, 16)
    g = gen(0)
    kp, vp = (torch.randn((8, 16, 2, 64), generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.rand((8, 2, 16), generator=g).cuda()
    table = torch.tensor([[0, 99, 2], [3, 4, 5], [6, 7, 1]], dtype=torch.int32).cuda()
    lens = torch.tensor([48, -5, 100], dtype=torch.int32).cuda()
    before = kp.clone()
    new, kept = ctx.evict(kp, vp, w, table, lens, 40, first=40 - 8, recent=8)
    assert ctx.read_device_errors() == pda.DEVERR_BAD_LENGTH | pda.DEVERR_BAD_BLOCK_ID
    assert new.tolist() == [40, 0, 40]
    assert (kept[1] == -1).all() and kept[0, 0].tolist() == list(range(32)) + list(range(40, 48))
    assert torch.equal(kp[3:6], before[3:6])
    assert torch.equal(kp[2, :8], before[2, 8:])


@formats
def test_together(dtype):
    """Prompts written, queries that sum their weights, the cache cut down, and decoded again with new tokens."""
    hq, hkv, d, bs, lens, keep = 8, 2, 128, 16, [150, 40, 333], 96
    g = gen(11)
    ctx = ctx_of(hq, hkv, d, bs)
    blocks = [-(-(n + 2) // bs) for n in lens]
    order = torch.randperm(sum(blocks) + 2, generator=g).int()
    table = torch.zeros((3, max(blocks)), dtype=torch.int32)
    at = 0
    for b, nb in enumerate(blocks):
        table[b, :nb] = order[at:at + nb]
        at += nb
    kp, vp, sc = ctx.new_cache(len(order), dtype)
    w = ctx.new_weights(len(order))
    w += 77.0  # what other sequences left
    starts = torch.tensor([0, lens[0], lens[0] + lens[1], sum(lens)], dtype=torch.int32).cuda()
    k, v = (torch.randn((sum(lens), hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    t, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ctx.append(k, v, kp, vp, t, ln, scales=sc, starts=starts)
    n = 4
    q = torch.randn((3, n, hq, d), generator=g).bfloat16().cuda()
    zero = torch.zeros_like(w)
    ctx.decode_scored(q, kp, vp, t, ln, weights=w, weights_from=zero, scales=sc)
    host = [x if x is None else x.cpu() for x in (kp, vp, sc)]
    _, _, sums = ref.scored64(q.cpu(), *host, table, lens, bs)
    after, added = ref.add_sums(zero.cpu(), sums, table, lens, bs, n)
    live = added.cuda() >= 0
    within(w[live], after[live.cpu()], (2.0 ** -10 * added + 2.0 ** -22 * after)[live.cpu()])
    sums = w.cpu().clone()
    kept = ref.evict64(sums, table, lens, bs, keep, 4, 16)
    new, got = ctx.evict(kp, vp, w, t, ln, keep, first=4, recent=16, scales=sc)
    for b in range(3):
        for h in range(hkv):
            assert [i for i in got[b, h].tolist() if i >= 0] == kept[b][h]
    # the next step: a new token, and attention over what is left
    new = new + 1
    k1, v1 = (torch.randn((3, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    ctx.append(k1, v1, kp, vp, t, new, scales=sc)
    q1 = torch.randn((3, 1, hq, d), generator=g).bfloat16().cuda()
    out = ctx.decode_scored(q1, kp, vp, t, new, weights=w, scales=sc)
    host = [x if x is None else x.cpu() for x in (kp, vp, sc)]
    want, size, got = ref.scored64(q1.cpu(), *host, table, new.tolist(), bs)
    within(out, want, BF16 * want.abs() + product(dtype) * size)
    # the kept tokens' old sums plus this step's; the new token has its own weight only
    for b in range(3):
        m = int(new[b]) - 1
        for h in range(hkv):
            i = torch.tensor(kept[b][h])
            old = sums[table[b].long()[i // bs], h, i % bs].double()
            j = torch.arange(m)
            have = w.cpu()[table[b].long()[j // bs], h, j % bs].double()
            assert ((have - old - got[b][:m, h]).abs() <= 2.0 ** -10 * got[b][:m, h] + 2.0 ** -22 * old).all()
            last = w.cpu()[table[b, m // bs].long(), h, m % bs].double()
            assert (last - got[b][m, h]).abs() <= 2.0 ** -10 * got[b][m, h]
    assert ctx.read_device_errors() == 0
