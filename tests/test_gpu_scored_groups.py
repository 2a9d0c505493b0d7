"""Groups of a shared prefix that sequences lead which do not share it: empty slots of a batch with a padding row, and
sequences that end inside the prefix.  Tolerances are those of the operators' tests."""
import numpy as np
import pytest
import torch

import scored_ref as ref
from test_gpu_scored import BF16, ctx_of, formats, gen, product, up, within

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# starts, shared blocks, own tokens, and the sequences that share nothing: their length (0: an empty slot).  Of their rows
# only the blocks of their own tokens are filled.
CASES = [
    ([0, 4], [20], [30, 5, 7, 1], {0: 0}),
    ([0, 5], [20], [30, 5, 7, 1, 0], {0: 0, 1: 100, 2: 319, 4: 0}),
    ([0, 3, 6], [4, 30], [3, 1, 2, 9, 40, 8], {0: 0, 3: 17, 4: 0}),
    ([0, 3, 5], [12, 9], [3, 1, 2, 9, 40], {0: 0, 1: 0, 2: 5}),              # nobody of the first group shares
    ([0, 60], [10], [1 + i for i in range(60)], {i: (i * 7) % 160 for i in range(59)}),   # the last one alone does
    ([0, 40, 80], [10, 3], [1 + i % 9 for i in range(80)], {**{i: 0 for i in range(33)}, **{40 + i: 0 for i in range(39)}}),
    ([2 * i for i in range(21)], [1 + i for i in range(20)], [2 + i for i in range(40)], {i: 0 for i in range(0, 40, 3)}),
]


@formats
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("hq,hkv,d,bs,n,pad", [(8, 2, 128, 16, 1, -1), (4, 1, 64, 16, 2, 1 << 20), (4, 2, 256, 4, 1, 0)])
def test_groups_that_others_lead(dtype, case, hq, hkv, d, bs, n, pad):
    """With rows padded by ids outside the pool, which a read would flag, and by block 0, which it would take."""
    starts, shared, own, short = CASES[case]
    rng, g = np.random.default_rng(case), gen(case)
    own = [max(x, n) for x in own]
    table, lens, pool = ref.shared_table(rng, own, bs, starts, shared)
    for b, L in short.items():
        group = int(np.searchsorted(starts, b, side="right")) - 1
        lens[b] = min(L, max(0, shared[group] * bs + n - 2))  # (its first query misses the prefix's last token)
        used = -(-lens[b] // bs)
        table[b, :used] = torch.from_numpy(rng.integers(0, pool, used).astype(np.int32))  # its own blocks, whichever
        table[b, used:] = pad
    cache = ref.random_cache(g, pool, bs, hkv, d, dtype)
    q = torch.randn((len(own), n, hq, d), generator=g).bfloat16()
    want, size, _ = ref.scored64(q, *cache, table.clamp(0, pool - 1), lens, bs)
    ctx = ctx_of(hq, hkv, d, bs, max_seqs=len(own) * n)
    kp, vp, sc, t, qq = up(*cache, table, q)
    for _ in range(2):
        got = ctx.decode_shared(qq, kp, vp, t, i32(lens), i32(shared), starts=i32(starts), scales=sc)
        assert ctx.read_device_errors() == 0
        within(got, want, BF16 * want.abs() + product(dtype) * size)


@formats
@pytest.mark.parametrize("shared", [1 << 25, (1 << 26) + 1, (1 << 26) + 2])
def test_prefixes_past_31_bits_of_tokens(dtype, shared):
    """2^31 and 2^32 + 64 tokens, as a table of that width may be told to share: longer than any sequence, so that all
    are decoded alone, where 32 bits of tokens wrap to a prefix of nothing, one or two blocks."""
    hq, hkv, d, bs, lens = 4, 1, 64, 64, [200]
    g = gen(3)
    cache = ref.random_cache(g, 5, bs, hkv, d, dtype)
    q = torch.randn((1, 1, hq, d), generator=g).bfloat16()
    row = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32)
    want, size, _ = ref.scored64(q, *cache, row, lens, bs)
    kp, vp, sc, qq = up(*cache, q)
    table = torch.zeros((1, (1 << 26) + 8), dtype=torch.int32, device="cuda")
    table[:, :4] = row.cuda()
    ctx = ctx_of(hq, hkv, d, bs)
    got = ctx.decode_shared(qq, kp, vp, table, i32(lens), i32([shared]), scales=sc)
    within(got, want, BF16 * want.abs() + product(dtype) * size)
    assert ctx.read_device_errors() == 0
