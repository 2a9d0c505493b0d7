"""Arrays of sums and of lengths that overlap in part are refused, before any device is touched."""
import pytest

import paged_gqa_decode_05_gb300 as pda
from test_cache_ops_cpu import env, lib  # noqa: F401
from test_scored_cpu import evict, scored


@pytest.mark.parametrize("by", [4, 64, 4 * 4 * 2 * 16 - 4])  # (4 blocks of 2 kv heads and 16 slots)
def test_sums_that_overlap_in_part(lib, env, by):  # noqa: F811
    a = env["addr"]
    for w_in, w_out in ((a, a + by), (a + by, a)):
        assert scored(lib, env, w_in=w_in, w_out=w_out) == pda.ERR_INVALID_ARG
    assert b"apart" in lib.pda_last_error()


def test_sums_in_place_and_apart(lib, env):  # noqa: F811
    a, size = env["addr"], 4 * 4 * 2 * 16
    for w_in, w_out in ((a, a), (None, a), (a, a + size), (a + size, a)):
        assert scored(lib, env, w_in=w_in, w_out=w_out) == pda.OK


@pytest.mark.parametrize("by", [-12, -4, 0, 4, 12])
def test_new_lengths_over_the_old_ones(lib, env, by):  # noqa: F811
    a = env["addr"] + 64
    assert evict(lib, env, batch=4, lens=a, new_lens=a + by) == pda.ERR_INVALID_ARG
    assert b"new_lens" in lib.pda_last_error()
