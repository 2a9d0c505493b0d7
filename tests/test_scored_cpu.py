"""Scored decode, shared prefixes and eviction on a machine without a GPU: their refusals, all before any device is
touched, what the binding checks, and the fp64 definitions that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import paged_gqa_decode_05_gb300 as pda
import scored_ref as ref
from fake_binding import B, D, HKV, HQ, POOL, SCALES, Tensor, bf16, ctx, f32, heads, i32, pools  # noqa: F401
from test_cache_ops_cpu import cache, env, lib, ref_of  # noqa: F401


def scoring(**kw):
    f = dict(softcap=0.0, reserved=0, slopes=None)
    f.update(kw)
    return pda._Scoring(*f.values())


def scored(lib, env, **kw):  # noqa: F811
    a = env["addr"]
    k = dict(ctx=env["ctx"], q=a, cache=cache(env), table=a, width=2, lens=a, batch=0, q_len=1, scale=math.nan,
             scoring=None, w_in=None, w_out=None, scratch=None, size=0, out=a)
    k.update(kw)
    return lib.pda_decode_scored(k["ctx"], k["q"], ref_of(k["cache"]), k["table"], k["width"], k["lens"], k["batch"],
                                 k["q_len"], k["scale"], ref_of(k["scoring"]), k["w_in"], k["w_out"], k["scratch"], k["size"],
                                 k["out"], 0, None)


def shared(lib, env, **kw):  # noqa: F811
    a = env["addr"]
    k = dict(ctx=env["ctx"], q=a, cache=cache(env), table=a, width=2, lens=a, batch=0, q_len=1, shared=a, starts=None,
             groups=1, scale=math.nan, scoring=None, scratch=a, size=1 << 40, out=a)
    k.update(kw)
    return lib.pda_decode_shared(k["ctx"], k["q"], ref_of(k["cache"]), k["table"], k["width"], k["lens"], k["batch"],
                                 k["q_len"], k["shared"], k["starts"], k["groups"], k["scale"], ref_of(k["scoring"]),
                                 k["scratch"], k["size"], k["out"], 0, None)


def evict(lib, env, **kw):  # noqa: F811
    a = env["addr"]
    k = dict(ctx=env["ctx"], cache=cache(env), weights=a, table=a, width=2, lens=a, batch=2, keep=8, first=0, recent=0,
             out_table=None, out_width=0, kept=a, new_lens=a + 64)
    k.update(kw)
    return lib.pda_evict(k["ctx"], ref_of(k["cache"]), k["weights"], k["table"], k["width"], k["lens"], k["batch"], k["keep"],
                         k["first"], k["recent"], k["out_table"], k["out_width"], k["kept"], k["new_lens"], None)


BAD_CALLS = [dict(ctx=None), dict(batch=-1), dict(batch=9), dict(batch=3, q_len=3), dict(q_len=0), dict(q_len=1025),
             dict(batch=2, q=None), dict(batch=2, out=None), dict(batch=2, table=None), dict(batch=2, lens=None),
             dict(batch=2, width=0), dict(batch=2, scale=math.inf), dict(cache=None)]
BAD_SCORINGS = [dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=1e-4), dict(softcap=2e6)]


@pytest.mark.parametrize("call", [scored, shared])
@pytest.mark.parametrize("bad", BAD_CALLS)
def test_refused_calls(lib, env, call, bad):  # noqa: F811
    assert call(lib, env) == pda.OK  # no sequences: nothing to do
    assert call(lib, env, **bad) == pda.ERR_INVALID_ARG
    assert lib.pda_last_error()


@pytest.mark.parametrize("call", [scored, shared])
def test_refused_scorings_and_alignments(lib, env, call):  # noqa: F811
    for bad in BAD_SCORINGS:
        assert call(lib, env, scoring=scoring(**bad)) == pda.ERR_INVALID_ARG, bad
    assert call(lib, env, scoring=scoring(slopes=env["addr"] + 2)) == pda.ERR_INVALID_ARG
    assert call(lib, env, scoring=scoring(softcap=1e-3)) == call(lib, env, scoring=scoring(softcap=1e6)) == pda.OK
    for bad in ("q", "out"):
        assert call(lib, env, batch=2, **{bad: env["addr"] + 8}) == pda.ERR_INVALID_ARG
    for bad in ("table", "lens"):
        assert call(lib, env, batch=2, **{bad: env["addr"] + 2}) == pda.ERR_INVALID_ARG
    for bad in (dict(format=3), dict(k_pool=None), dict(scales=None), dict(num_blocks=0), dict(tok_stride=8)):
        assert call(lib, env, cache=cache(env, **bad)) == pda.ERR_INVALID_ARG, bad


def test_refused_weights(lib, env):  # noqa: F811
    a = env["addr"]
    assert scored(lib, env, w_in=a) == pda.ERR_INVALID_ARG
    assert scored(lib, env, w_out=a + 2) == pda.ERR_INVALID_ARG
    for bad in (dict(), dict(scratch=a), dict(scratch=a + 8, size=1 << 40), dict(scratch=a, size=1 << 40, width=1 << 27)):
        assert scored(lib, env, batch=2, w_out=a, **bad) == pda.ERR_INVALID_ARG, bad


def test_refused_groups(lib, env):  # noqa: F811
    a = env["addr"]
    for bad in (dict(groups=0), dict(groups=1025), dict(groups=-1), dict(batch=4, groups=3), dict(batch=2, shared=None),
                dict(batch=2, shared=a + 1), dict(batch=2, starts=a + 2), dict(batch=2, scratch=None),
                dict(batch=2, scratch=a + 8), dict(batch=2, size=1000),
                dict(batch=2, width=(1 << 31) - 1, groups=1024, starts=a)):
        assert shared(lib, env, **bad) == pda.ERR_INVALID_ARG, bad


def test_refused_evictions(lib, env):  # noqa: F811
    a = env["addr"]
    assert evict(lib, env, batch=0) == pda.OK
    for bad in (dict(ctx=None), dict(cache=None), dict(batch=-1), dict(batch=9), dict(keep=0), dict(keep=-1), dict(first=-1),
                dict(recent=-1), dict(first=5, recent=4), dict(first=(1 << 31) - 1, recent=(1 << 31) - 1), dict(weights=None),
                dict(table=None), dict(lens=None), dict(kept=None), dict(new_lens=None), dict(new_lens=a), dict(weights=a + 2),
                dict(kept=a + 1), dict(out_table=a + 2, out_width=4), dict(width=0), dict(width=1 << 27),
                dict(out_table=a + 128, out_width=0), dict(out_table=a + 128, out_width=2, keep=33, width=3),
                dict(out_table=a, out_width=3), dict(cache=cache(env, format=7)), dict(cache=cache(env, scales=None))):
        assert evict(lib, env, **bad) == pda.ERR_INVALID_ARG, bad
    assert lib.pda_last_error()


def test_scratch_sizes(lib, env):  # noqa: F811
    size = ctypes.c_int64()
    for fn, last in ((lib.pda_decode_scored_scratch, 4), (lib.pda_decode_shared_scratch, 1)):
        for args in ((None, 1, 1, last), (env["ctx"], -1, 1, last), (env["ctx"], 1, 0, last), (env["ctx"], 9, 1, last),
                     (env["ctx"], 4, 3, last), (env["ctx"], 1, 1, 0)):
            assert fn(*args, ctypes.byref(size)) == pda.ERR_INVALID_ARG, args
        assert fn(env["ctx"], 1, 1, last, None) == pda.ERR_INVALID_ARG
    assert lib.pda_decode_shared_scratch(env["ctx"], 2, 1, 1025, ctypes.byref(size)) == pda.ERR_INVALID_ARG


def calls(c):
    kp, vp = pools(torch.bfloat16)
    k8, v8 = pools(torch.int8)
    w = f32(5, HKV, 16)
    return {
        "scored": lambda q=heads(HQ), out=None, dt=None, **kw: c.decode_scored(q, kp, vp, i32(B, 2), i32(B), out=out, out_dtype=dt, **kw),
        "scored 8 bits": lambda q=heads(HQ), out=None, dt=None, **kw: c.decode_scored(q, k8, v8, i32(B, 2), i32(B), scales=f32(*SCALES),
                                                                                  out=out, out_dtype=dt, **kw),
        "shared": lambda q=heads(HQ), out=None, dt=None, **kw: c.decode_shared(q, kp, vp, i32(B, 2), i32(B), i32(1), out=out,
                                                                            out_dtype=dt, **kw),
        "weights": lambda q=heads(HQ), out=None, dt=None, **kw: c.decode_scored(q, kp, vp, i32(B, 2), i32(B), weights=w, out=out,
                                                                             out_dtype=dt, **kw),
    }


@pytest.fixture
def uint8_too(monkeypatch, ctx):  # noqa: F811
    pda._TORCH.uint8 = torch.uint8
    monkeypatch.setattr(Tensor, "numel", lambda self: int(torch.Size(self.shape).numel()), raising=False)
    return ctx


@pytest.mark.parametrize("name", ["scored", "scored 8 bits", "shared", "weights"])
def test_outputs_of_another_type_or_shape_are_refused(uint8_too, name):
    c = uint8_too
    call = calls(c)[name]
    for dt, other in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        out = Tensor((B, HQ, D), dt)
        assert call(out=out) is out and call(out=out, dt=dt) is out
        launched = len(c.calls)
        for bad in (Tensor((B - 1, HQ, D), dt), Tensor((B, HQ, D), torch.int32)):
            with pytest.raises(ValueError):
                call(out=bad)
        with pytest.raises(ValueError):
            call(out=out, dt=other)
        with pytest.raises(ValueError):
            call(dt=torch.float16)
        with pytest.raises(ValueError):
            call(q=bf16(B + 1, HQ, D))
        with pytest.raises(ValueError):
            call(alibi_slopes=f32(HQ + 1))
        with pytest.raises(ValueError):
            call(alibi_slopes=Tensor((HQ,), torch.bfloat16))
        assert not [n for n, _ in c.calls[launched:] if n in ("pda_decode_scored", "pda_decode_shared")]


def test_bad_tensors_of_weights_groups_and_evictions(uint8_too):
    c = uint8_too
    kp, vp = pools(torch.bfloat16)
    t, n, w = i32(B, 2), i32(B), f32(5, HKV, 16)
    q = heads(HQ)
    for bad in (lambda: c.decode_scored(q, kp, vp, t, n, weights=f32(4, HKV, 16)),
                lambda: c.decode_scored(q, kp, vp, t, n, weights=Tensor((5, HKV, 16), torch.bfloat16)),
                lambda: c.decode_scored(q, kp, vp, t, n, weights_from=w),
                lambda: c.decode_scored(q, kp, vp, t, n, weights=w, weights_from=f32(5, HKV, 8)),
                lambda: c.decode_scored(q, kp, vp, t, n, weights=w, scratch=f32(100)),
                lambda: c.decode_shared(q, kp, vp, t, n, i32(1, 1)),
                lambda: c.decode_shared(q, kp, vp, t, n, f32(1)),
                lambda: c.decode_shared(q, kp, vp, t, n, i32(2), starts=i32(2)),
                lambda: c.evict(kp, vp, f32(5, HKV, 8), t, n, 8),
                lambda: c.evict(kp, vp, w, t, n, 0),
                lambda: c.evict(kp, vp, w, t, n, 8, first=5, recent=4),
                lambda: c.evict(kp, vp, w, t, n, 8, out_table=i32(B + 1, 2)),
                lambda: c.evict(kp, vp, w, t, n, 8, kept=i32(B, HKV, 9)),
                lambda: c.evict(kp, vp, w, t, n, 8, new_lens=i32(B + 1)),
                lambda: c.evict(kp, vp, w, t, n, 8, new_lens=f32(B)),
                lambda: c.evict(*pools(torch.int8), w, t, n, 8)):
        with pytest.raises(ValueError):
            bad()
    assert not [x for x, _ in c.calls if x in ("pda_decode_scored", "pda_decode_shared", "pda_evict")]


def test_new_tensors_are_made_on_the_calls_stream(uint8_too):
    c = uint8_too
    kp, vp = pools(torch.bfloat16)
    w = f32(5, HKV, 16)
    for call in (lambda s: c.decode_scored(heads(HQ), kp, vp, i32(B, 2), i32(B), weights=w, stream=s),
                 lambda s: c.decode_shared(heads(HQ), kp, vp, i32(B, 2), i32(B), i32(1), stream=s),
                 lambda s: c.evict(kp, vp, w, i32(B, 2), i32(B), 8, stream=s)):
        for stream, where in ((None, 5), (77, 77), (c.stream_of(77), 77), (0, 0)):
            del c.made[:]
            c.current[0] = 5
            call(stream)
            assert len(c.made) == 2 and all(t.made_on == where for t in c.made)


def test_a_closed_context_is_refused(uint8_too):
    c = uint8_too
    kp, vp = pools(torch.bfloat16)
    call = c.bind_evict(kp, vp, f32(5, HKV, 16), i32(B, 2), i32(B), 8)
    c._ctx = None
    with pytest.raises(pda.PdaError):
        call()
    with pytest.raises(pda.PdaError):
        c.decode_shared(heads(HQ), kp, vp, i32(B, 2), i32(B), i32(1))


# ------------------------------------------------------------------ the definitions

def test_definitions_agree_with_plain_ones():
    g = torch.Generator().manual_seed(0)
    lens, bs, hq, hkv, d, n = [9, 3, 0], 4, 4, 2, 64, 2
    import numpy as np
    table, pool = ref.ref.sequences(np.random.default_rng(0), lens, bs)
    kp, vp, sc = ref.random_cache(g, pool, bs, hkv, d, torch.bfloat16)
    q = torch.randn((3, n, hq, d), generator=g).bfloat16()
    out, size, sums = ref.scored64(q, kp, vp, sc, table, lens, bs)
    plain, _ = ref.ref.decode64(q, kp.float().bfloat16(), vp, None, table, lens, bs)
    assert torch.allclose(out, plain, atol=1e-12)
    assert all(abs(float(s.sum()) - hq * n) < 1e-9 for s in sums[:2]) and sums[2].numel() == 0
    # a large cap changes nothing, no slope is no bias; a cap of almost nothing gives plain means
    same, _, _ = ref.scored64(q, kp, vp, sc, table, lens, bs, softcap=1e6, slopes=torch.zeros(hq))
    assert torch.allclose(out, same, atol=1e-9)
    flat, _, _ = ref.scored64(q, kp, vp, sc, table, lens, bs, softcap=1e-9)
    v = ref.ref.rows64(vp, None, 1, table[0], 9, bs)
    assert torch.allclose(flat[0, 1].reshape(hkv, 2, d), v.mean(0)[:, None].expand(hkv, 2, d), atol=1e-6)
    # steep slopes leave each query its own token
    near, _, _ = ref.scored64(q, kp, vp, sc, table, lens, bs, slopes=torch.full((hq,), 1e3))
    assert torch.allclose(near[0, 1].reshape(hkv, 2, d), v[8][:, None].expand(hkv, 2, d), atol=1e-9)
    old = torch.rand((pool, hkv, bs), generator=g)
    after, added = ref.add_sums(old, sums, table, lens, bs, n)
    assert float(after[table[0, 2].long(), 0, 0]) == float(sums[0][8, 0])  # a query's own token starts anew
    assert (added >= 0).sum() == hkv * 12


def test_eviction_definition():
    w = torch.tensor([[[5.0, 1.0, 3.0, 3.0]], [[float("nan"), 0.0, 3.0, 9.0]]])
    table = torch.tensor([[1, 0]])
    assert ref.evict64(w, table, [8], 4, 3, 0, 0) == [[[0, 3, 4]]]
    assert ref.evict64(w, table, [8], 4, 4, 1, 1) == [[[0, 3, 4, 7]]]
    assert ref.evict64(w, table, [7], 4, 5, 2, 0) == [[[0, 1, 2, 3, 4]]]
    assert ref.evict64(w, table, [2], 4, 5, 2, 0) == [[[0, 1]]]
