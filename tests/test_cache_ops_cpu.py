"""The operators around the decode on a machine without a GPU: every refusal comes before any device is touched,
so a context's dims alone (its first field) are enough for the calls to check their arguments against."""
import ctypes
import math

import pytest
import torch

import cache_ref as ref
import paged_gqa_decode_05_gb300 as pda
from paged_gqa_decode_05_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pda.lib()


@pytest.fixture(scope="module")
def env(lib):
    """A context-sized block of zeros that begins with dims (4 q heads, 2 kv heads, D 64, blocks of 16)."""
    ctx = ctypes.create_string_buffer(1 << 16)
    dims = pda.Dims(8, 4, 2, 64, 16, 4)
    ctypes.memmove(ctx, ctypes.byref(dims), ctypes.sizeof(dims))
    buf = ctypes.create_string_buffer(4096)
    addr = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    return dict(ctx=ctypes.addressof(ctx), addr=addr, keep=(ctx, buf))


def cache(env, **kw):
    f = dict(format=pda.CACHE_E4M3, reserved=0, k_pool=env["addr"], v_pool=env["addr"], scales=env["addr"], num_blocks=4,
             blk_stride=2048, tok_stride=128, kvh_stride=64)
    f.update(kw)
    return pda._Cache(*f.values())


def heads(env, **kw):
    f = dict(data=env["addr"], tok_stride=512, head_stride=64)
    f.update(kw)
    return pda._Heads(*f.values())


def prep(env, **kw):
    f = dict(q_weight=env["addr"], k_weight=env["addr"], weights_f32=0, eps=1e-6, cos_sin=env["addr"], max_positions=8,
             rotary_dim=64, interleaved=0, reserved=0)
    f.update(kw)
    return pda._Prep(*f.values())


def ref_of(x):
    return None if x is None else ctypes.addressof(x)


def append(lib, env, **kw):
    a = dict(k=heads(env), v=heads(env), cache=cache(env), table=env["addr"], width=2, lens=env["addr"], batch=0,
             starts=None, positions=None, tokens=6, prep=prep(env), q=heads(env), q_out=heads(env))
    a.update(kw)
    return lib.pda_append(env["ctx"], ref_of(a["k"]), ref_of(a["v"]), ref_of(a["cache"]), a["table"], a["width"], a["lens"],
                          a["batch"], a["starts"], a["positions"], a["tokens"], ref_of(a["prep"]), ref_of(a["q"]),
                          ref_of(a["q_out"]), None)


@pytest.mark.parametrize("bad", [
    dict(format=3), dict(format=-1), dict(k_pool=None), dict(v_pool=None), dict(scales=None), dict(num_blocks=0),
    dict(num_blocks=1 << 31), dict(blk_stride=0), dict(tok_stride=-128), dict(kvh_stride=72), dict(tok_stride=8)])
def test_bad_caches(lib, env, bad):
    for key in ("k_pool", "v_pool", "scales"):
        assert append(lib, env, cache=cache(env, **{key: env["addr"] + 4})) == pda.ERR_INVALID_ARG
    c = cache(env, **bad)
    assert append(lib, env, cache=c) == pda.ERR_INVALID_ARG
    assert lib.pda_read_cache(env["ctx"], ref_of(c), env["addr"], 2, env["addr"], 0, None, 0, env["addr"], env["addr"],
                              0, None) == pda.ERR_INVALID_ARG
    assert lib.pda_decode_cache(env["ctx"], env["addr"], ref_of(c), env["addr"], 2, env["addr"], 0, 1, math.nan,
                                env["addr"], 0, None) == pda.ERR_INVALID_ARG
    assert lib.pda_last_error()


def test_bf16_cache_needs_no_scales(lib, env):
    assert append(lib, env, cache=cache(env, format=pda.CACHE_BF16, scales=None)) == pda.OK
    assert append(lib, env, cache=cache(env, format=pda.CACHE_BF16, kvh_stride=8)) == pda.OK


@pytest.mark.parametrize("bad", [
    dict(batch=9), dict(batch=-1), dict(tokens=-1), dict(tokens=1 << 31), dict(batch=4), dict(batch=2, table=None),
    dict(batch=2, lens=None), dict(batch=2, width=0), dict(q=None), dict(q_out=None), dict(cache=None),
    dict(batch=2, k=None), dict(batch=2, v=None)])
def test_append_refusals(lib, env, bad):
    assert append(lib, env, **bad) == pda.ERR_INVALID_ARG
    assert append(lib, env) == pda.OK  # no sequences: nothing to do


@pytest.mark.parametrize("bad", [dict(data=None), dict(tok_stride=0), dict(head_stride=6), dict(tok_stride=-512)])
@pytest.mark.parametrize("which", ["k", "v", "q", "q_out"])
def test_bad_heads(lib, env, bad, which):
    assert append(lib, env, batch=2, **{which: heads(env, **bad)}) == pda.ERR_INVALID_ARG
    assert append(lib, env, batch=2, **{which: heads(env, data=env["addr"] + 4)}) == pda.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=4), dict(rotary_dim=66), dict(rotary_dim=72), dict(rotary_dim=0), dict(max_positions=0),
    dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)])
def test_bad_prep(lib, env, bad):
    assert append(lib, env, prep=prep(env, **bad)) == pda.ERR_INVALID_ARG
    assert lib.pda_norm_rope(env["ctx"], ref_of(heads(env)), None, env["addr"], 0, ref_of(prep(env, **bad)),
                             ref_of(heads(env)), None, None) == pda.ERR_INVALID_ARG


def test_norm_rope_refusals(lib, env):
    h, p = heads(env), prep(env)

    def call(q=h, k=h, positions=env["addr"], tokens=4, prep=p, q_out=h, k_out=h, ctx=env["ctx"]):
        return lib.pda_norm_rope(ctx, ref_of(q), ref_of(k), positions, tokens, ref_of(prep), ref_of(q_out), ref_of(k_out),
                                 None)

    assert call(tokens=0) == pda.OK
    for bad in (dict(q=None), dict(k_out=None), dict(q=None, k=None, q_out=None, k_out=None), dict(prep=None),
                dict(positions=None), dict(positions=env["addr"] + 2), dict(tokens=-1), dict(ctx=None)):
        assert call(**bad) == pda.ERR_INVALID_ARG, bad


def test_read_and_decode_refusals(lib, env):
    c = cache(env)
    a = env["addr"]

    def read(batch=2, rows=4, k=a, v=a, width=2, starts=None):
        return lib.pda_read_cache(env["ctx"], ref_of(c), a, width, a, batch, starts, rows, k, v, 0, None)

    assert read(batch=0) == read(rows=0) == pda.OK
    for bad in (dict(k=None, v=None), dict(k=a + 8), dict(v=a + 8), dict(rows=5), dict(width=0), dict(batch=9),
                dict(starts=a + 2)):
        assert read(**bad) == pda.ERR_INVALID_ARG, bad

    def decode(q=a, batch=2, q_len=1, scale=math.nan, out=a, table=a, width=2, ctx=env["ctx"], f32=0, cache=c):
        return lib.pda_decode_cache(ctx, q, ref_of(cache), table, width, a, batch, q_len, scale, out, f32, None)

    assert decode(batch=0) == pda.OK
    for bad in (dict(q=None), dict(q=a + 8), dict(out=None), dict(out=a + 8), dict(q_len=0), dict(q_len=5), dict(batch=9),
                dict(table=None), dict(width=0), dict(scale=math.inf), dict(ctx=None), dict(batch=-1)):
        assert decode(**bad) == pda.ERR_INVALID_ARG, bad
    assert decode(q_len=2, f32=1, cache=cache(env, format=pda.CACHE_BF16)) == pda.ERR_UNSUPPORTED


def test_rope_table():
    t = pda.rope_table(70000, 64, base=5e5, device="cpu")
    i, p = 5, 69999
    angle = p * 5e5 ** (-2 * i / 64)
    assert t.dtype == torch.float32 and t.shape == (70000, 64)
    assert abs(float(t[p, i]) - math.cos(angle)) < 1e-6 and abs(float(t[p, 32 + i]) - math.sin(angle)) < 1e-6
    f = pda.rope_table(4, 8, inv_freq=[1.0, 0.5, 0.25, 0.1], device="cpu")
    assert abs(float(f[3, 1]) - math.cos(1.5)) < 1e-6
    with pytest.raises(ValueError):
        pda.rope_table(4, 8, inv_freq=[1.0], device="cpu")


def test_reference_twins_agree():
    """The test's fp64 attention reduces to a plain mean for equal keys, and its codes stand for their rows."""
    g = torch.Generator().manual_seed(0)
    for dtype in ref.FORMATS:
        x = torch.randn((5, 64), generator=g)
        c, s = ref.codes32(x, dtype)
        y = x.double() / s.double()[:, None]
        assert ((c.double() - y).abs() <= ref.half_step(y, dtype) + 1e-4).all()
    kp, vp, sc = ref.random_cache(g, 3, 4, 1, 64, torch.int8)
    kp[:] = 0
    table = torch.tensor([[2, 0, 1]])
    out, _ = ref.decode64(torch.randn((1, 2, 1, 64), generator=g), kp, vp, sc, table, [6], 4)
    rows = ref.rows64(vp, sc, 1, table[0], 6, 4)[:, 0]
    assert torch.allclose(out[0, 1, 0], rows.mean(0)) and torch.allclose(out[0, 0, 0], rows[:5].mean(0))
