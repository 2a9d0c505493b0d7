"""Outputs that a call makes itself are made on the call's stream, not on the current one."""
import pytest
import torch

from fake_binding import B, D, HKV, HQ, SCALES, bf16, ctx, f32, heads, i32, pools  # noqa: F401

CALL = 77

CALLS = {
    "read_cache": lambda c, s: c.read_cache(*pools(torch.int8), i32(B, 2), i32(B), scales=f32(*SCALES), stream=s),
    "read_cache bf16": lambda c, s: c.read_cache(*pools(torch.bfloat16), i32(B, 2), i32(B), stream=s),
    "norm_rope": lambda c, s: c.norm_rope(heads(HQ), heads(HKV), stream=s),
    "append": lambda c, s: c.append(heads(HKV), heads(HKV), *pools(torch.bfloat16), i32(B, 2), i32(B), q=heads(HQ), stream=s),
    "decode 8 bits": lambda c, s: c.decode(heads(HQ), *pools(torch.int8), i32(B, 2), i32(B), scales=f32(*SCALES), stream=s),
    "decode": lambda c, s: c.decode(heads(HQ), *pools(torch.bfloat16), i32(B, 2), i32(B), stream=s),
    "decode_multi 8 bits": lambda c, s: c.decode_multi(bf16(B, 2, HQ, D), *pools(torch.int8), i32(B, 2), i32(B),
                                                       scales=f32(*SCALES), stream=s),
    "decode_multi": lambda c, s: c.decode_multi(bf16(B, 2, HQ, D), *pools(torch.bfloat16), i32(B, 2), i32(B), stream=s),
    "decode_contiguous": lambda c, s: c.decode_contiguous(heads(HQ), bf16(B, 32, HKV, D), bf16(B, 32, HKV, D), i32(B),
                                                          stream=s),
    "finalize": lambda c, s: c.finalize(B, stream=s),
    "export_state": lambda c, s: c.export_state(B, stream=s),
    "merge_states": lambda c, s: c.merge_states(f32(2, B, HQ), f32(2, B, HQ), f32(2, B, HQ, D), stream=s),
    "debug_gather": lambda c, s: c.debug_gather(*pools(torch.bfloat16), i32(B, 2), i32(B), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_new_outputs_are_made_on_the_calls_stream(ctx, name):
    for stream, where in ((None, 5), (CALL, CALL), (ctx.stream_of(CALL), CALL), (0, 0), (ctx.stream_of(0), 0)):
        del ctx.made[:]
        ctx.current[0] = 5
        CALLS[name](ctx, stream)
        assert ctx.made and all(t.made_on == where for t in ctx.made), (name, [t.made_on for t in ctx.made])
