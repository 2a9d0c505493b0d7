"""Outputs given to a call: of the type that it writes and large enough, or refused before anything is launched."""
import pytest
import torch

from fake_binding import B, D, HQ, SCALES, Tensor, bf16, ctx, f32, heads, i32, pools  # noqa: F401

SHAPE = (B, HQ, D)


def calls_with_out(c):
    """(name, call of (out, out_dtype))"""
    kp, vp = pools(torch.bfloat16)
    k8, v8 = pools(torch.int8)
    parts = f32(2, B, HQ), f32(2, B, HQ), f32(2, B, HQ, D)
    return {
        "decode": lambda out, dt: c.decode(heads(HQ), kp, vp, i32(B, 2), i32(B), out=out, out_dtype=dt),
        "decode 8 bits": lambda out, dt: c.decode(heads(HQ), k8, v8, i32(B, 2), i32(B), scales=f32(*SCALES), out=out,
                                                  out_dtype=dt),
        "finalize": lambda out, dt: c.finalize(B, out=out, out_dtype=dt),
        "merge_states": lambda out, dt: c.merge_states(*parts, out=out, out_dtype=dt),
    }


@pytest.mark.parametrize("name", ["decode", "decode 8 bits", "finalize", "merge_states"])
def test_an_output_of_another_type_or_too_small_is_refused(ctx, name):  # noqa: F811
    call = calls_with_out(ctx)[name]
    for dt, good, other in ((torch.float32, torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16, torch.float32)):
        out = Tensor(SHAPE, good)
        assert call(out, dt) is out
        launched = len(ctx.calls)
        for bad in (Tensor(SHAPE, other), Tensor((B - 1, HQ, D), good)):
            with pytest.raises(ValueError):
                call(bad, dt)
        assert not [n for n, _ in ctx.calls[launched:] if not n.endswith("_strides")]
