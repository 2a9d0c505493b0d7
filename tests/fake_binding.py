"""A Context without a GPU: a torch whose tensors record the stream that was current when they were made, and a library
that launches nothing and notes its calls."""
import contextlib
import types

import pytest
import torch

import paged_gqa_decode_05_gb300 as pda

HQ, HKV, D, BS, B = 4, 2, 64, 16, 3


class Tensor:
    """What the binding looks at in a tensor on device 0."""

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on, self.is_cuda = torch.Size(shape), dtype, made_on, True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def stride(self, i):
        return int(torch.Size(self.shape[i + 1:]).numel())


@pytest.fixture
def ctx(monkeypatch):
    current = [0]
    made, calls = [], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = before

    def make(*shape, dtype=None, device=None):
        made.append(Tensor(shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape, dtype, current[0]))
        return made[-1]

    def like(t):
        return make(t.shape, dtype=t.dtype)

    def stream_of(handle, device=None):
        return types.SimpleNamespace(cuda_stream=int(handle))

    def external(handle, device=None):  # torch takes a handle of 0 for none and gives a stream of its pool
        return stream_of(handle or 99)

    fake = types.SimpleNamespace(
        bfloat16=torch.bfloat16, float32=torch.float32, float8_e4m3fn=torch.float8_e4m3fn, int8=torch.int8,
        int32=torch.int32, Size=torch.Size, empty=make, zeros=make, empty_like=like, zeros_like=like,
        cuda=types.SimpleNamespace(stream=on, ExternalStream=external, default_stream=lambda device=None: stream_of(0),
                                   current_stream=lambda: stream_of(current[0])),
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: current[0]))
    monkeypatch.setattr(pda, "_TORCH", fake)

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, args))
                if name.endswith("_strides"):
                    args[1][:] = [BS * HKV * D, HKV * D, D]
                return 0
            return call

    monkeypatch.setattr(pda, "_LIB", Lib())
    c = object.__new__(pda.Context)
    c.dims = pda.Dims(16, HQ, HKV, D, BS, 4)
    c.device, c._index, c._ctx, c.G = torch.device("cuda", 0), 0, 1, HQ // HKV
    c.made, c.calls, c.stream_of, c.current = made, calls, stream_of, current
    yield c
    c._ctx = None


def bf16(*shape):
    return Tensor(shape, torch.bfloat16)


def i32(*shape):
    return Tensor(shape, torch.int32)


def f32(*shape):
    return Tensor(shape, torch.float32)


POOL = (5, BS, HKV, D)
SCALES = (5, HKV, 2, BS)


def pools(dtype):
    return Tensor(POOL, dtype), Tensor(POOL, dtype)


def heads(n):
    return bf16(B, n, D)
