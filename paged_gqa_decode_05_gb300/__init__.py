"""Paged grouped-query decode attention for GB300 (sm_103a).

A thin ctypes binding of ``libpda.so`` (C ABI in ``include/pda.h``).  Every
step of the computation runs in the library's CUDA kernels; this module only
checks tensor shapes/dtypes and passes pointers, sizes and the current torch
stream.  PyTorch supplies device memory and streams.  There is no CPU
fallback: if the library is missing, every call raises ``RuntimeError``.

Typical use::

    import paged_gqa_decode_05_gb300 as pda
    ctx = pda.Context(max_seqs=32, num_q_heads=32, num_kv_heads=8, head_dim=128,
                      block_size=16)
    out = ctx.decode(q, k_pool, v_pool, block_table, seq_lens)   # bf16 [B, Hq, D]

Tiled lifecycle (tiled_attention.rs: begin_step / step_tile / finalize)::

    ctx.begin_step(B)
    for tile_blocks, counts, last_valid in tiles:
        ctx.step_tile(q, k_pool, v_pool, tile_blocks, counts, last_valid)
    out = ctx.finalize(B)

A layer's step over a cache in 8 bits (one scale per token and kv head)::

    k_pool, v_pool, scales = ctx.new_cache(num_blocks, torch.float8_e4m3fn)   # or torch.int8
    q = ctx.append(k, v, k_pool, v_pool, block_table, seq_lens, scales=scales, q=q,
                   q_weight=wq, k_weight=wk, cos_sin=pda.rope_table(max_len, 128))
    out = ctx.decode(q, k_pool, v_pool, block_table, seq_lens, scales=scales)
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

__all__ = ["Context", "PdaError", "lib", "library_path", "check_dims", "paged_strides",
           "slot_strides", "plan_units", "gather_states", "rope_table", "DEVERR_BAD_BLOCK_ID",
           "DEVERR_BAD_LENGTH", "DEVERR_BAD_POSITION", "DEVERR_TIMEOUT"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBPATH = os.path.join(_HERE, "libpda.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_NO_DEVICE, ERR_DEVICE_DATA = range(6)
DEVERR_BAD_BLOCK_ID, DEVERR_BAD_LENGTH, DEVERR_TIMEOUT, DEVERR_BAD_POSITION = 0x1, 0x2, 0x4, 0x8
CACHE_BF16, CACHE_E4M3, CACHE_INT8 = range(3)


class PdaError(RuntimeError):
    """A libpda call returned a non-zero status."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("max_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("tile_capacity", ctypes.c_int32)]


class LaunchInfo(ctypes.Structure):
    _fields_ = [("split_ctas", ctypes.c_int32), ("ctas_per_sm", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("stage_tokens", ctypes.c_int32),
                ("partial_slots", ctypes.c_int64), ("unit_cost", ctypes.c_int32)]


class MultiInfo(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int32), ("queries_per_walk", ctypes.c_int32),
                ("rows_per_walk", ctypes.c_int32), ("walks_per_seq", ctypes.c_int32),
                ("split_ctas", ctypes.c_int32), ("stages", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("blk_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64), ("kvh_stride", ctypes.c_int64)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Prep(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weights_f32", ctypes.c_int32),
                ("eps", ctypes.c_float), ("cos_sin", ctypes.c_void_p), ("max_positions", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_LIB: Optional[ctypes.CDLL] = None
ABI_VERSION = 5  # PDA_ABI_VERSION of include/pda.h that these signatures follow


def library_path() -> str:
    return _LIBPATH


def lib() -> ctypes.CDLL:
    """The loaded libpda.so (raises RuntimeError if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(_LIBPATH):
        raise RuntimeError(f"{_LIBPATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(_LIBPATH)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sig = {
        "pda_abi_version": (I32, []),
        "pda_status_string": (ctypes.c_char_p, [I32]),
        "pda_last_error": (ctypes.c_char_p, []),
        "pda_check_dims": (I32, [ctypes.POINTER(Dims)]),
        "pda_paged_strides": (I32, [ctypes.POINTER(Dims), ctypes.POINTER(I64)]),
        "pda_slot_strides": (I32, [ctypes.POINTER(Dims), ctypes.POINTER(I64)]),
        "pda_create": (I32, [ctypes.POINTER(Dims), ctypes.POINTER(P)]),
        "pda_destroy": (None, [P]),
        "pda_decode": (I32, [P, P, P, P, I64, P, I32, P, I32, F, P, P]),
        "pda_decode_strided": (I32, [P, P, P, P, I64, I64, I64, I64, P, I32, P, I32, F, P, P]),
        "pda_decode_f32": (I32, [P, P, P, P, I64, I64, I64, I64, P, I32, P, I32, F, P, P]),
        "pda_decode_contiguous": (I32, [P, P, P, P, I32, P, I32, F, P, P]),
        "pda_decode_multi": (I32, [P, P, P, P, I64, P, I32, P, I32, I32, F, P, P]),
        "pda_begin_step": (I32, [P, I32, P]),
        "pda_step_tile": (I32, [P, P, P, P, I64, P, P, P, I32, I64, I64, I64, F, P]),
        "pda_finalize": (I32, [P, P, I32, P]),
        "pda_finalize_f32": (I32, [P, P, I32, P]),
        "pda_export_state": (I32, [P, I32, P, P, P, P]),
        "pda_merge_states": (I32, [P, I32, I32, P, P, P, P, P]),
        "pda_merge_states_f32": (I32, [P, I32, I32, P, P, P, P, P]),
        "pda_norm_rope": (I32, [P, P, P, P, I64, P, P, P, P]),
        "pda_append": (I32, [P, P, P, P, P, I32, P, I32, P, P, I64, P, P, P, P]),
        "pda_read_cache": (I32, [P, P, P, I32, P, I32, P, I64, P, P, I32, P]),
        "pda_decode_cache": (I32, [P, P, P, P, I32, P, I32, I32, F, P, I32, P]),
        "pda_debug_gather": (I32, [P, P, P, I64, I64, I64, I64, P, I32, P, I32, P, P, P]),
        "pda_read_device_errors": (I32, [P, ctypes.POINTER(ctypes.c_uint32), I32, P]),
        "pda_set_timing_events": (I32, [P, P, P, P]),
        "pda_check_wait_timeout": (I32, [P, I64, P]),
        "pda_get_launch_info": (I32, [P, ctypes.POINTER(LaunchInfo)]),
        "pda_get_multi_info": (I32, [P, I32, ctypes.POINTER(MultiInfo)]),
        "pda_set_tile_overlap": (I32, [P, I32]),
        "pda_set_multi_tc": (I32, [P, I32]),
        "pda_plan_units": (I32, [P, I32, I32, I32, I32, I32, I32, I32, P, P, ctypes.POINTER(I64)]),
    }
    for name, (res, args) in sig.items():
        try:
            fn = getattr(L, name)
        except AttributeError:  # entry points are added within an ABI version
            raise RuntimeError(f"{_LIBPATH} is older than this binding, which calls {name}: rebuild it") from None
        fn.restype = res
        fn.argtypes = args
    if L.pda_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{_LIBPATH} has ABI version {L.pda_abi_version()}, this binding "
                           f"expects {ABI_VERSION}: rebuild it")
    _LIB = L
    return L


def _check(status: int) -> None:
    if status != OK:
        L = lib()
        raise PdaError(status, f"{L.pda_status_string(status).decode()}: "
                               f"{L.pda_last_error().decode()}")


def _dims(max_seqs, num_q_heads, num_kv_heads, head_dim, block_size, tile_capacity) -> Dims:
    return Dims(int(max_seqs), int(num_q_heads), int(num_kv_heads), int(head_dim),
                int(block_size), int(tile_capacity))


def check_dims(**kw) -> int:
    """Status of pda_check_dims for the given dims (host only, no GPU)."""
    d = _dims(kw.get("max_seqs", 1), kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"],
              kw["block_size"], kw.get("tile_capacity", 1))
    return lib().pda_check_dims(ctypes.byref(d))


def _strides(fn, **kw) -> Tuple[int, int, int]:
    d = _dims(1, kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"], kw["block_size"], 1)
    out = (ctypes.c_int64 * 3)()
    _check(fn(ctypes.byref(d), out))
    return int(out[0]), int(out[1]), int(out[2])


def paged_strides(**kw) -> Tuple[int, int, int]:
    """(block, token, kv-head) element strides of [num_blocks, bs, Hkv, D]."""
    return _strides(lib().pda_paged_strides, **kw)


def slot_strides(**kw) -> Tuple[int, int, int]:
    """(block, token, kv-head) element strides of the slot layout [slot, K|V, Hkv, bs, D]."""
    return _strides(lib().pda_slot_strides, **kw)


def plan_units(lens: Sequence[int], *, block_size: int, num_kv_heads: int, split_ctas: int,
               blocks_given: bool = False, unit_cost: int = 0, stage_tokens: int = 0):
    """(first_cta, last_cta, total_blocks) of the split plan (host only); a
    context's unit_cost and stage_tokens are in its launch_info() (stage_tokens
    0: the even split for every batch, without the small-batch unit plan)."""
    import numpy as np
    lens = np.ascontiguousarray(lens, dtype=np.int32)
    n = lens.shape[0] * num_kv_heads
    first = np.zeros(max(n, 1), dtype=np.int32)
    last = np.zeros(max(n, 1), dtype=np.int32)
    total = ctypes.c_int64()
    _check(lib().pda_plan_units(lens.ctypes.data, lens.shape[0], int(blocks_given), block_size,
                                num_kv_heads, split_ctas, unit_cost, stage_tokens, first.ctypes.data,
                                last.ctypes.data, ctypes.byref(total)))
    return first[:n], last[:n], int(total.value)


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, inv_freq=None, device="cuda"):
    """The cos_sin table of norm_rope and append: [max_positions, rotary_dim] fp32, a row's
    rotary_dim / 2 cosines before its sines, of the angles position * inv_freq (by default
    base ** (-2 i / rotary_dim)).  Angles are taken in fp64: far positions lose nothing."""
    torch = _torch()
    if inv_freq is None:
        inv_freq = float(base) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    inv_freq = torch.as_tensor(inv_freq).to(device=device, dtype=torch.float64)
    if inv_freq.shape != (rotary_dim // 2,):
        raise ValueError("inv_freq must hold rotary_dim / 2 values")
    a = torch.arange(max_positions, dtype=torch.float64, device=inv_freq.device)[:, None] * inv_freq
    return torch.cat([a.cos(), a.sin()], 1).float()


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Context:
    """Owns the running (m, l, o) state and split workspace on one device
    (tiled_attention.rs: TiledAttention)."""

    def __init__(self, max_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 block_size: int, tile_capacity: int = 64, device=None):
        torch = _torch()
        self.dims = _dims(max_seqs, num_q_heads, num_kv_heads, head_dim, block_size, tile_capacity)
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index or 0)
        self._index = self.device.index
        self._ctx = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().pda_create(ctypes.byref(self.dims), ctypes.byref(self._ctx)))
        self.G = num_q_heads // num_kv_heads

    # -- properties
    @property
    def num_q_heads(self) -> int:
        return self.dims.num_q_heads

    @property
    def num_kv_heads(self) -> int:
        return self.dims.num_kv_heads

    @property
    def head_dim(self) -> int:
        return self.dims.head_dim

    @property
    def block_size(self) -> int:
        return self.dims.block_size

    def close(self) -> None:
        if self._ctx:
            lib().pda_destroy(self._ctx)
            self._ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    def launch_info(self) -> dict:
        info = LaunchInfo()
        _check(lib().pda_get_launch_info(self._ctx, ctypes.byref(info)))
        return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}

    def multi_info(self, q_len: int) -> dict:
        """The launch decode_multi makes for q_len queries per sequence (pda_get_multi_info);
        form 0: n8, 1: row form on mma.sync, 2: row form on tcgen05."""
        info = MultiInfo()
        _check(lib().pda_get_multi_info(self._ctx, int(q_len), ctypes.byref(info)))
        return {f: getattr(info, f) for f, _ in MultiInfo._fields_}

    def set_multi_tc(self, enable: bool) -> None:
        """decode_multi takes the tcgen05 row form where it applies, or the mma.sync row form
        (the default) (pda_set_multi_tc)."""
        _check(lib().pda_set_multi_tc(self._ctx, int(bool(enable))))

    # -- argument checks (marshalling only)
    def _bf16(self, t, name, shape=None):
        torch = _torch()
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        return t

    def _i32(self, t, name, ndim):
        torch = _torch()
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != ndim:
            raise ValueError(f"{name} must be a contiguous {ndim}-D int32 CUDA tensor")
        return t

    def _pool(self, k_pool, v_pool, strides, num_blocks):
        d = self.dims
        if strides is None:
            shape = (k_pool.shape[0], d.block_size, d.num_kv_heads, d.head_dim)
            self._bf16(k_pool, "k_pool", shape)
            self._bf16(v_pool, "v_pool", shape)
            strides = paged_strides(num_q_heads=d.num_q_heads, num_kv_heads=d.num_kv_heads,
                                    head_dim=d.head_dim, block_size=d.block_size)
            num_blocks = k_pool.shape[0]
        else:
            if k_pool.dtype != _torch().bfloat16 or v_pool.dtype != _torch().bfloat16:
                raise ValueError("k_pool / v_pool must be bfloat16")
            if num_blocks is None:
                raise ValueError("num_blocks is required with explicit strides")
        return tuple(int(s) for s in strides), int(num_blocks)

    def _cache(self, k_pool, v_pool, scales, strides, num_blocks) -> _Cache:
        """The pda_cache of pools of any format; 8-bit pools come with their scales."""
        torch = _torch()
        d = self.dims
        dtype = k_pool.dtype
        fmt = CACHE_E4M3 if dtype is torch.float8_e4m3fn else CACHE_INT8 if dtype is torch.int8 else \
            CACHE_BF16 if dtype is torch.bfloat16 else None
        if fmt is None or v_pool.dtype is not dtype:
            raise ValueError("k_pool / v_pool must both be bfloat16, float8_e4m3fn or int8")
        if k_pool.get_device() != self._index or v_pool.get_device() != self._index:
            self._here(k_pool, "k_pool")
            self._here(v_pool, "v_pool")
        bs, hkv, hd = d.block_size, d.num_kv_heads, d.head_dim
        if strides is None:
            shape = k_pool.shape
            num_blocks = shape[0]
            if shape != (num_blocks, bs, hkv, hd) or v_pool.shape != shape or not k_pool.is_contiguous() or \
                    not v_pool.is_contiguous():
                raise ValueError(f"k_pool / v_pool must be contiguous [num_blocks, {bs}, {hkv}, {hd}], alike")
            strides = (bs * hkv * hd, hkv * hd, hd)
        elif num_blocks is None:
            raise ValueError("num_blocks is required with explicit strides")
        if fmt == CACHE_BF16:
            if scales is not None:
                raise ValueError("a bfloat16 cache has no scales")
        else:
            shape = (num_blocks, hkv, 2, bs)
            if scales is None or scales.dtype is not torch.float32 or scales.shape != shape or not scales.is_contiguous():
                raise ValueError(f"scales of an 8-bit cache must be a contiguous float32 tensor of shape {shape}")
            self._here(scales, "scales")
        return _Cache(fmt, 0, k_pool.data_ptr(), v_pool.data_ptr(), _ptr(scales), num_blocks, *strides)

    def _here(self, t, name):
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}, the context's device")
        return t

    def _heads(self, t, name, tokens, heads) -> _Heads:
        if t.dtype != _torch().bfloat16 or tuple(t.shape) != (tokens, heads, self.dims.head_dim) or t.stride(2) != 1:
            raise ValueError(f"{name} must be bfloat16 [{tokens}, {heads}, {self.dims.head_dim}] with contiguous rows")
        self._here(t, name)
        # the strides of an axis of one entry say nothing
        return _Heads(_ptr(t), t.stride(0) if tokens > 1 else heads * self.dims.head_dim,
                      t.stride(1) if heads > 1 else self.dims.head_dim)

    def _prep(self, q_weight, k_weight, eps, cos_sin, interleaved) -> _Prep:
        torch = _torch()
        given = [w for w in (q_weight, k_weight) if w is not None]
        for w in given:
            if w.dtype not in (torch.bfloat16, torch.float32) or w.dtype != given[0].dtype or \
                    tuple(w.shape) != (self.dims.head_dim,) or not w.is_contiguous():
                raise ValueError("q_weight / k_weight must be contiguous bfloat16 or float32 (both the same) "
                                 f"[{self.dims.head_dim}]")
            self._here(w, "norm weights")
        rows = cols = 0
        if cos_sin is not None:
            if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
                raise ValueError("cos_sin must be a contiguous float32 [max_positions, rotary_dim] tensor")
            self._here(cos_sin, "cos_sin")
            rows, cols = cos_sin.shape
        return _Prep(_ptr(q_weight), _ptr(k_weight), int(bool(given) and given[0].dtype == torch.float32), float(eps),
                     _ptr(cos_sin), int(rows), int(cols), int(bool(interleaved)), 0)

    def _sequences(self, block_table, seq_lens, starts):
        """Checks a block table, its lengths and token starts; returns (table width, sequences)."""
        i32, on = _torch().int32, self._index
        for t, name, ndim in ((block_table, "block_table", 2), (seq_lens, "seq_lens", 1), (starts, "starts", 1)):
            if t is not None and (t.dtype is not i32 or t.get_device() != on or t.dim() != ndim or not t.is_contiguous()):
                self._here(self._i32(t, name, ndim), name)
        B = seq_lens.size(0)
        rows, width = block_table.shape
        if rows != B:
            raise ValueError("block_table must have one row per sequence")
        if starts is not None and starts.size(0) != B + 1:
            raise ValueError("starts must hold one entry per sequence and the end")
        return width, B

    def _make(self, fn, shape, dtype, stream):
        """A new output, fn(shape), on the call's stream: a fill comes before the call's kernels there, and memory that
        work of another stream may still use is not handed out."""
        torch = _torch()
        if stream is None:
            return fn(shape, dtype=dtype, device=self.device)
        if not hasattr(stream, "cuda_stream"):
            # (a handle of 0 is the default stream, which ExternalStream does not take)
            stream = torch.cuda.ExternalStream(int(stream), device=self.device) if int(stream) else \
                torch.cuda.default_stream(self.device)
        with torch.cuda.stream(stream):
            return fn(shape, dtype=dtype, device=self.device)

    def _out(self, out, shape, f32, stream):
        """`out` as a contiguous CUDA tensor of bfloat16, or float32 where f32, with room for shape; a new one if None."""
        torch = _torch()
        dtype = torch.float32 if f32 else torch.bfloat16
        if out is None:
            return self._make(torch.empty, shape, dtype, stream)
        shape = torch.Size(shape)
        if out.dtype != dtype or not out.is_cuda or not out.is_contiguous() or out.shape.numel() < shape.numel():
            raise ValueError(f"out must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
        return out

    def _scale(self, scale) -> float:
        return float("nan") if scale is None else float(scale)

    # -- one-shot decode
    def decode(self, q, k_pool, v_pool, block_table, seq_lens, scale: Optional[float] = None,
               out=None, strides: Optional[Sequence[int]] = None, num_blocks: Optional[int] = None,
               stream=None, out_dtype=None, scales=None):
        """softmax(scale * q K^T) V over each sequence's paged KV -> [B, Hq, D].

        ``out_dtype=torch.float32`` returns the fp32 quotient o / l (no bf16 rounding).
        Pools in 8 bits (float8_e4m3fn, int8) come with their ``scales``
        [num_blocks, Hkv, 2, block_size] (pda_decode_cache).
        """
        torch = _torch()
        if scales is not None or k_pool.dtype in (torch.float8_e4m3fn, torch.int8):
            B = int(seq_lens.shape[0])
            self._bf16(q, "q", (B, self.dims.num_q_heads, self.dims.head_dim))
            if out is None or out_dtype is not None:
                out = self._out(out, q.shape, out_dtype == torch.float32, stream)
            return self._decode_cache(q, 1, k_pool, v_pool, scales, block_table, seq_lens, scale, out, strides,
                                      num_blocks, stream)()
        d = self.dims
        B = int(seq_lens.shape[0])
        self._bf16(q, "q", (B, d.num_q_heads, d.head_dim))
        self._i32(block_table, "block_table", 2)
        self._i32(seq_lens, "seq_lens", 1)
        if block_table.shape[0] != B:
            raise ValueError("block_table must have one row per sequence")
        (bs_, ts_, hs_), nblk = self._pool(k_pool, v_pool, strides, num_blocks)
        f32 = out_dtype == torch.float32
        out = self._out(out, (B, d.num_q_heads, d.head_dim), f32, stream)
        L = lib()
        if f32:
            _check(L.pda_decode_f32(self._ctx, _ptr(q), _ptr(k_pool), _ptr(v_pool), nblk, bs_, ts_,
                                    hs_, _ptr(block_table), int(block_table.shape[1]),
                                    _ptr(seq_lens), B, self._scale(scale), _ptr(out),
                                    _stream(stream)))
        else:
            self._bf16(out, "out", (B, d.num_q_heads, d.head_dim))
            _check(L.pda_decode_strided(self._ctx, _ptr(q), _ptr(k_pool), _ptr(v_pool), nblk, bs_,
                                        ts_, hs_, _ptr(block_table), int(block_table.shape[1]),
                                        _ptr(seq_lens), B, self._scale(scale), _ptr(out),
                                        _stream(stream)))
        return out

    def bind_decode(self, q, k_pool, v_pool, block_table, seq_lens, out,
                    scale: Optional[float] = None, strides: Optional[Sequence[int]] = None,
                    num_blocks: Optional[int] = None, stream=None, scales=None):
        """Validates one decode's tensors once and returns a zero-argument callable
        that reruns it (the same buffers, their contents free to change between
        calls) with only the C call: for decode loops over persistent buffers
        that do not use CUDA graphs.  The callable keeps the tensors and this
        context alive, launches on the stream current at binding (or `stream`),
        and raises once the context is closed."""
        d = self.dims
        if scales is not None or k_pool.dtype in (_torch().float8_e4m3fn, _torch().int8):
            self._bf16(q, "q", (int(seq_lens.shape[0]), d.num_q_heads, d.head_dim))
            return self._decode_cache(q, 1, k_pool, v_pool, scales, block_table, seq_lens, scale, out, strides,
                                      num_blocks, stream)
        B = int(seq_lens.shape[0])
        self._bf16(q, "q", (B, d.num_q_heads, d.head_dim))
        self._i32(block_table, "block_table", 2)
        self._i32(seq_lens, "seq_lens", 1)
        if block_table.shape[0] != B:
            raise ValueError("block_table must have one row per sequence")
        self._bf16(out, "out", (B, d.num_q_heads, d.head_dim))
        (bs_, ts_, hs_), nblk = self._pool(k_pool, v_pool, strides, num_blocks)
        args = (_ptr(q), _ptr(k_pool), _ptr(v_pool), nblk, bs_, ts_, hs_, _ptr(block_table),
                int(block_table.shape[1]), _ptr(seq_lens), B, self._scale(scale), _ptr(out),
                _stream(stream))
        return _Bound(self, lib().pda_decode_strided, args,
                      (q, k_pool, v_pool, block_table, seq_lens, out))

    def decode_multi(self, q, k_pool, v_pool, block_table, seq_lens, scale: Optional[float] = None,
                     out=None, stream=None, scales=None, strides: Optional[Sequence[int]] = None,
                     num_blocks: Optional[int] = None, out_dtype=None):
        """Causal multi-query decode: q [B, q_len, Hq, D] are each sequence's last q_len
        tokens; query i sees tokens up to seq_lens[b] - q_len + i.  Returns [B, q_len, Hq, D].
        Pools in 8 bits come with their ``scales``, ``strides`` and ``num_blocks`` place
        pools of other layouts, and ``out_dtype=torch.float32`` returns o / l unrounded, as for
        decode (over bfloat16 pools for q_len 1 only)."""
        torch = _torch()
        d = self.dims
        B = int(seq_lens.shape[0])
        if q.dim() != 4 or q.shape[0] != B or q.shape[2:] != (d.num_q_heads, d.head_dim):
            raise ValueError("q must be [B, q_len, Hq, D]")
        self._bf16(q, "q")
        f32 = out_dtype == torch.float32
        if scales is not None or strides is not None or f32 or k_pool.dtype in (torch.float8_e4m3fn, torch.int8):
            if out is None or out_dtype is not None:
                out = self._out(out, q.shape, f32, stream)
            return self._decode_cache(q, int(q.shape[1]), k_pool, v_pool, scales, block_table, seq_lens, scale, out,
                                      strides, num_blocks, stream)()
        self._i32(block_table, "block_table", 2)
        self._i32(seq_lens, "seq_lens", 1)
        (bs_, ts_, hs_), nblk = self._pool(k_pool, v_pool, None, None)
        if out is None:
            out = self._make(torch.empty, q.shape, torch.bfloat16, stream)
        self._bf16(out, "out", tuple(q.shape))
        _check(lib().pda_decode_multi(self._ctx, _ptr(q), _ptr(k_pool), _ptr(v_pool), nblk,
                                      _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                      B, int(q.shape[1]), self._scale(scale), _ptr(out),
                                      _stream(stream)))
        return out

    def decode_contiguous(self, q, k, v, seq_lens, scale: Optional[float] = None, out=None,
                          stream=None):
        """Decode over a contiguous cache k, v [B, S, Hkv, D] (S a multiple of block_size)."""
        torch = _torch()
        d = self.dims
        B = int(seq_lens.shape[0])
        self._bf16(q, "q", (B, d.num_q_heads, d.head_dim))
        self._i32(seq_lens, "seq_lens", 1)
        if k.dim() != 4 or k.shape[0] != B or k.shape[2:] != (d.num_kv_heads, d.head_dim):
            raise ValueError("k must be [B, S, Hkv, D]")
        self._bf16(k, "k")
        self._bf16(v, "v", tuple(k.shape))
        if out is None:
            out = self._make(torch.empty, (B, d.num_q_heads, d.head_dim), torch.bfloat16, stream)
        self._bf16(out, "out", (B, d.num_q_heads, d.head_dim))
        _check(lib().pda_decode_contiguous(self._ctx, _ptr(q), _ptr(k), _ptr(v), int(k.shape[1]),
                                           _ptr(seq_lens), B, self._scale(scale), _ptr(out),
                                           _stream(stream)))
        return out

    def _decode_cache(self, q, q_len, k_pool, v_pool, scales, block_table, seq_lens, scale, out, strides,
                      num_blocks, stream):
        torch = _torch()
        width, B = self._sequences(block_table, seq_lens, None)
        cache = self._cache(k_pool, v_pool, scales, strides, num_blocks)
        self._here(q, "q")
        if out.dtype not in (torch.bfloat16, torch.float32) or out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bfloat16 or float32 tensor of shape {tuple(q.shape)}")
        self._here(out, "out")
        args = (_ptr(q), ctypes.addressof(cache), _ptr(block_table), width, _ptr(seq_lens), B, q_len,
                self._scale(scale), _ptr(out), int(out.dtype == torch.float32), self._stream_of(stream))
        return _Bound(self, lib().pda_decode_cache, args,
                      (cache, q, k_pool, v_pool, scales, block_table, seq_lens, out), out)

    def _stream_of(self, stream):
        """`stream`, or the current stream of this context's device."""
        return _torch()._C._cuda_getCurrentRawStream(self._index) if stream is None else _stream(stream)

    # -- around the decode: q / k preparation, cache writes and read-backs
    def new_cache(self, num_blocks: int, dtype=None):
        """A zeroed cache of num_blocks blocks: (k_pool, v_pool, scales), pools
        [num_blocks, block_size, Hkv, D] of `dtype` (bfloat16, float8_e4m3fn or int8) and
        scales [num_blocks, Hkv, 2, block_size] float32 (None for bfloat16)."""
        torch = _torch()
        d = self.dims
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.int8):
            raise ValueError("a cache is bfloat16, float8_e4m3fn or int8")
        shape = (int(num_blocks), d.block_size, d.num_kv_heads, d.head_dim)
        size = torch.empty((), dtype=dtype).element_size()
        pools = [torch.zeros((*shape[:3], shape[3] * size), dtype=torch.int8, device=self.device).view(dtype)
                 for _ in range(2)]
        scales = None if dtype == torch.bfloat16 else torch.zeros((shape[0], d.num_kv_heads, 2, d.block_size),
                                                                  device=self.device)
        return pools[0], pools[1], scales

    def norm_rope(self, q, k, positions=None, *, q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
                  interleaved: bool = False, q_out=None, k_out=None, stream=None):
        """RMS norm of each query and key head (where its weight [D] is given) and rotation by
        cos_sin[positions] (rope_table), in one pass: q [T, Hq, D], k [T, Hkv, D] bf16, of any
        token and head strides (slices of a fused projection); q or k may be None.  Returns
        (q_out, k_out), new tensors unless given (they may be q and k themselves)."""
        return self.bind_norm_rope(q, k, positions, q_weight=q_weight, k_weight=k_weight, eps=eps, cos_sin=cos_sin,
                                   interleaved=interleaved, q_out=q_out, k_out=k_out, stream=stream)()

    def bind_norm_rope(self, q, k, positions=None, *, q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
                       interleaved: bool = False, q_out=None, k_out=None, stream=None):
        """norm_rope with its tensors validated once: a callable as bind_decode's."""
        torch = _torch()
        d = self.dims
        if q is None and k is None:
            raise ValueError("neither q nor k given")
        T = int((k if q is None else q).shape[0])
        prep = self._prep(q_weight, k_weight, eps, cos_sin, interleaved)
        self._positions(positions, T)
        if cos_sin is not None and positions is None:
            raise ValueError("the rotation needs positions")
        pairs, outs = [], []
        for x, out, name, heads in ((q, q_out, "q", d.num_q_heads), (k, k_out, "k", d.num_kv_heads)):
            if x is not None and out is None:
                out = self._make(torch.empty, x.shape, torch.bfloat16, stream)
            pairs.append((None, None) if x is None else
                         (self._heads(x, name, T, heads), self._heads(out, name + "_out", T, heads)))
            outs.append(None if x is None else out)
        (qh, qo), (kh, ko) = pairs
        at = [None if h is None else ctypes.addressof(h) for h in (qh, kh, qo, ko)]
        args = (at[0], at[1], _ptr(positions), T, ctypes.addressof(prep), at[2], at[3], self._stream_of(stream))
        return _Bound(self, lib().pda_norm_rope, args,
                      (prep, pairs, q, k, positions, q_weight, k_weight, cos_sin), tuple(outs))

    def _positions(self, positions, tokens):
        if positions is not None:
            self._here(self._i32(positions, "positions", 1), "positions")
            if positions.shape[0] != tokens:
                raise ValueError("positions must hold one entry per token")

    def append(self, k, v, k_pool, v_pool, block_table, seq_lens, *, scales=None, starts=None, positions=None, q=None,
               q_out=None, q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None, interleaved: bool = False,
               strides: Optional[Sequence[int]] = None, num_blocks: Optional[int] = None, stream=None):
        """Writes the new tokens' k, v [T, Hkv, D] into the cache (quantised where its pools are
        8-bit), k normed and rotated on the way as in norm_rope where k_weight / cos_sin are
        given; with q [T, Hq, D] the queries too, returned as q_out (None without q).

        seq_lens counts the new tokens: sequence b's are its last starts[b+1] - starts[b]
        (starts [B+1] int32; None: T / B each).  The rotation position is positions[row], or
        the token's index in its sequence (pda_append)."""
        return self.bind_append(k, v, k_pool, v_pool, block_table, seq_lens, scales=scales, starts=starts,
                                positions=positions, q=q, q_out=q_out, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                cos_sin=cos_sin, interleaved=interleaved, strides=strides, num_blocks=num_blocks,
                                stream=stream)()

    def bind_append(self, k, v, k_pool, v_pool, block_table, seq_lens, *, scales=None, starts=None, positions=None,
                    q=None, q_out=None, q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
                    interleaved: bool = False, strides: Optional[Sequence[int]] = None,
                    num_blocks: Optional[int] = None, stream=None):
        """append with its tensors validated once: a callable as bind_decode's."""
        torch = _torch()
        d = self.dims
        T = int(k.shape[0])
        width, B = self._sequences(block_table, seq_lens, starts)
        cache = self._cache(k_pool, v_pool, scales, strides, num_blocks)
        prep = self._prep(q_weight, k_weight, eps, cos_sin, interleaved)
        self._positions(positions, T)
        kh, vh = self._heads(k, "k", T, d.num_kv_heads), self._heads(v, "v", T, d.num_kv_heads)
        qh = qo = None
        if q is not None:
            if q_out is None:
                q_out = self._make(torch.empty, q.shape, torch.bfloat16, stream)
            qh, qo = self._heads(q, "q", T, d.num_q_heads), self._heads(q_out, "q_out", T, d.num_q_heads)
        elif q_out is not None:
            raise ValueError("q_out without q")
        at = [None if h is None else ctypes.addressof(h) for h in (kh, vh, cache, prep, qh, qo)]
        args = (at[0], at[1], at[2], _ptr(block_table), width, _ptr(seq_lens), B, _ptr(starts), _ptr(positions), T,
                at[3], at[4], at[5], self._stream_of(stream))
        return _Bound(self, lib().pda_append, args,
                      (kh, vh, cache, prep, qh, qo, k, v, q, k_pool, v_pool, scales, block_table, seq_lens, starts,
                       positions, q_weight, k_weight, cos_sin), q_out)

    def read_cache(self, k_pool, v_pool, block_table, seq_lens, *, scales=None, starts=None, k_out=None, v_out=None,
                   out_dtype=None, strides: Optional[Sequence[int]] = None, num_blocks: Optional[int] = None,
                   stream=None):
        """The first seq_lens[b] tokens of every sequence, gathered and dequantised.  With starts
        [B+1] int32 token t of sequence b is row starts[b] + t of k_out, v_out [rows, Hkv, D]
        (given); without, the outputs are [B, S, Hkv, D], by default S the table's width in
        tokens (the layout of decode_contiguous).  bf16, or fp32; rows of no token are left as
        they were (zeros in new outputs)."""
        torch = _torch()
        d = self.dims
        width, B = self._sequences(block_table, seq_lens, starts)
        cache = self._cache(k_pool, v_pool, scales, strides, num_blocks)
        if k_out is None and v_out is None:
            if starts is not None:
                raise ValueError("starts needs k_out / v_out")
            shape = (B, width * d.block_size, d.num_kv_heads, d.head_dim)
            k_out, v_out = (self._make(torch.zeros, shape, out_dtype or torch.bfloat16, stream) for _ in range(2))
        like = v_out if k_out is None else k_out
        shape, dtype, ndim = like.shape, like.dtype, 4 if starts is None else 3
        good = (dtype is torch.bfloat16 or dtype is torch.float32) and (out_dtype is None or out_dtype is dtype) and \
            len(shape) == ndim and shape[-2] == d.num_kv_heads and shape[-1] == d.head_dim and \
            (starts is not None or shape[0] == B)
        for t in (k_out, v_out):
            if t is None:
                continue
            if not good or (t is not like and (t.dtype is not dtype or t.shape != shape)) or not t.is_contiguous():
                raise ValueError("k_out / v_out must be contiguous bfloat16 or float32 "
                                 f"[{'B, S' if starts is None else 'rows'}, {d.num_kv_heads}, {d.head_dim}], alike")
            if t.get_device() != self._index:
                self._here(t, "k_out / v_out")
        rows = shape[0] * shape[1] if starts is None else shape[0]
        status = lib().pda_read_cache(self._ctx, ctypes.addressof(cache), block_table.data_ptr(), width,
                                      seq_lens.data_ptr(), B, _ptr(starts), rows, _ptr(k_out), _ptr(v_out),
                                      dtype is torch.float32, self._stream_of(stream))
        if status:
            _check(status)
        return k_out, v_out

    # -- tiled lifecycle
    def set_tile_overlap(self, enable: bool) -> None:
        """Tile steps of one step on one stream overlap (default) or each waits (pda_set_tile_overlap)."""
        _check(lib().pda_set_tile_overlap(self._ctx, int(bool(enable))))

    def begin_step(self, num_seqs: int, stream=None) -> None:
        _check(lib().pda_begin_step(self._ctx, int(num_seqs), _stream(stream)))

    def step_tile(self, q, k_pool, v_pool, tile_blocks, tile_block_counts, tile_last_valid=None,
                  scale: Optional[float] = None, strides: Optional[Sequence[int]] = None,
                  num_blocks: Optional[int] = None, stream=None) -> None:
        d = self.dims
        S = int(tile_block_counts.shape[0])
        self._bf16(q, "q")
        if q.dim() != 3 or q.shape[0] < S or q.shape[1:] != (d.num_q_heads, d.head_dim):
            raise ValueError("q must be [>=num_seqs, Hq, D]")
        self._i32(tile_blocks, "tile_blocks", 2)
        self._i32(tile_block_counts, "tile_block_counts", 1)
        if tile_blocks.shape[0] < S or tile_blocks.shape[1] != d.tile_capacity:
            raise ValueError(f"tile_blocks must be [num_seqs, tile_capacity={d.tile_capacity}]")
        if tile_last_valid is not None:
            self._i32(tile_last_valid, "tile_last_valid", 1)
        (bs_, ts_, hs_), nblk = self._pool(k_pool, v_pool, strides, num_blocks)
        _check(lib().pda_step_tile(self._ctx, _ptr(q), _ptr(k_pool), _ptr(v_pool), nblk,
                                   _ptr(tile_blocks), _ptr(tile_block_counts), _ptr(tile_last_valid),
                                   S, bs_, ts_, hs_, self._scale(scale), _stream(stream)))

    def finalize(self, num_seqs: int, out=None, out_dtype=None, stream=None):
        torch = _torch()
        d = self.dims
        f32 = out_dtype == torch.float32
        out = self._out(out, (num_seqs, d.num_q_heads, d.head_dim), f32, stream)
        fn = lib().pda_finalize_f32 if f32 else lib().pda_finalize
        _check(fn(self._ctx, _ptr(out), int(num_seqs), _stream(stream)))
        return out

    # -- partial states across contexts (context-parallel decode)
    def export_state(self, num_seqs: int, stream=None):
        """The running (m, l, o) of sequences [0, num_seqs) as fp32 tensors
        [num_seqs, Hq], [num_seqs, Hq], [num_seqs, Hq, D]: m the reference (natural-log
        units of the scaled scores; the running max or up to 8 ln 2 below it),
        l = sum exp(s - m), o = sum exp(s - m) v."""
        torch = _torch()
        d = self.dims
        m, l = (self._make(torch.empty, (num_seqs, d.num_q_heads), torch.float32, stream) for _ in range(2))
        o = self._make(torch.empty, (num_seqs, d.num_q_heads, d.head_dim), torch.float32, stream)
        _check(lib().pda_export_state(self._ctx, int(num_seqs), _ptr(m), _ptr(l), _ptr(o),
                                      _stream(stream)))
        return m, l, o

    def merge_states(self, m_parts, l_parts, o_parts, out=None, out_dtype=None, stream=None):
        """o / l of P exported states per (sequence, q head): m_parts, l_parts
        [P, S, Hq], o_parts [P, S, Hq, D] (fp32, CUDA) -> [S, Hq, D]."""
        torch = _torch()
        d = self.dims
        P_, S = int(m_parts.shape[0]), int(m_parts.shape[1])
        for t, name, shape in ((m_parts, "m_parts", (P_, S, d.num_q_heads)),
                               (l_parts, "l_parts", (P_, S, d.num_q_heads)),
                               (o_parts, "o_parts", (P_, S, d.num_q_heads, d.head_dim))):
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or \
                    tuple(t.shape) != shape:
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape {shape}")
        f32 = out_dtype == torch.float32
        out = self._out(out, (S, d.num_q_heads, d.head_dim), f32, stream)
        fn = lib().pda_merge_states_f32 if f32 else lib().pda_merge_states
        _check(fn(self._ctx, P_, S, _ptr(m_parts), _ptr(l_parts), _ptr(o_parts), _ptr(out),
                  _stream(stream)))
        return out

    # -- checks and hooks
    def debug_gather(self, k_pool, v_pool, block_table, seq_lens, strides=None, num_blocks=None,
                     stream=None):
        """The K/V rows the decode kernel's loader staged, [B, Hkv, max_blocks*bs, D] each."""
        torch = _torch()
        d = self.dims
        B = int(seq_lens.shape[0])
        self._i32(block_table, "block_table", 2)
        self._i32(seq_lens, "seq_lens", 1)
        (bs_, ts_, hs_), nblk = self._pool(k_pool, v_pool, strides, num_blocks)
        rows = int(block_table.shape[1]) * d.block_size
        k_rows, v_rows = (self._make(torch.zeros, (B, d.num_kv_heads, rows, d.head_dim), torch.bfloat16, stream)
                          for _ in range(2))
        _check(lib().pda_debug_gather(self._ctx, _ptr(k_pool), _ptr(v_pool), nblk, bs_, ts_, hs_,
                                      _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                      B, _ptr(k_rows), _ptr(v_rows), _stream(stream)))
        return k_rows, v_rows

    def read_device_errors(self, clear: bool = True, stream=None) -> int:
        """PDA_DEVERR_* flags raised by kernels since the last clear (synchronises)."""
        flags = ctypes.c_uint32()
        st = lib().pda_read_device_errors(self._ctx, ctypes.byref(flags), int(clear),
                                          _stream(stream))
        if st not in (OK, ERR_DEVICE_DATA):
            _check(st)
        return int(flags.value)

    def check_wait_timeout(self, limit_ns: int = 20_000_000, stream=None) -> int:
        """Runs a bounded wait that cannot complete; returns the device flags after it."""
        _check(lib().pda_check_wait_timeout(self._ctx, int(limit_ns), _stream(stream)))
        return self.read_device_errors(stream=stream)

    def set_timing_events(self, ev_begin=None, ev_split=None, ev_end=None) -> None:
        h = [None if e is None else e.cuda_event for e in (ev_begin, ev_split, ev_end)]
        _check(lib().pda_set_timing_events(self._ctx, *h))


class _Bound:
    """A call with its arguments marshalled once (Context.bind_decode and its like)."""

    __slots__ = ("_owner", "_fn", "_args", "_keep", "_out")

    def __init__(self, owner, fn, args, keep, out=None):
        self._owner, self._fn, self._args, self._keep, self._out = owner, fn, args, keep, out

    def __call__(self):
        ctx = self._owner._ctx
        if not ctx:
            raise PdaError(ERR_INVALID_ARG, "the context of this bound call is closed")
        status = self._fn(ctx, *self._args)
        if status:
            _check(status)
        return self._out


def gather_states(m, l, o, group=None):
    """All-gathers one exported state (m, l, o) per rank over a torch.distributed
    process group into part-major stacks [world, ...] (rank order), ready for
    Context.merge_states.  Tensors stay on their device (NCCL for CUDA tensors)."""
    torch = _torch()
    import torch.distributed as dist
    world = dist.get_world_size(group)
    out = []
    for t in (m, l, o):
        t = t.contiguous()
        parts = [torch.empty_like(t) for _ in range(world)]
        dist.all_gather(parts, t, group=group)
        out.append(torch.stack(parts))
    return tuple(out)

