"""ctypes binding of the C ABI in include/paged_decode_attn.h.

Argument marshalling only: torch tensors are checked for dtype, shape,
device and contiguity and passed as raw device pointers together with the
current CUDA stream. Every step of the computation runs in the CUDA library;
there is no fallback. If the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

PDA_OK, PDA_EINVAL, PDA_EUNSUPPORTED, PDA_ENOMEM, PDA_ECUDA, PDA_EALIAS, PDA_EDEVICE = (
    0, -1, -2, -3, -4, -5, -6)
PDA_BF16, PDA_FP16, PDA_F32 = 0, 1, 2
ABI_VERSION = 2

_STATUS_NAMES = {0: "PDA_OK", -1: "PDA_EINVAL", -2: "PDA_EUNSUPPORTED", -3: "PDA_ENOMEM",
                 -4: "PDA_ECUDA", -5: "PDA_EALIAS", -6: "PDA_EDEVICE"}
_DT = {torch.bfloat16: PDA_BF16, torch.float16: PDA_FP16, torch.float32: PDA_F32}
_DT16 = {torch.bfloat16: PDA_BF16, torch.float16: PDA_FP16}

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpaged_decode_attn.so")

# Every function the header declares (tests check the library exports them).
EXPORTS = [
    "paged_decode_attn_abi_version",
    "paged_decode_attn_last_error",
    "paged_decode_attn_create",
    "paged_decode_attn_destroy",
    "paged_decode_attn_run",
    "paged_decode_attn_run_ex",
    "paged_decode_attn_run_scaled",
    "paged_decode_attn_plan",
    "paged_decode_attn_launch_shape",
    "paged_decode_attn_merge",
    "paged_decode_attn_validate",
    "paged_decode_attn_check_device_error",
    "paged_decode_attn_run_noalloc",
    "paged_decode_attn_rope_kv_write",
    "paged_decode_attn_copy_blocks",
    "paged_decode_attn_gather_kv",
    "paged_decode_attn_scatter_kv",
    "paged_decode_attn_remap_table",
    "paged_decode_attn_append_kv_fp8",
    "paged_decode_attn_rope_append_kv_fp8",
    "paged_decode_attn_gather_kv_fp8",
    "paged_decode_attn_run_block_scaled",
]


class PDAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("block_size", ctypes.c_int),
                ("dtype", ctypes.c_int), ("max_batch", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("max_splits", ctypes.c_int),
                ("device", ctypes.c_int), ("kv_fp8", ctypes.c_int)]


_lib = None
_lock = threading.Lock()


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load the CUDA library (built by ``paged_gqa_decode_attention_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library {p} is missing: run paged_gqa_decode_attention_gb300.build.build()")
        lib = ctypes.CDLL(p)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.paged_decode_attn_abi_version.argtypes = []
        lib.paged_decode_attn_abi_version.restype = I
        lib.paged_decode_attn_last_error.argtypes = []
        lib.paged_decode_attn_last_error.restype = ctypes.c_char_p
        lib.paged_decode_attn_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(P)]
        lib.paged_decode_attn_create.restype = I
        lib.paged_decode_attn_destroy.argtypes = [P]
        lib.paged_decode_attn_destroy.restype = None
        lib.paged_decode_attn_run.argtypes = [P, P, P, P, P, P, I, I, I64, F, P, P]
        lib.paged_decode_attn_run.restype = I
        lib.paged_decode_attn_run_ex.argtypes = [P, P, P, P, P, P, I, I, I64, F, P, P, I, I, I]
        lib.paged_decode_attn_run_ex.restype = I
        lib.paged_decode_attn_run_scaled.argtypes = [P, P, P, P, P, P, I, I, I64, F, P, P, I, P,
                                                     P, I, I, I]
        lib.paged_decode_attn_run_scaled.restype = I
        lib.paged_decode_attn_plan.argtypes = [ctypes.POINTER(Config), I, I, I, I,
                                               ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.paged_decode_attn_plan.restype = I
        lib.paged_decode_attn_launch_shape.argtypes = [P, I, I, I, I] + [ctypes.POINTER(I)] * 4
        lib.paged_decode_attn_launch_shape.restype = I
        lib.paged_decode_attn_merge.argtypes = [P, P, I, I, I, P, I, I, P]
        lib.paged_decode_attn_merge.restype = I
        lib.paged_decode_attn_validate.argtypes = [P, P, P, I, I, I64, P]
        lib.paged_decode_attn_validate.restype = I
        lib.paged_decode_attn_check_device_error.argtypes = [P, ctypes.POINTER(I),
                                                             ctypes.POINTER(I), P]
        lib.paged_decode_attn_check_device_error.restype = I
        lib.paged_decode_attn_run_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I64, F,
                                                      P, I, I, P]
        lib.paged_decode_attn_run_noalloc.restype = I
        lib.paged_decode_attn_rope_kv_write.argtypes = [P, I64, P, I64, P, I64, P, P, P, I, I, I,
                                                        I, I, I, I, I, P, I64, P, P, I64, P, I,
                                                        P]
        lib.paged_decode_attn_rope_kv_write.restype = I
        lib.paged_decode_attn_copy_blocks.argtypes = [P, P, I64, I64, P, I, P, I, P]
        lib.paged_decode_attn_copy_blocks.restype = I
        lib.paged_decode_attn_gather_kv.argtypes = [P, P, I64, I, I64, P, I, P, P, I, I, P, P, P,
                                                    I, P]
        lib.paged_decode_attn_gather_kv.restype = I
        lib.paged_decode_attn_scatter_kv.argtypes = [P, P, I64, I64, P, P, P, I64, P, I, P]
        lib.paged_decode_attn_scatter_kv.restype = I
        lib.paged_decode_attn_remap_table.argtypes = [P, I, I, P, I, P, I64, P, I, P]
        lib.paged_decode_attn_remap_table.restype = I
        lib.paged_decode_attn_run_block_scaled.argtypes = [P, P, P, P, P, P, P, P, I, I, I64, F, P,
                                                           P, I, I, I]
        lib.paged_decode_attn_run_block_scaled.restype = I
        cache_args = [P, P, P, P, I64, I, P, I, P, P, I, P, I, P]
        lib.paged_decode_attn_append_kv_fp8.argtypes = [P, I64, P, I64, I64, I, I, I] + cache_args
        lib.paged_decode_attn_append_kv_fp8.restype = I
        lib.paged_decode_attn_rope_append_kv_fp8.argtypes = (
            [P, I64, P, I64, P, I64, P, P, I, I, I, I64, I, I, I, I, P, I64] + cache_args)
        lib.paged_decode_attn_rope_append_kv_fp8.restype = I
        lib.paged_decode_attn_gather_kv_fp8.argtypes = [P, P, P, P, I64, I, I, I, P, I, P, P, I, I,
                                                        P, P, I64, I, P, I, P]
        lib.paged_decode_attn_gather_kv_fp8.restype = I
        if lib.paged_decode_attn_abi_version() != ABI_VERSION:
            raise RuntimeError("ABI version mismatch between binding and library")
        if path is None:
            _lib = lib
        return lib


def _check(lib, status: int):
    if status != PDA_OK:
        raise PDAError(status, lib.paged_decode_attn_last_error().decode())


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dev_ptr(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def make_config(num_q_heads: int, num_kv_heads: int, head_dim: int = 128, block_size: int = 16,
                dtype=torch.bfloat16, max_batch: int = 256, max_blocks_per_seq: int = 4096,
                max_splits: int = 64, device: int = 0, kv_fp8: bool = False) -> Config:
    return Config(num_q_heads, num_kv_heads, head_dim, block_size, _DT[dtype], max_batch,
                  max_blocks_per_seq, max_splits, device, int(bool(kv_fp8)))


def plan(config: Config, num_sms: int, batch: int, max_blocks: int,
         max_context_len_hint: int = 0) -> tuple[int, int]:
    """(num_splits, chunk_pages) the split heuristic picks (host only)."""
    lib = load_library()
    s, c = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib, lib.paged_decode_attn_plan(ctypes.byref(config), num_sms, batch, max_blocks,
                                           max_context_len_hint, ctypes.byref(s),
                                           ctypes.byref(c)))
    return s.value, c.value


class PagedDecodeAttention:
    """One library handle: fixed geometry, owns the split-K workspace."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int = 128,
                 block_size: int = 16, dtype=torch.bfloat16, max_batch: int = 256,
                 max_blocks_per_seq: int = 4096, max_splits: int = 64, device=None,
                 kv_fp8: bool = False):
        self.lib = load_library()
        if device is None:
            device = torch.cuda.current_device()
        if isinstance(device, torch.device):
            device = device.index if device.index is not None else torch.cuda.current_device()
        self.device = int(device)
        self.dtype = dtype
        self.kv_fp8 = bool(kv_fp8)
        self._geometry = (num_q_heads, num_kv_heads, block_size, head_dim)
        self.config = make_config(num_q_heads, num_kv_heads, head_dim, block_size, dtype,
                                  max_batch, max_blocks_per_seq, max_splits, self.device,
                                  self.kv_fp8)
        h = ctypes.c_void_p(None)
        _check(self.lib, self.lib.paged_decode_attn_create(ctypes.byref(self.config),
                                                           ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.paged_decode_attn_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def run(self, q, k_cache, v_cache, block_table, context_lens, scale: float | None = None,
            out=None, num_splits: int = 0, max_context_len_hint: int = 0, out_dtype=None,
            stream=None, k_scale=None, v_scale=None):
        """out[B, Hq, D] = paged decode attention; asynchronous on ``stream``
        (default: torch's current stream). With FP8 caches (kv_fp8), k_cache
        and v_cache are torch.float8_e4m3fn (or uint8) tensors; k_scale and
        v_scale are fp32 device tensors of Hkv (per kv head) or 1 values, or,
        for a block-scaled cache (append_kv_fp8), both [num_blocks, Hkv]."""
        if self.kv_fp8 and (_is_block_scale(k_scale, self._geometry[1]) or
                            _is_block_scale(v_scale, self._geometry[1]) or
                            self._one_block_scales(q, k_cache, v_cache, block_table,
                                                   context_lens, out, k_scale, v_scale)):
            return self._run_block_scaled(q, k_cache, v_cache, block_table, context_lens, scale,
                                          out, num_splits, max_context_len_hint, out_dtype,
                                          stream, k_scale, v_scale)
        c = self.config
        B = q.shape[0]
        if scale is None:
            scale = 1.0 / math.sqrt(c.head_dim)
        if out_dtype is None:
            out_dtype = self.dtype
        if out is None:
            out = torch.empty((B, c.num_q_heads, c.head_dim), dtype=out_dtype, device=q.device)
        if self.kv_fp8:
            for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
                if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                    raise ValueError(f"{name} must be float8_e4m3fn or uint8 for an FP8 cache")
            kp, vp = _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache")
        else:
            kp = _dev_ptr(k_cache, "k_cache", self.dtype)
            vp = _dev_ptr(v_cache, "v_cache", self.dtype)
        per_head = 0
        for t in (k_scale, v_scale):
            if t is not None:
                if t.numel() not in (1, c.num_kv_heads):
                    raise ValueError("k_scale / v_scale must hold 1 or Hkv values")
                per_head = int(t.numel() == c.num_kv_heads and c.num_kv_heads > 1)
        if (k_scale is not None and v_scale is not None and
                k_scale.numel() != v_scale.numel()):
            raise ValueError("k_scale and v_scale must have the same size")
        args = (self.handle,
                _dev_ptr(q, "q", self.dtype), kp, vp,
                _dev_ptr(block_table, "block_table", torch.int32),
                _dev_ptr(context_lens, "context_lens", torch.int32),
                B, block_table.shape[1], k_cache.shape[0], float(scale),
                _dev_ptr(k_scale, "k_scale", torch.float32) if k_scale is not None else None,
                _dev_ptr(v_scale, "v_scale", torch.float32) if v_scale is not None else None,
                per_head, _dev_ptr(out, "out", out_dtype), _stream_ptr(stream),
                int(num_splits), int(max_context_len_hint), _DT[out_dtype])
        _check(self.lib, self.lib.paged_decode_attn_run_scaled(*args))
        return out

    def _one_block_scales(self, q, k_cache, v_cache, block_table, context_lens, out, k_scale,
                          v_scale) -> bool:
        """[1, Hkv] scales of a cache of one block: the heads' scales as well, but fp16 queries
        keep all their bits in the block-scaled call. Tensors in other shapes than it takes
        (a flat q, a table of more rows than the batch) go on as per-head calls."""
        Hq, Hkv, bs, D = self._geometry
        if k_scale is None or v_scale is None or k_scale.shape != (1, Hkv) or v_scale.shape != (1, Hkv):
            return False
        one, B = (1, bs, Hkv, D), len(q)
        return (k_cache.shape == one and v_cache.shape == one and q.shape == (B, Hq, D) and
                block_table.dim() == 2 and len(block_table) == B and context_lens.shape == (B,) and
                (out is None or out.shape == q.shape))

    def _run_block_scaled(self, q, k_cache, v_cache, block_table, context_lens, scale, out,
                          num_splits, max_context_len_hint, out_dtype, stream, k_scale, v_scale):
        dt, dev = self.dtype, self.device
        Hq, Hkv, bs, D = self._geometry
        if k_scale is None or v_scale is None:
            raise ValueError("block scales: k_scale and v_scale must both be [num_blocks, Hkv]")
        nb, c_bs, c_hkv, c_d = _fp8_shape(k_cache, v_cache, k_scale, v_scale)
        if c_bs != bs or c_hkv != Hkv or c_d != D:
            raise ValueError("caches must be [num_blocks, block_size, Hkv, D] with the handle's sizes")
        B = len(q)
        if q.dim() != 3 or q.numel() != B * Hq * D or q.shape[1] != Hq:
            raise ValueError("q must be [batch, Hq, D] with the handle's sizes")
        if block_table.dim() != 2 or len(block_table) != B or context_lens.shape != (B,):
            raise ValueError("block_table must be [batch, max_blocks] and context_lens [batch]")
        if out_dtype is None:
            out_dtype = dt
        if out is None:
            out = torch.empty_like(q, dtype=out_dtype)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        p = _pointers(dev, (("q", q, dt), ("k_cache", k_cache, None), ("v_cache", v_cache, None),
                            ("k_scale", k_scale, torch.float32),
                            ("v_scale", v_scale, torch.float32),
                            ("block_table", block_table, torch.int32),
                            ("context_lens", context_lens, torch.int32), ("out", out, out_dtype)))
        status = self.lib.paged_decode_attn_run_block_scaled(
            self.handle, *p[:7], B, block_table.shape[1], nb,
            D ** -0.5 if scale is None else scale, p[7],
            _raw_stream(dev) if stream is None else _stream_ptr(stream), num_splits,
            max_context_len_hint, _DT[out_dtype])
        if status:
            _check(self.lib, status)
        return out

    def run_raw(self, q_ptr: int, k_ptr: int, v_ptr: int, table_ptr: int, lens_ptr: int,
                batch: int, max_blocks: int, num_blocks: int, scale: float, out_ptr: int,
                stream: int = 0) -> int:
        """paged_decode_attn_run on raw device pointers; returns the status."""
        return self.lib.paged_decode_attn_run(self.handle, q_ptr, k_ptr, v_ptr, table_ptr,
                                              lens_ptr, batch, max_blocks, num_blocks,
                                              float(scale), out_ptr, stream)

    def launch_shape(self, batch: int, max_blocks: int, num_splits: int = 0,
                     max_context_len_hint: int = 0) -> dict:
        """How a run with these sizes is launched: splits, chunk_pages, ctas,
        cluster (CTAs per thread-block cluster; 1 = no clusters)."""
        out = [ctypes.c_int(0) for _ in range(4)]
        _check(self.lib, self.lib.paged_decode_attn_launch_shape(
            self.handle, batch, max_blocks, max_context_len_hint, num_splits,
            *[ctypes.byref(o) for o in out]))
        return dict(zip(("splits", "chunk_pages", "ctas", "cluster"), (o.value for o in out)))

    def validate(self, block_table, context_lens, num_blocks: int, stream=None):
        B = context_lens.shape[0]
        _check(self.lib, self.lib.paged_decode_attn_validate(
            self.handle, _dev_ptr(block_table, "block_table", torch.int32),
            _dev_ptr(context_lens, "context_lens", torch.int32), B, block_table.shape[1],
            int(num_blocks), _stream_ptr(stream)))

    def check_device_error(self, stream=None) -> tuple[int, int]:
        code, detail = ctypes.c_int(0), ctypes.c_int(0)
        _check(self.lib, self.lib.paged_decode_attn_check_device_error(
            self.handle, ctypes.byref(code), ctypes.byref(detail), _stream_ptr(stream)))
        return code.value, detail.value


def merge(partial_o: torch.Tensor, partial_lse: torch.Tensor, out_dtype=torch.float32,
          out=None, stream=None) -> torch.Tensor:
    """LSE merge: partial_o [rows, S, D] fp32, partial_lse [rows, S] fp32
    (natural log, -inf = empty split) -> out [rows, D]."""
    lib = load_library()
    rows, S, D = partial_o.shape
    if out is None:
        out = torch.empty((rows, D), dtype=out_dtype, device=partial_o.device)
    dev = partial_o.device.index if partial_o.device.index is not None else 0
    _check(lib, lib.paged_decode_attn_merge(
        _dev_ptr(partial_o, "partial_o", torch.float32),
        _dev_ptr(partial_lse, "partial_lse", torch.float32), rows, S, D,
        _dev_ptr(out, "out", out_dtype), _DT[out_dtype], dev, _stream_ptr(stream)))
    return out


def _token_rows(t: torch.Tensor, name: str, dtype) -> tuple[int, int]:
    """Pointer and token stride (elements) of a [T, H, D] tensor whose heads
    are contiguous within a token (a packed tensor or a view into a fused
    projection output)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    T, H, D = t.shape
    if t.stride(2) != 1 or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: heads must be contiguous within a token")
    if T > 1 and t.stride(0) < H * D:
        raise ValueError(f"{name}: tokens must not overlap (a broadcast view)")
    return t.data_ptr(), (t.stride(0) if T > 1 else H * D)


def rope_kv_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                  slot_mapping: torch.Tensor, cos_sin_cache: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, neox: bool = True,
                  q_out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """RoPE on q and k plus the paged-cache write of k and v, one launch.

    q [T, Hq, D], k/v [T, Hkv, D] (bf16/fp16; token-strided views allowed),
    positions [T] int32, slot_mapping [T] int64 (< 0: no cache write),
    cos_sin_cache [max_position, rot_dim] fp32 (cosines then sines),
    k_cache/v_cache [num_blocks, block_size, Hkv, D]. Returns q_out (a new
    tensor, or ``q_out``; pass ``q_out=q`` to rotate in place). ``err`` is an
    optional int32 [2] device tensor receiving the first bad token."""
    lib = load_library()
    dt = q.dtype
    qp, qs = _token_rows(q, "q", dt)
    kp, ks = _token_rows(k, "k", dt)
    vp, vs = _token_rows(v, "v", dt)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D):
        raise ValueError("k and v must be [T, Hkv, D] with q's T and D")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    qop, qos = _token_rows(q_out, "q_out", dt)
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    if k_cache.shape != v_cache.shape or k_cache.dim() != 4 or k_cache.shape[2:] != (Hkv, D):
        raise ValueError("caches must be [num_blocks, block_size, Hkv, D]")
    if cos_sin_cache.dim() != 2:
        raise ValueError("cos_sin_cache must be [max_position, rot_dim]")
    max_pos, rot_dim = cos_sin_cache.shape
    if positions.shape != (T,) or slot_mapping.shape != (T,):
        raise ValueError("positions and slot_mapping must be [T]")
    dev = q.device.index if q.device.index is not None else 0
    _check(lib, lib.paged_decode_attn_rope_kv_write(
        qp, qs, kp, ks, vp, vs, _dev_ptr(positions, "positions", torch.int32),
        _dev_ptr(slot_mapping, "slot_mapping", torch.int64),
        _dev_ptr(cos_sin_cache, "cos_sin_cache", torch.float32), max_pos, rot_dim,
        int(bool(neox)), T, Hq, Hkv, D, _DT[dt], qop, qos, _dev_ptr(k_cache, "k_cache", dt),
        _dev_ptr(v_cache, "v_cache", dt), k_cache.shape[0] * k_cache.shape[1],
        _dev_ptr(err, "err", torch.int32) if err is not None else None, dev,
        _stream_ptr(stream)))
    return q_out


# ------------------------------ KV-cache movement ------------------------------

def _cache_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor):
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [num_blocks, block_size, Hkv, D] alike")
    nb, bs = k_cache.shape[0], k_cache.shape[1]
    row_bytes = k_cache.shape[2] * k_cache.shape[3] * k_cache.element_size()
    return nb, bs, row_bytes


def _opt_err(err):
    return _dev_ptr(err, "err", torch.int32) if err is not None else None


def _device_of(t: torch.Tensor) -> int:
    return t.device.index if t.device.index is not None else torch.cuda.current_device()


def copy_blocks(k_cache, v_cache, pairs: torch.Tensor, err=None, stream=None):
    """Block pairs[i, 1] := block pairs[i, 0] in both caches (in place);
    pairs is an int64 [n, 2] device tensor."""
    lib = load_library()
    nb, bs, row_bytes = _cache_geometry(k_cache, v_cache)
    n = pairs.shape[0] if pairs.numel() else 0
    _check(lib, lib.paged_decode_attn_copy_blocks(
        _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), nb, bs * row_bytes,
        _dev_ptr(pairs, "pairs", torch.int64) if n else None, n, _opt_err(err),
        _device_of(k_cache), _stream_ptr(stream)))


def gather_kv(k_cache, v_cache, block_table, lens, cu_rows=None, max_len: int | None = None,
              k_out=None, v_out=None, err=None, stream=None):
    """Each sequence's tokens, in order, into contiguous [rows, Hkv, D] buffers
    (sequence b from row cu_rows[b]; default: exclusive prefix sums of lens,
    computed on the host from lens). Returns (k_out, v_out)."""
    lib = load_library()
    nb, bs, row_bytes = _cache_geometry(k_cache, v_cache)
    B = lens.shape[0]
    if cu_rows is None or max_len is None or k_out is None:
        lens_h = lens.cpu().to(torch.int64)
        if cu_rows is None:
            cu_rows = (torch.cumsum(lens_h, 0) - lens_h).to(k_cache.device)
        if max_len is None:
            max_len = int(lens_h.max()) if B else 0
        total = int(lens_h.sum())
    else:
        total = k_out.shape[0]
    shape = (total,) + tuple(k_cache.shape[2:])
    if k_out is None:
        k_out = torch.empty(shape, dtype=k_cache.dtype, device=k_cache.device)
        v_out = torch.empty(shape, dtype=k_cache.dtype, device=k_cache.device)
    _check(lib, lib.paged_decode_attn_gather_kv(
        _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), nb, bs, row_bytes,
        _dev_ptr(block_table, "block_table", torch.int32), block_table.shape[1],
        _dev_ptr(lens, "lens", torch.int32), _dev_ptr(cu_rows, "cu_rows", torch.int64), B,
        int(max_len), _dev_ptr(k_out, "k_out"), _dev_ptr(v_out, "v_out"), _opt_err(err),
        _device_of(k_cache), _stream_ptr(stream)))
    return k_out, v_out


def scatter_kv(k_rows, v_rows, slot_mapping, k_cache, v_cache, err=None, stream=None):
    """Row r of k_rows / v_rows ([n, Hkv, D]) into cache slot slot_mapping[r]
    (int64; < 0 skips), in place."""
    lib = load_library()
    nb, bs, row_bytes = _cache_geometry(k_cache, v_cache)
    if k_rows.dtype != k_cache.dtype or v_rows.dtype != k_cache.dtype:
        raise ValueError("rows and caches must share a dtype")
    n = k_rows.shape[0]
    _check(lib, lib.paged_decode_attn_scatter_kv(
        _dev_ptr(k_rows, "k_rows"), _dev_ptr(v_rows, "v_rows"), n, row_bytes,
        _dev_ptr(slot_mapping, "slot_mapping", torch.int64), _dev_ptr(k_cache, "k_cache"),
        _dev_ptr(v_cache, "v_cache"), nb * bs, _opt_err(err), _device_of(k_cache),
        _stream_ptr(stream)))


def remap_table(block_table, lens, block_size: int, new_id, err=None, stream=None):
    """In place: every used entry e of block_table becomes new_id[e]."""
    lib = load_library()
    _check(lib, lib.paged_decode_attn_remap_table(
        _dev_ptr(block_table, "block_table", torch.int32), block_table.shape[0],
        block_table.shape[1], _dev_ptr(lens, "lens", torch.int32), int(block_size),
        _dev_ptr(new_id, "new_id", torch.int32), new_id.shape[0], _opt_err(err),
        _device_of(block_table), _stream_ptr(stream)))


# --------------------------- block-scaled FP8 caches ---------------------------
# A decode step makes these calls once a layer, and a small one is bound by the
# host: the checks of a call run over its tensors once, without helpers per tensor.

_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _refuse(name: str, t: torch.Tensor, device: int, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _pointers(device: int, named) -> list[int]:
    """Pointers of (name, tensor, dtype or None) on one device, each checked."""
    out = []
    for name, t, dtype in named:
        if t.get_device() != device or not t.is_contiguous() or (
                dtype is not None and t.dtype is not dtype):
            _refuse(name, t, device, dtype)
        out.append(t.data_ptr())
    return out


def _is_block_scale(t, num_kv_heads: int) -> bool:
    """Two dimensions and more values than heads."""
    return t is not None and t.dim() == 2 and t.numel() not in (1, num_kv_heads)


def _rows16(name: str, t: torch.Tensor, device: int, dtype) -> tuple[int, int]:
    """Pointer and token stride of [rows, heads, D] with the heads contiguous in a row."""
    if t.get_device() != device or t.dtype != dtype:
        _refuse(name, t, device, dtype)
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (H > 1 and s1 != D):
        raise ValueError(f"{name}: heads must be contiguous within a token")
    if T > 1 and s0 < H * D:
        raise ValueError(f"{name}: tokens must not overlap (a broadcast view)")
    return t.data_ptr(), (s0 if T > 1 else H * D)


# torch's current stream of a device, which need not be the current one
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _fp8_shape(k_cache, v_cache, k_scale, v_scale):
    """(num_blocks, block_size, Hkv, D) of a block-scaled FP8 cache: [num_blocks, block_size,
    Hkv, D] E4M3 bytes and [num_blocks, Hkv] fp32 scales."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_blocks, block_size, Hkv, D] alike")
    if k_cache.dtype not in _FP8 or v_cache.dtype not in _FP8:
        raise ValueError("k_cache and v_cache must be float8_e4m3fn or uint8")
    want = (shape[0], shape[2])
    if k_scale.shape != want or v_scale.shape != want:
        raise ValueError("k_scale and v_scale must be [num_blocks, Hkv]")
    return shape


def _cuda_device(t: torch.Tensor) -> int:
    device = t.get_device()
    if device < 0:
        raise ValueError("k_cache must be a CUDA tensor")
    return device


def _append_args(device, k, v, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                 cu_rows, err, stream):
    """Checks shared by the two appends; the cache and sequence arguments of the C calls."""
    nb, bs, Hkv, D = _fp8_shape(k_cache, v_cache, k_scale, v_scale)
    rows = k.shape
    if v.shape != rows or rows[1] != Hkv or rows[2] != D:
        raise ValueError("k and v must be [rows, Hkv, D] with the cache's Hkv and D")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_blocks]")
    B, width = block_table.shape
    if context_lens.shape != (B,) or cu_rows.shape != (B + 1,):
        raise ValueError("context_lens must be [batch] and cu_rows [batch + 1]")
    named = [("k_cache", k_cache, None), ("v_cache", v_cache, None),
             ("k_scale", k_scale, torch.float32), ("v_scale", v_scale, torch.float32),
             ("block_table", block_table, torch.int32),
             ("context_lens", context_lens, torch.int32), ("cu_rows", cu_rows, torch.int64)]
    if err is not None:
        if err.numel() < 2:
            raise ValueError("err must hold two int32 values")
        named.append(("err", err, torch.int32))
    ptr = _pointers(device, named)
    return (*ptr[:4], nb, bs, ptr[4], width, ptr[5], ptr[6], B,
            ptr[7] if err is not None else None, device,
            _raw_stream(device) if stream is None else _stream_ptr(stream))


def append_kv_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                  context_lens: torch.Tensor, cu_rows: torch.Tensor,
                  err: torch.Tensor | None = None, stream=None) -> None:
    """Quantise the rows of k and v and append them to a block-scaled FP8
    cache (in place: caches and scales).

    k, v [rows, Hkv, D] (bf16/fp16; token-strided views allowed), caches
    [num_blocks, block_size, Hkv, D] float8_e4m3fn or uint8, scales
    [num_blocks, Hkv] fp32, block_table [batch, max_blocks] int32. Sequence b's
    last tokens, up to context_lens[b] (int32, the new ones included), are the
    rows cu_rows[b] .. cu_rows[b + 1] - 1 (cu_rows: int64, [batch + 1]). A block
    is written for one sequence: one shared with another sequence is copied
    first (copy_blocks and, for the scales, ``scale[dst] = scale[src]``)."""
    lib = _lib or load_library()
    dt = k.dtype
    if dt not in _DT16 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("k and v must be bfloat16 or float16 [rows, heads, head_dim]")
    dev = _cuda_device(k_cache)
    kp, ks = _rows16("k", k, dev, dt)
    vp, vs = _rows16("v", v, dev, dt)
    args = _append_args(dev, k, v, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                        cu_rows, err, stream)
    T, Hkv, D = k.shape
    status = lib.paged_decode_attn_append_kv_fp8(kp, ks, vp, vs, T, Hkv, D, _DT16[dt], *args)
    if status:
        _check(lib, status)


def rope_append_kv_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       positions: torch.Tensor, cos_sin_cache: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                       v_scale: torch.Tensor, block_table: torch.Tensor,
                       context_lens: torch.Tensor, cu_rows: torch.Tensor, neox: bool = True,
                       q_out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """RoPE on q and k, then append_kv_fp8 of the rotated k and of v, in one
    launch. positions [rows] int32, cos_sin_cache [max_position, rot_dim] fp32
    (cosines then sines; angles scaled for long contexts are the table's
    matter), neox as in rope_kv_write. Returns q_out (a new tensor, or
    ``q_out``; pass ``q_out=q`` to rotate in place); its rows that belong to no
    sequence are not written."""
    lib = _lib or load_library()
    dt = q.dtype
    if dt not in _DT16 or q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be bfloat16 or float16 [rows, heads, head_dim]")
    T, Hq, D = q.shape
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError("k and v must have q's rows and head_dim")
    dev = _cuda_device(k_cache)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    if cos_sin_cache.dim() != 2:
        raise ValueError("cos_sin_cache must be [max_position, rot_dim]")
    if positions.shape != (T,):
        raise ValueError("positions must be [rows]")
    qp, qs = _rows16("q", q, dev, dt)
    kp, ks = _rows16("k", k, dev, dt)
    vp, vs = _rows16("v", v, dev, dt)
    qop, qos = (qp, qs) if q_out is q else _rows16("q_out", q_out, dev, dt)
    args = _append_args(dev, k, v, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                        cu_rows, err, stream)
    pos, cs = _pointers(dev, (("positions", positions, torch.int32),
                              ("cos_sin_cache", cos_sin_cache, torch.float32)))
    max_pos, rot_dim = cos_sin_cache.shape
    status = lib.paged_decode_attn_rope_append_kv_fp8(
        qp, qs, kp, ks, vp, vs, pos, cs, max_pos, rot_dim, 1 if neox else 0, T, Hq, k.shape[1], D,
        _DT16[dt], qop, qos, *args)
    if status:
        _check(lib, status)
    return q_out


def gather_kv_fp8(k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_rows=None,
                  max_len: int | None = None, k_out=None, v_out=None, dtype=torch.bfloat16,
                  err=None, stream=None):
    """gather_kv from a block-scaled FP8 cache: each sequence's tokens, in
    order, dequantised (scale * value) into contiguous [rows, Hkv, D] buffers
    of ``dtype`` (or k_out's): sequence b from row cu_rows[b] (int64; default:
    exclusive prefix sums of lens, computed on the host from lens). Returns
    (k_out, v_out)."""
    lib = _lib or load_library()
    nb, bs, Hkv, D = _fp8_shape(k_cache, v_cache, k_scale, v_scale)
    dev = _cuda_device(k_cache)
    if (k_out is None) != (v_out is None):
        raise ValueError("pass both k_out and v_out, or neither")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_blocks]")
    B, width = block_table.shape
    if cu_rows is None or max_len is None or k_out is None:
        lens_h = lens.cpu().to(torch.int64)
        total = int(lens_h.sum())
        if cu_rows is None:
            cu_rows = (torch.cumsum(lens_h, 0) - lens_h).to(k_cache.device)
        elif B:
            total = int((cu_rows.cpu() + lens_h).max())
        if max_len is None:
            max_len = int(lens_h.max()) if B else 0
        if k_out is None:
            k_out = torch.empty((total, Hkv, D), dtype=dtype, device=k_cache.device)
            v_out = torch.empty((total, Hkv, D), dtype=dtype, device=k_cache.device)
    if lens.shape != (B,) or cu_rows.shape != (B,):
        raise ValueError("lens and cu_rows must be [batch]")
    shape, dt = k_out.shape, k_out.dtype
    if len(shape) != 3 or shape[1:] != (Hkv, D) or v_out.shape != shape or v_out.dtype != dt:
        raise ValueError("k_out and v_out must be [rows, Hkv, D] alike")
    if dt not in _DT:
        raise ValueError("k_out and v_out must be bfloat16, float16 or float32")
    named = [("k_cache", k_cache, None), ("v_cache", v_cache, None),
             ("k_scale", k_scale, torch.float32), ("v_scale", v_scale, torch.float32),
             ("block_table", block_table, torch.int32), ("lens", lens, torch.int32),
             ("cu_rows", cu_rows, torch.int64), ("k_out", k_out, None), ("v_out", v_out, None)]
    if err is not None:
        if err.numel() < 2:
            raise ValueError("err must hold two int32 values")
        named.append(("err", err, torch.int32))
    p = _pointers(dev, named)
    status = lib.paged_decode_attn_gather_kv_fp8(
        p[0], p[1], p[2], p[3], nb, bs, Hkv, D, p[4], width, p[5], p[6], B, int(max_len), p[7],
        p[8], shape[0], _DT[dt], p[9] if err is not None else None, dev,
        _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if status:
        _check(lib, status)
    return k_out, v_out
